// Attention of one new token per sequence over every key of its paged cache (or of its last
// window of chunks):
//   s_j = q.k_j scale,  out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  m = max_j s_j,
// and log sum_j exp(s_j).
//
// Bound by HBM: every key and value is read once.  The G query heads of a KV head share each
// of them, which at G = 8 is 16 flops a byte in bf16 -- 105 TFLOP/s at the card's bandwidth,
// beyond the CUDA cores -- so the bf16 products run on the tensor cores with the keys as the
// M = 16 rows and the heads as the N = 8 columns of mma.m16n8k16.
//
// Split.  The tiles (kTile keys of one (sequence, KV head), "units") of the whole batch are
// numbered in a row, and CTA i of kDenseCtas takes units [i per, (i + 1) per): every SM reads
// the same number of bytes whatever the lengths are, and the host needs none of them (the
// launch is the same for every step, so a graph can hold it).  A (sequence, KV head) whose
// units all lie in one CTA is written by it.  One that is cut leaves partials (max, sum,
// unnormalised output) in the workspace, at most two per CTA; the CTA that takes the last
// ticket joins them in CTA order, so that the result does not depend on who that is.  No CTA
// waits for another.
//
// Within a CTA, the kTileWarps warps of group j take units j, j + kGroups, ... and feed
// themselves: they read their part of the block table 32 units at a time, and a lane of the
// group's first warp refills a stage of the group's own ring by TMA (K and V tile, 128-byte
// swizzle) as soon as the group has consumed it.  Nobody else is waited for: each warp keeps its
// own running maximum, sum and output, and the warps are joined in shared memory at the end of
// each (sequence, KV head).  (One producer warp feeding all through full and empty barriers was
// tried first: its loop took about 500 cycles a unit, which 16 KB units -- 700 cycles of the SM's
// share of HBM -- do not hide.)
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

#include "common.cuh"
#include "kernels.cuh"
#include "tc_util.cuh"

namespace hils {

namespace {

constexpr int kDenseWarps = 8;
constexpr int kDenseThreads = kDenseWarps * 32;
constexpr int kDenseCtas = 148;          // one per SM
constexpr int kDenseSeqs = 1024;         // sequences of one launch (their prefix sums in shared memory)
constexpr int kDenseRing = 128 * 1024;   // bytes of the rings of a CTA
constexpr int kDenseMaxTiles = 2;        // units of a chunk and KV head, at most
constexpr int kDenseMinUnits = 2;        // units of a CTA, at least

// T element, D head dim, G heads per KV head.
template <typename T, int D, int G>
struct DenseCfg {
  static constexpr int kTile = sizeof(T) == 2 ? 64 : 32;         // keys per unit
  static constexpr int kTileWarps = 2;                           // warps that share a unit
  static constexpr int kSlice = kTile / kTileWarps;              // keys of it that one warp takes
  static constexpr int kGroups = kDenseWarps / kTileWarps;
  static constexpr int kCols = 128 / (int)sizeof(T);             // columns of a swizzled sub-tile
  static constexpr int kSubs = D / kCols;
  static constexpr uint32_t kSub = kTile * 128u;                 // bytes of a sub-tile
  static constexpr uint32_t kHalf = kSubs * kSub;                // K (or V) of a stage
  static constexpr uint32_t kStage = 2 * kHalf;
  static constexpr int kStages = kDenseRing / kGroups / (int)kStage;  // of a group
  static constexpr int kVec = G * D / 4;                         // float4 columns of an output
  // shared memory behind the rings, in floats
  static constexpr int kJoin = kDenseWarps * G * D > 2560 ? kDenseWarps * G * D : 2560;
  static constexpr int kQ = sizeof(T) == 4 ? G * D : 0;
  static constexpr int kP = sizeof(T) == 4 ? kDenseWarps * 16 * G : 0;
  static constexpr uint32_t kRings = kGroups * kStages * kStage;
  static constexpr size_t kSmem = 1024 + (size_t)kRings + 4ull * (kJoin + kQ + kP);
  static_assert(kStages >= 1 && kSmem <= 227 * 1024 - 10 * 1024, "room for the static shared variables");
};

struct alignas(64) DenseKernelArgs {
  CUtensorMap tmap_k, tmap_v;  // pages as [P g][B][D], boxes of kCols columns and kTile rows
  DenseArgs a;                 // of this launch's sequences
  float* part;                 // [2 kDenseCtas][G D]
  float2* part_ml;             // [2 kDenseCtas][G]
  unsigned* ticket;            // [b g], zero between calls
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// c += a b: a 16 x 16 (row), b 16 x 8 (col), bf16 with fp32 sums.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float4 lds4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float2 lds2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// Running softmax of one warp over its keys, logits in units of log 2: one step of a maximum.
// Returns the factor of what was summed so far; base is the finite number to subtract.
__device__ __forceinline__ float raise_max(float& m, float t, float& base) {
  const float mn = fmaxf(m, t);
  base = mn == -INFINITY ? 0.f : mn;  // only -inf so far: every exp2 below is 0
  const float c = exp2f(m - base);
  m = mn;
  return c;
}

// bf16: the warp's state over its slices of 16 NS keys.  Lane l holds heads 2 (l % 4), + 1, as the
// columns of the transposed score tile S^T = K Q^T and of O^T = V^T P^T.  P is split into
// bf16 hi + lo parts (two products), so that its rounding (2^-17) stays below that of the
// output; the tensor cores have the room at this byte rate.
template <int D, int G, int NS>
struct WarpStateBf16 {
  float m[2], l[2], o[D / 16][4];
  uint32_t q[D / 16][2];

  __device__ void start(const DenseArgs& a, int bi, int gi, float*, int lane, int) {
    const int hh = lane >> 2;
    const uint32_t* row = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                            ((size_t)bi * a.h + gi * G + hh) * D);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      q[k][0] = hh < G ? __ldg(row + k * 8 + (lane & 3)) : 0u;
      q[k][1] = hh < G ? __ldg(row + k * 8 + 4 + (lane & 3)) : 0u;
      o[k][0] = o[k][1] = o[k][2] = o[k][3] = 0.f;
    }
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }

  // Keys [row0, row0 + 16 NS) of a tile with `valid` keys (> row0): NS 16-key products side by
  // side, one step of the running maximum for all.
  __device__ void consume(uint32_t sk, uint32_t sv, int row0, int valid, float scale, const float*, float*, int lane) {
    constexpr uint32_t kSub = DenseCfg<__nv_bfloat16, D, G>::kSub;
    float s[NS][4];
#pragma unroll
    for (int i = 0; i < NS; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        uint32_t f[4];
        ldsm4(sk + (k >> 2) * kSub + tc::sw128_chunk(row0 + 16 * i + (lane & 15), (k & 3) * 2 + (lane >> 4)), f);
        mma16816(s[i], f, q[k][0], q[k][1]);
      }
    }
    // s[i]: keys r, r (heads 2c, 2c + 1), r + 8, r + 8, r = row0 + 16 i + lane / 4
    float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool ok = row0 + 16 * i + 8 * e + (lane >> 2) < valid;
        s[i][2 * e] = ok ? s[i][2 * e] * scale : -INFINITY;
        s[i][2 * e + 1] = ok ? s[i][2 * e + 1] * scale : -INFINITY;
        t0 = fmaxf(t0, s[i][2 * e]);
        t1 = fmaxf(t1, s[i][2 * e + 1]);
      }
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, d));
      t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, d));
    }
    float b0, b1;
    const float c0 = raise_max(m[0], t0, b0), c1 = raise_max(m[1], t1, b1);
    l[0] *= c0;
    l[1] *= c1;
    if (__any_sync(0xffffffffu, c0 != 1.f || c1 != 1.f)) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        o[k][0] *= c0; o[k][1] *= c1; o[k][2] *= c0; o[k][3] *= c1;
      }
    }
    // P^T as the second operand: bf16 hi and lo parts of keys (0-7, 8-15) of each slice
    uint32_t ph[NS][2], pl[NS][2], keep[NS][2];
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float p0 = exp2f(s[i][2 * e] - b0), p1 = exp2f(s[i][2 * e + 1] - b1);
        l[0] += p0;
        l[1] += p1;
        const uint32_t h = tc::pack_bf16x2(p0, p1);
        ph[i][e] = transpose8(h);
        pl[i][e] = transpose8(tc::pack_bf16x2(p0 - __uint_as_float(h << 16), p1 - __uint_as_float(h & 0xffff0000u)));
        // values behind the last key may be anything: they are cleared, not only weighted by 0
        const int k0 = row0 + 16 * i + 8 * e + (lane & 3) * 2;
        keep[i][e] = (k0 < valid ? 0xffffu : 0u) | (k0 + 1 < valid ? 0xffff0000u : 0u);
      }
    const bool tail = row0 + 16 * NS > valid;
    const uint32_t vrow = row0 + (lane & 7) + ((lane >> 4) << 3), vch = (lane >> 3) & 1;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        uint32_t f[4];
        ldsm4_t(sv + (k >> 2) * kSub + tc::sw128_chunk(vrow + 16 * i, (k & 3) * 2 + vch), f);
        if (tail) {
          f[0] &= keep[i][0]; f[1] &= keep[i][0]; f[2] &= keep[i][1]; f[3] &= keep[i][1];
        }
        mma16816(o[k], f, ph[i][0], ph[i][1]);
        mma16816(o[k], f, pl[i][0], pl[i][1]);
      }
    }
  }

  // so [G][D], sm and sl [G]: this warp's place in shared memory
  __device__ void finish(float* so, float* sm, float* sl, int lane) {
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], d);
      l[1] += __shfl_xor_sync(0xffffffffu, l[1], d);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int hh = (lane & 3) * 2 + e;
      if (hh < G) {
        if (lane < 4) {
          sm[hh] = m[e];
          sl[hh] = l[e];
        }
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          so[hh * D + k * 16 + (lane >> 2)] = o[k][e];
          so[hh * D + k * 16 + 8 + (lane >> 2)] = o[k][2 + e];
        }
      }
    }
  }
};

// fp32: CUDA cores.  For the scores lane l takes keys pr and pr + 8 of the slice, pr a
// permutation of l / 4 that keeps the swizzled 16-byte reads free of bank conflicts, and the
// quarter l % 4 of the head; for the output it owns D / 32 adjacent columns of every head.
template <int D, int G>
struct WarpStateF32 {
  static constexpr int kCpl = D / 32;
  float m[G], l[G], o[G][kCpl];

  __device__ void start(const DenseArgs& a, int bi, int gi, float* sq, int, int ct) {
    const float* row = static_cast<const float*>(a.q) + ((size_t)bi * a.h + gi * G) * D;
    for (int x = ct; x < G * D; x += kDenseThreads) sq[x] = __ldg(row + x);
    __syncthreads();
#pragma unroll
    for (int hh = 0; hh < G; ++hh) {
      m[hh] = -INFINITY;
      l[hh] = 0.f;
#pragma unroll
      for (int x = 0; x < kCpl; ++x) o[hh][x] = 0.f;
    }
  }

  // Keys [row0, row0 + 16) of a tile with `valid` keys (> row0).
  __device__ void consume(uint32_t sk, uint32_t sv, int row0, int valid, float scale, const float* sq, float* sp,
                          int lane) {
    constexpr uint32_t kSub = DenseCfg<float, D, G>::kSub;
    const int rr = lane >> 2, c = lane & 3;
    const int pr = ((rr & 1) << 2) | (rr >> 1);
    float sa[G], sb[G];
#pragma unroll
    for (int hh = 0; hh < G; ++hh) sa[hh] = sb[hh] = 0.f;
#pragma unroll 4
    for (int i = 0; i < D / 16; ++i) {
      const uint32_t base = sk + (i >> 1) * kSub, j = c + 4 * (i & 1);
      const float4 ka = lds4(base + tc::sw128_chunk(row0 + pr, j)), kb = lds4(base + tc::sw128_chunk(row0 + 8 + pr, j));
#pragma unroll
      for (int hh = 0; hh < G; ++hh) {
        const float4 q = *reinterpret_cast<const float4*>(sq + hh * D + (c + 4 * i) * 4);
        sa[hh] = fmaf(q.x, ka.x, fmaf(q.y, ka.y, fmaf(q.z, ka.z, fmaf(q.w, ka.w, sa[hh]))));
        sb[hh] = fmaf(q.x, kb.x, fmaf(q.y, kb.y, fmaf(q.z, kb.z, fmaf(q.w, kb.w, sb[hh]))));
      }
    }
#pragma unroll
    for (int hh = 0; hh < G; ++hh) {
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        sa[hh] += __shfl_xor_sync(0xffffffffu, sa[hh], d);
        sb[hh] += __shfl_xor_sync(0xffffffffu, sb[hh], d);
      }
      const float xa = row0 + pr < valid ? sa[hh] * scale : -INFINITY;
      const float xb = row0 + 8 + pr < valid ? sb[hh] * scale : -INFINITY;
      float t = fmaxf(xa, xb), base;
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
      const float f = raise_max(m[hh], t, base);
      const float pa = exp2f(xa - base), pb = exp2f(xb - base);
      l[hh] = l[hh] * f + (pa + pb);
#pragma unroll
      for (int x = 0; x < kCpl; ++x) o[hh][x] *= f;
      if ((hh & 3) == c) {
        sp[pr * G + hh] = pa;
        sp[(8 + pr) * G + hh] = pb;
      }
    }
    __syncwarp();
    const int nk = min(16, valid - row0);  // the values behind the last key are not read
    const uint32_t piece = lane * kCpl / 4;
    const uint32_t vb = sv + (piece >> 3) * kSub + (lane * kCpl % 4) * 4;
#pragma unroll 4
    for (int j = 0; j < nk; ++j) {
      const uint32_t addr = vb + tc::sw128_chunk(row0 + j, piece & 7);
      float v[kCpl];
      if constexpr (kCpl == 4) {
        const float4 x = lds4(addr);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
      } else {
        const float2 x = lds2(addr);
        v[0] = x.x; v[1] = x.y;
      }
#pragma unroll
      for (int hh = 0; hh < G; ++hh) {
        const float p = sp[j * G + hh];
#pragma unroll
        for (int x = 0; x < kCpl; ++x) o[hh][x] = fmaf(p, v[x], o[hh][x]);
      }
    }
    __syncwarp();
  }

  __device__ void finish(float* so, float* sm, float* sl, int lane) {
#pragma unroll
    for (int hh = 0; hh < G; ++hh) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], d);
      if (lane == 0) {
        sm[hh] = m[hh];
        sl[hh] = l[hh];
      }
#pragma unroll
      for (int x = 0; x < kCpl; ++x) so[hh * D + lane * kCpl + x] = o[hh][x];
    }
  }
};

template <typename T, int D, int G> struct WarpState;
template <int D, int G>
struct WarpState<__nv_bfloat16, D, G> : WarpStateBf16<D, G, DenseCfg<__nv_bfloat16, D, G>::kSlice / 16> {};
template <int D, int G> struct WarpState<float, D, G> : WarpStateF32<D, G> {};

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(tc::pack_bf16x2(v.x, v.y), tc::pack_bf16x2(v.z, v.w));
}

// First tile that the new token attends to, and the tiles from there on, for L keys.
template <int kTile>
__device__ __forceinline__ int first_tile(int L, int n_win) {
  if (n_win == 0 || L <= 0) return 0;
  return max(0, (L - 1) / kChunk + 1 - n_win) * (kChunk / kTile);
}
template <int kTile>
__device__ __forceinline__ int n_tiles(int L, int n_win) {
  return L <= 0 ? 0 : (L - 1) / kTile + 1 - first_tile<kTile>(L, n_win);
}

// The sequence whose units hold u: the last b with prefix[b] <= u (and units of its own).
__device__ __forceinline__ int seq_of(const unsigned* prefix, int n, unsigned u) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= u) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace

template <typename T, int D, int G>
__global__ void __launch_bounds__(kDenseThreads, 1) decode_dense_kernel(const __grid_constant__ DenseKernelArgs ka) {
  using C = DenseCfg<T, D, G>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ unsigned s_prefix[kDenseSeqs + 1];  // units before each sequence
  __shared__ int s_len[kDenseSeqs];
  __shared__ __align__(16) unsigned s_scan[kDenseWarps];
  __shared__ uint64_t s_full[C::kGroups][C::kStages];
  __shared__ float s_m[kDenseWarps][G], s_l[kDenseWarps][G], s_M[G], s_z[G];
  __shared__ int s_abort, s_last;

  const DenseArgs& a = ka.a;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const uint32_t ring0 = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
  const int group = warp / C::kTileWarps, row0 = warp % C::kTileWarps * C::kSlice;
  const bool feeds = warp % C::kTileWarps == 0;  // the group's first warp issues its copies
  const uint32_t ring = ring0 + group * C::kStages * C::kStage;
  float* s_join = reinterpret_cast<float*>(smem_raw + (ring0 - tc::smem_u32(smem_raw)) + C::kRings);
  float* s_q = s_join + C::kJoin;
  float* s_p = s_q + C::kQ + warp * 16 * G;

  if (feeds && lane == 0) {
    for (int s = 0; s < C::kStages; ++s) tc::mbar_init(tc::smem_u32(&s_full[group][s]), 1);
    tc::mbar_fence_init();
  }
  if (t == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&ka.tmap_k) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&ka.tmap_v) : "memory");
    s_abort = 0;
    s_prefix[0] = 0;
  }
  {  // units before each sequence: thread t counts sequences 4 t .. 4 t + 3
    constexpr int kPer = kDenseSeqs / kDenseThreads;
    unsigned mine[kPer], sum = 0;
    const long long cap = (long long)a.max_chunks * kChunk;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = t * kPer + i;
      int L = b < a.b ? a.seq_lens[b] : 0;
      if (L > cap) {
        if (blockIdx.x == 0) set_error(a.err, kErrBadPage);
        L = (int)cap;
      }
      s_len[b] = L;
      sum += (unsigned)n_tiles<C::kTile>(L, a.n_win) * (unsigned)a.g;
      mine[i] = sum;
    }
    unsigned inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += y;
    }
    if (lane == 31) s_scan[warp] = inc;
    sum = inc - sum;  // before this thread, within the warp
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kDenseWarps; ++w) sum += w < warp ? s_scan[w] : 0u;
#pragma unroll
    for (int i = 0; i < kPer; ++i) s_prefix[t * kPer + i + 1] = sum + mine[i];
  }
  __syncthreads();
  const unsigned total = s_prefix[a.b];
  const unsigned per = max((unsigned)kDenseMinUnits, (total + kDenseCtas - 1) / kDenseCtas);
  const unsigned u0 = min(total, blockIdx.x * per), u1 = min(total, u0 + per);

  // The group's units: number i is unit u0 + group + kGroups i.  Lane j knows the place of number
  // base + j (z: block of the pool, -1 for a bad page; y: row in it) and of the 32 after those.
  auto locate = [&](unsigned i, int& y, int& z) {
    const unsigned u = u0 + group + i * C::kGroups;
    z = -1;
    y = 0;
    if (u >= u1) return;
    const int b = seq_of(s_prefix, a.b, u);
    const int L = s_len[b];
    const int nt = n_tiles<C::kTile>(L, a.n_win);
    const int rem = (int)(u - s_prefix[b]);
    const int tile = first_tile<C::kTile>(L, a.n_win) + rem % nt;
    const int page = a.block_table[(size_t)b * a.max_chunks + tile * C::kTile / kChunk];
    y = tile * C::kTile % kChunk;
    if (page >= 0 && page < a.n_pages) z = page * a.g + rem / nt;
    else set_error(a.err, kErrBadPage);
  };
  const unsigned mine = u0 + group < u1 ? (u1 - u0 - group + C::kGroups - 1) / C::kGroups : 0;
  unsigned issued = 0, base = 0, bad = 0;  // bad: bit s, stage s has no page
  int y, z, yn = 0, zn = -1;
  locate(lane, y, z);
  if (mine > 32) locate(32 + lane, yn, zn);
  auto issue = [&]() {  // the next unit's copies (every lane of the group calls it)
    if (issued - base == 32) {
      base += 32;
      y = yn;
      z = zn;
      if (base + 32 < mine) locate(base + 32 + lane, yn, zn);
    }
    const int yi = __shfl_sync(0xffffffffu, y, issued - base), zi = __shfl_sync(0xffffffffu, z, issued - base);
    const int st = (int)(issued % C::kStages);
    bad = zi < 0 ? bad | 1u << st : bad & ~(1u << st);
    if (feeds && lane == 0 && zi >= 0) {
      const uint32_t full = tc::smem_u32(&s_full[group][st]), dst = ring + st * C::kStage;
      tc::fence_async_smem();  // the stage's last reads, before the copies into it
      tc::mbar_arrive_expect_tx(full, C::kStage);
#pragma unroll
      for (int s = 0; s < C::kSubs; ++s) {
        tc::tma_load_3d(dst + s * C::kSub, &ka.tmap_k, s * C::kCols, yi, zi, full);
        tc::tma_load_3d(dst + C::kHalf + s * C::kSub, &ka.tmap_v, s * C::kCols, yi, zi, full);
      }
    }
    ++issued;
  };
  while (issued < mine && issued < (unsigned)C::kStages) issue();
  unsigned phases = 0;  // bit s: parity of the next fill of stage s to wait for

  auto group_sync = [&]() {
    if constexpr (C::kTileWarps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(C::kTileWarps * 32) : "memory");
  };

  T* out = static_cast<T*>(a.out);
  // sequences without keys
  for (int b = blockIdx.x; b < a.b; b += kDenseCtas) {
    if (s_len[b] > 0) continue;
    for (int x = t; x < a.h * D / 4; x += kDenseThreads)
      store4(out + (size_t)b * a.h * D + x * 4, make_float4(0.f, 0.f, 0.f, 0.f));
    if (a.lse)
      for (int x = t; x < a.h; x += kDenseThreads) a.lse[(size_t)b * a.h + x] = -INFINITY;
  }
  const float scale = a.scale * 1.4426950408889634f;  // logits in units of log 2
  bool failed = false;

  // Writes head hh's columns [col, col + 4) and, once per head, its log-sum-exp.
  auto write_row = [&](int bi, int gi, int x, float4 acc, float M, float z) {
    const int hh = x * 4 / D;
    const size_t row = (size_t)bi * a.h + gi * G + hh;
    const float inv = z == 0.f ? 0.f : 1.f / z;  // no key with a finite logit: a zero row
    acc.x *= inv; acc.y *= inv; acc.z *= inv; acc.w *= inv;
    store4(out + row * D + x * 4 % D, acc);
    if (a.lse && x * 4 % D == 0) a.lse[row] = z == 0.f ? -INFINITY : (M + log2f(z)) * 0.69314718055994531f;
  };

  int bi = u0 < u1 ? seq_of(s_prefix, a.b, u0) : 0;
  unsigned i = 0, stuck = 0;  // the group's next unit; the one this warp gave up at
  for (unsigned u = u0; u < u1;) {
    while (s_prefix[bi + 1] <= u) ++bi;
    const int L = s_len[bi], nt = n_tiles<C::kTile>(L, a.n_win), t0 = first_tile<C::kTile>(L, a.n_win);
    const int gi = (int)(u - s_prefix[bi]) / nt;
    const unsigned seg0 = s_prefix[bi] + (unsigned)gi * nt, seg1 = seg0 + nt;
    const unsigned ue = min(u1, seg1);
    WarpState<T, D, G> w;
    w.start(a, bi, gi, s_q, lane, t);
    for (unsigned v = u0 + group + i * C::kGroups; v < ue; v += C::kGroups, ++i) {
      const int st = (int)(i % C::kStages);
      if (!failed && !(bad >> st & 1u)) {
        // a warp that gives up goes on meeting the barriers below
        if (__all_sync(0xffffffffu, tc::mbar_wait(tc::smem_u32(&s_full[group][st]), phases >> st & 1u, a.poll))) {
          phases ^= 1u << st;
          const int valid = min(C::kTile, L - (t0 + (int)(v - seg0)) * C::kTile);
          const uint32_t sk = ring + st * C::kStage;
          if (row0 < valid) w.consume(sk, sk + C::kHalf, row0, valid, scale, s_q, s_p, lane);
        } else {
          failed = true;
          stuck = i;
        }
      }
      if (i + C::kStages < mine) {  // refill the stage once the group is done with it
        group_sync();
        if (!failed) issue();
      }
    }
    if (failed && lane == 0) {
      set_error(a.err, kErrTimeout);
      s_abort = 1;
    }
    // join the warps
    w.finish(s_join + warp * G * D, s_m[warp], s_l[warp], lane);
    __syncthreads();
    const bool whole = u == seg0 && ue == seg1;
    const bool aborted = s_abort != 0;
    const int slot = 2 * blockIdx.x + (seg0 >= u0 ? 1 : 0);
    if (t < C::kVec) {
      const int hh = t * 4 / D;
      float M = -INFINITY, z = 0.f;
#pragma unroll
      for (int k = 0; k < kDenseWarps; ++k) M = fmaxf(M, s_m[k][hh]);
      const float base = M == -INFINITY ? 0.f : M;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kDenseWarps; ++k) {
        const float e = exp2f(s_m[k][hh] - base);
        const float4 x = *reinterpret_cast<const float4*>(s_join + k * G * D + t * 4);
        z = fmaf(e, s_l[k][hh], z);
        acc.x = fmaf(e, x.x, acc.x); acc.y = fmaf(e, x.y, acc.y);
        acc.z = fmaf(e, x.z, acc.z); acc.w = fmaf(e, x.w, acc.w);
      }
      if (whole) {
        if (!aborted) write_row(bi, gi, t, acc, M, z);
      } else {
        __stcg(reinterpret_cast<float4*>(ka.part + (size_t)slot * G * D) + t, acc);
        // NaN as the maximum (which is never one) marks a part that was given up
        if (t * 4 % D == 0) __stcg(ka.part_ml + (size_t)slot * G + hh, make_float2(aborted ? NAN : M, z));
      }
    }
    __syncthreads();  // the warps' places are free again, and the partial is written
    if (!whole) {
      const int first = (int)(seg0 / per), last = (int)((seg1 - 1) / per), n = last - first + 1;
      if (t == 0) {
        __threadfence();  // the CTA's partial, ordered before by the barrier, is visible before the ticket
        // counts n - 1 up to itself and starts again at 0: ready for the next call
        s_last = atomicInc(ka.ticket + (size_t)bi * a.g + gi, (unsigned)(n - 1)) == (unsigned)(n - 1);
        __threadfence();
      }
      __syncthreads();
      if (s_last) {
        // part j of the segment: slot 1 of the CTA where it begins, slot 0 of the others
        auto slot_of = [&](int j) { return (size_t)(2 * (first + j) + (j == 0 ? 1 : 0)); };
        // kNp threads share a float4 column: each sums every kNp-th part, then they are joined.
        // The first kFirst parts are on their way while the weights are computed.
        constexpr int kNp = kDenseThreads / C::kVec, kFirst = 4;
        const int v = t % C::kVec, np = t / C::kVec, hv = v * 4 / D;
        auto part_at = [&](int j) { return __ldcg(reinterpret_cast<const float4*>(ka.part + slot_of(j) * G * D) + v); };
        float4 x[kFirst];
#pragma unroll
        for (int i = 0; i < kFirst; ++i)
          x[i] = np + i * kNp < n ? part_at(np + i * kNp) : make_float4(0.f, 0.f, 0.f, 0.f);
        bool gone = false;
        if (warp < G) {
          constexpr int kMl = (kDenseCtas + 31) / 32;
          float2 ml[kMl];
          float M = -INFINITY, z = 0.f;
#pragma unroll
          for (int i = 0; i < kMl; ++i) {
            ml[i] = lane + 32 * i < n ? __ldcg(ka.part_ml + slot_of(lane + 32 * i) * G + warp) : make_float2(-INFINITY, 0.f);
            gone |= ml[i].x != ml[i].x;
            M = fmaxf(M, ml[i].x);
          }
          M = warp_max(M);
          const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
          for (int i = 0; i < kMl; ++i) {
            const float e = exp2f(ml[i].x - base);
            if (lane + 32 * i < n) s_join[warp * n + lane + 32 * i] = e;
            z = fmaf(e, ml[i].y, z);
          }
          z = warp_sum(z);
          if (lane == 0) {
            s_M[warp] = M;
            s_z[warp] = z;
          }
        }
        if (gone) s_abort = 1;
        __syncthreads();
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](const float4& y, int j) {
          const float e = s_join[hv * n + j];
          acc.x = fmaf(e, y.x, acc.x); acc.y = fmaf(e, y.y, acc.y);
          acc.z = fmaf(e, y.z, acc.z); acc.w = fmaf(e, y.w, acc.w);
        };
#pragma unroll
        for (int i = 0; i < kFirst; ++i)
          if (np + i * kNp < n) add(x[i], np + i * kNp);
#pragma unroll 8
        for (int j = np + kFirst * kNp; j < n; j += kNp) add(part_at(j), j);
        if constexpr (kNp > 1) {
          float4* sj = reinterpret_cast<float4*>(s_join + 1536);  // behind the weights: G n <= 1184
          sj[np * C::kVec + v] = acc;
          __syncthreads();
          if (np == 0) {
#pragma unroll
            for (int k = 1; k < kNp; ++k) {
              const float4 y = sj[k * C::kVec + v];
              acc.x += y.x; acc.y += y.y; acc.z += y.z; acc.w += y.w;
            }
          }
        }
        if (np == 0 && !s_abort) write_row(bi, gi, v, acc, s_M[hv], s_z[hv]);
        __syncthreads();
      }
    }
    u = ue;
  }
  // A feeding warp that gave up has copies in flight (units stuck .. issued - 1): they land before
  // the CTA can end.
  if (feeds && failed)
    for (; stuck < issued; ++stuck) {
      const int st = (int)(stuck % C::kStages);
      if (!(bad >> st & 1u)) tc::mbar_wait(tc::smem_u32(&s_full[group][st]), phases >> st & 1u, kDrainPolls);
    }
}

// ---- host -------------------------------------------------------------------
static PFN_cuTensorMapEncodeTiled_v12000 dense_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Pages [P g][B][D] as a rank-3 map with boxes of one 128-byte sub-tile column and `rows` rows.
static bool encode_pages_map(CUtensorMap* m, const void* base, int D, long long blocks, bool bf16, int rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = dense_map_encoder();
  if (!enc) return false;
  const cuuint64_t es = bf16 ? 2 : 4;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)kChunk, (cuuint64_t)blocks};
  const cuuint64_t strides[2] = {D * es, kChunk * D * es};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / es), (cuuint32_t)rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, int G>
static cudaError_t launch_dense(const DenseKernelArgs& ka, cudaStream_t st) {
  using C = DenseCfg<T, D, G>;
  static std::atomic<unsigned long long> ready{0};  // devices whose attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev > 63 || !(ready.load() & bit)) {
    e = cudaFuncSetAttribute(decode_dense_kernel<T, D, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev <= 63) ready.fetch_or(bit);
  }
  decode_dense_kernel<T, D, G><<<kDenseCtas, kDenseThreads, C::kSmem, st>>>(ka);
  return cudaGetLastError();
}

template <typename T, int D>
static cudaError_t launch_dense_g(const DenseKernelArgs& ka, cudaStream_t st) {
  switch (ka.a.h / ka.a.g) {
    case 1: return launch_dense<T, D, 1>(ka, st);
    case 2: return launch_dense<T, D, 2>(ka, st);
    case 4: return launch_dense<T, D, 4>(ka, st);
    case 8: return launch_dense<T, D, 8>(ka, st);
  }
  return cudaErrorInvalidValue;
}

// Units are counted in 32 bits, and the pool's blocks are a TMA coordinate.
bool decode_dense_supported(int g, int max_chunks, int n_pages) {
  return (long long)kDenseMaxTiles * g * max_chunks < (1ll << 31) && (long long)n_pages * g < (1ll << 31);
}
DenseScratch decode_dense_scratch(int b, int h, int g, int d) {
  DenseScratch s;
  const size_t G = h / g;
  s.part = 0;
  s.part_ml = 2ull * kDenseCtas * G * d * 4;
  s.ticket = s.part_ml + 2ull * kDenseCtas * G * 8;
  s.total = s.ticket + 4ull * (b < kDenseSeqs ? b : kDenseSeqs) * g;
  return s;
}

cudaError_t run_decode_dense(const DenseArgs& a, void* scratch, cudaStream_t st) {
  const DenseScratch S = decode_dense_scratch(a.b, a.h, a.g, a.d);
  const size_t es = a.bf16 ? 2 : 4;
  DenseKernelArgs ka;
  const int rows = a.bf16 ? DenseCfg<__nv_bfloat16, 64, 1>::kTile : DenseCfg<float, 64, 1>::kTile;
  if (!encode_pages_map(&ka.tmap_k, a.k_pages, a.d, (long long)a.n_pages * a.g, a.bf16, rows) ||
      !encode_pages_map(&ka.tmap_v, a.v_pages, a.d, (long long)a.n_pages * a.g, a.bf16, rows))
    return cudaErrorInvalidValue;
  char* w = static_cast<char*>(scratch);
  ka.part = reinterpret_cast<float*>(w + S.part);
  ka.part_ml = reinterpret_cast<float2*>(w + S.part_ml);
  ka.ticket = reinterpret_cast<unsigned*>(w + S.ticket);
  // sequences of one launch: their prefix sums fit shared memory, their units 32 bits
  const long long fit = ((1ll << 31) - 1) / ((long long)kDenseMaxTiles * a.g * a.max_chunks);
  const int step = (int)(fit < kDenseSeqs ? fit : kDenseSeqs);
  for (int b0 = 0; b0 < a.b; b0 += step) {
    ka.a = a;
    ka.a.b = a.b - b0 < step ? a.b - b0 : step;
    ka.a.q = static_cast<const char*>(a.q) + (size_t)b0 * a.h * a.d * es;
    ka.a.out = static_cast<char*>(a.out) + (size_t)b0 * a.h * a.d * es;
    ka.a.lse = a.lse ? a.lse + (size_t)b0 * a.h : nullptr;
    ka.a.block_table = a.block_table + (size_t)b0 * a.max_chunks;
    ka.a.seq_lens = a.seq_lens + b0;
    cudaError_t e;
    if (a.bf16)
      e = a.d == 64 ? launch_dense_g<__nv_bfloat16, 64>(ka, st) : launch_dense_g<__nv_bfloat16, 128>(ka, st);
    else
      e = a.d == 64 ? launch_dense_g<float, 64>(ka, st) : launch_dense_g<float, 128>(ka, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace hils
