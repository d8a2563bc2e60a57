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
// Split.  The tiles (kTile keys of one (sequence, KV head), "units", 16 KB of K and V each) of
// the whole batch are numbered in a row.  CTA i of kDenseCtas takes units [i per, (i + 1) per),
// and each of its warps an equal run of those: every SM reads the same number of bytes whatever
// the lengths are, and the host needs none of them (the launch is the same for every step, so a
// graph can hold it).  A warp writes the (sequence, KV head)s that lie in its run; of those that
// are cut -- at most two of a warp -- it leaves partials (max, sum, unnormalised output) in
// shared memory, which the CTA joins when its warps are done.  A (sequence, KV head) that is cut
// between CTAs -- at most two of a CTA -- leaves a partial in the workspace, and the CTA that
// takes the last ticket joins them (in two steps where there are many).  Partials are joined in
// the order of the keys, so that the result does not depend on who comes last.  Nobody waits
// for another CTA.
//
// A warp feeds itself: it reads its part of the block table 32 units at a time, and its lane 0
// refills the stages of the warp's ring by TMA (128-byte swizzle) as soon as the warp has
// consumed them.  What was tried before: one producer warp and full and empty barriers (its loop
// took about 500 cycles a unit; a 16 KB unit is 700 cycles of the SM's share of HBM), and units
// dealt to the warps in turn, joined at the end of every (sequence, KV head) (about 2 us each,
// which batches of short sequences do not hide).
//
// Measured (events around graphs of 20 calls, caches beyond L2, bf16): 8 sequences of 32K, 16
// heads of 64, 164 us (1.07 GB, 6.6 TB/s); 33 sequences of 0 to 16K, 32 heads over 8 of 128,
// 171 us (1.13 GB, 6.6 TB/s); one of 512K, the same heads, 311 us (2.15 GB, 6.9 TB/s); 64 of up
// to 2K 51 us (5.4 TB/s); one of 1013 tokens 7.1 us, a chain of latencies: lengths, block
// table, copy, one unit's products, ticket, join.  The tensor pipe is 10 to 15% busy.  fp32 with
// one head or few per KV head reads at 6.1 to 6.6 TB/s.  With eight (262K of 2 KV heads: 61 us at
// d = 64, 4.4 TB/s, and 111 us at d = 128, 4.8 TB/s) no pipe is full -- FMA 32%, shared memory 41
// to 49%, an instruction in 47% of the cycles -- but a warp has no copy on its way while it
// computes, and two warps per scheduler do not cover that.
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
constexpr int kDenseMaxTiles = 4;        // units of a chunk and KV head, at most
// Units of a CTA, at least: more SMs for a short context read it sooner and then join more parts.
// Over fifteen short shapes (100 to 32K tokens, 1 to 16 KV heads, both types) 8% more time with 1,
// 6% with 2, 9% with 8: 100 tokens, 8 KV heads of 128: 6.6, 6.2, 4.7 (4), 5.8 us; 1013 of them
// 6.9, 6.9, 7.1, 8.1; 8K, one head of 64: 9.2, 8.9, 7.6, 8.0; window of 512 over 7 sequences 8.5,
// 8.5, 8.6, 9.5.
constexpr int kDenseMinUnits = 4;
// Partials joined in one step, one per lane; more (one KV head over up to 148 SMs) are joined in
// blocks of kJoinBlock first, by different SMs (262K of one KV head, 8 heads of 128: 37 us with
// all 148 parts read by one SM, 32 us so).
constexpr int kJoinMost = 32;
constexpr int kJoinBlock = 13;

// Bytes of a warp's ring: one unit.  Eight warps have 128 KB in flight, which reaches the card's
// read rate; more does not fit beside the partials.  Two units of 8 KB in it are 3% slower over ten
// shapes (32K of 16 heads: 164 and 169 us; 64 sequences up to 2K: 51 and 55), one of them (64 KB
// in flight) 8% (164 and 173, 512K: 313 and 352 us).
constexpr int kDenseRing = 16 * 1024;

// T element, D head dim, G heads per KV head.
template <typename T, int D, int G>
struct DenseCfg {
  static constexpr int kTile = 8192 / (D * (int)sizeof(T));      // keys per unit: 64, 32 (bf16), 32, 16 (fp32)
  static constexpr int kCols = 128 / (int)sizeof(T);             // columns of a swizzled sub-tile
  static constexpr int kSubs = D / kCols;
  static constexpr uint32_t kSub = kTile * 128u;                 // bytes of a sub-tile
  static constexpr uint32_t kHalf = kSubs * kSub;                // K (or V) of a stage
  static constexpr uint32_t kStage = 2 * kHalf;
  static constexpr int kStages = kDenseRing / (int)kStage;
  static constexpr int kVec = G * D / 4;                         // float4 columns of an output
  static constexpr uint32_t kRings = kDenseWarps * kDenseRing;
  // shared memory behind the rings, in floats
  static constexpr int kHeads = kDenseWarps * G * D;             // the warps' first partials (see slot_of)
  static constexpr int kWeights = G * kJoinMost;
  static constexpr int kSums = kDenseThreads * 4;
  static constexpr int kQ = sizeof(T) == 4 ? G * D : 0;          // per warp: queries and weights of the fp32 path
  static constexpr int kP = sizeof(T) == 4 ? (kTile + 4) * G : 0;
  static constexpr size_t kSmem = 1024 + (size_t)kRings + 4ull * (kHeads + kWeights + kSums + kDenseWarps * (kQ + kP));
  static_assert(kStages >= 1 && kTile % 16 == 0 && G * D * 4 <= kDenseRing, "a unit fills a stage, an output fits one");
};

struct alignas(64) DenseKernelArgs {
  CUtensorMap tmap_k, tmap_v;  // pages as [P g][B][D], boxes of kCols columns and kTile rows
  DenseArgs a;                 // of this launch's sequences
  float* part;                 // [2 kDenseCtas][G D]
  float2* part_ml;             // [2 kDenseCtas][G]
  unsigned* block_ticket;      // [2 kDenseCtas], zero between calls
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

// 1 / z, and log sum exp from the maximum (in units of log 2) and the sum; a row that no finite
// logit reached has z = 0 and becomes zero, -inf.
__device__ __forceinline__ float inverse_sum(float z) { return z == 0.f ? 0.f : 1.f / z; }
__device__ __forceinline__ float log_sum(float m, float z) {
  return z == 0.f ? -INFINITY : (m + log2f(z)) * 0.69314718055994531f;
}

// A weight p >= 0 as three bf16 parts, cut and not rounded: the leading 8 bits, the 8 after
// them, the rest.  Together they are p (to 2^-24, see below), and each is positive where p is, so
// that an infinite value times p is that infinity and not NaN: a part without bits of its own
// takes p 2^-25 instead of 0.
__device__ __forceinline__ float cut_bf16(float p) { return __uint_as_float(__float_as_uint(p) & 0xffff0000u); }
__device__ __forceinline__ void split3(float p, float& hi, float& mid, float& lo) {
  const float t = p * 0x1p-25f;
  hi = cut_bf16(p);
  const float r = fmaxf(p - hi, t);
  mid = cut_bf16(r);
  lo = fmaxf(r - mid, t);
}
// The upper halves of two floats as a pair of bf16.
__device__ __forceinline__ uint32_t upper_halves(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}

// bf16: the warp's state.  Lane l holds columns 2 (l % 4), + 1 of the transposed score tile
// S^T = K Q^T and of O^T = V^T P^T.  Column n belongs to head n % G.  P enters as three bf16 parts,
// which hold its fp32 value; two would leave 2^-17.  Where a tile has columns to spare (G < 8) they
// take the other parts of the same heads: one product with G = 1 or 2, two with 4, three with 8
// (over twelve shapes 1.5% slower than two rounded parts; with three products for each 2.4%).  A
// unit's products are summed by the tensor core, the small parts first, and added to the running
// sums with a rounding: the tensor core cuts its sums off, and a warp's whole run in one
// accumulator lost up to 2^-16.
template <int D, int G>
struct WarpStateBf16 {
  static constexpr int NS = DenseCfg<__nv_bfloat16, D, G>::kTile / 16;  // 16-key products of a unit
  static constexpr int kProducts = G == 8 ? 3 : G == 4 ? 2 : 1;        // products of a slice with its values
  float m[2], l[2], o[D / 16][4];
  uint32_t q[D / 16][2];

  __device__ void start(const DenseArgs& a, int bi, int gi, float*, int lane) {
    const uint32_t* row = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                            ((size_t)bi * a.h + gi * G + (lane >> 2) % G) * D);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      q[k][0] = row[k * 8 + (lane & 3)];
      q[k][1] = row[k * 8 + 4 + (lane & 3)];
      o[k][0] = o[k][1] = o[k][2] = o[k][3] = 0.f;
    }
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }

  // What column 2 (lane % 4) + e takes of a weight's parts in product j.  A column that is over
  // shares the low part with another, so that no column holds a zero (see split3).
  static __device__ __forceinline__ float part_of(int j, int e, int lane, float hi, float mid, float lo) {
    if constexpr (G == 8) return j == 0 ? lo : j == 1 ? mid : hi;
    else if constexpr (G == 4) return j == 0 ? 0.5f * lo : lane & 2 ? mid : hi;
    else if constexpr (G == 2) return (lane & 3) == 0 ? hi : (lane & 3) == 1 ? mid : 0.5f * lo;
    else return lane & 3 ? 0.5f * lo : e ? mid : hi;
  }

  // A unit with `valid` keys (> 0): NS 16-key products side by side, one step of the running
  // maximum for all.
  __device__ void consume(uint32_t sk, uint32_t sv, int valid, float scale, const float*, float*, int lane) {
    constexpr uint32_t kSub = DenseCfg<__nv_bfloat16, D, G>::kSub;
    float s[NS][4];
#pragma unroll
    for (int i = 0; i < NS; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        uint32_t f[4];
        ldsm4(sk + (k >> 2) * kSub + tc::sw128_chunk(16 * i + (lane & 15), (k & 3) * 2 + (lane >> 4)), f);
        mma16816(s[i], f, q[k][0], q[k][1]);
      }
    }
    // s[i]: keys r, r (columns 2c, 2c + 1), r + 8, r + 8, r = 16 i + lane / 4
    float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool ok = 16 * i + 8 * e + (lane >> 2) < valid;
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
    // P^T as the second operand: the parts of keys (0-7, 8-15) of each slice
    uint32_t pt[kProducts][NS][2], keep[NS][2];
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float p0 = exp2f(s[i][2 * e] - b0), p1 = exp2f(s[i][2 * e + 1] - b1);
        l[0] += p0;
        l[1] += p1;
        float h0, h1, m0, m1, l0, l1;
        split3(p0, h0, m0, l0);
        split3(p1, h1, m1, l1);
#pragma unroll
        for (int j = 0; j < kProducts; ++j)
          pt[j][i][e] = transpose8(upper_halves(part_of(j, 0, lane, h0, m0, l0), part_of(j, 1, lane, h1, m1, l1)));
        // values behind the last key may be anything: they are cleared, not only weighted by 0
        const int k0 = 16 * i + 8 * e + (lane & 3) * 2;
        keep[i][e] = (k0 < valid ? 0xffffu : 0u) | (k0 + 1 < valid ? 0xffff0000u : 0u);
      }
    const bool tail = 16 * NS > valid;
    const uint32_t vrow = (lane & 7) + ((lane >> 4) << 3), vch = (lane >> 3) & 1;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t f[NS][4];
      float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        ldsm4_t(sv + (k >> 2) * kSub + tc::sw128_chunk(vrow + 16 * i, (k & 3) * 2 + vch), f[i]);
        if (tail) {
          f[i][0] &= keep[i][0]; f[i][1] &= keep[i][0]; f[i][2] &= keep[i][1]; f[i][3] &= keep[i][1];
        }
      }
#pragma unroll
      for (int j = 0; j < kProducts; ++j)
#pragma unroll
        for (int i = 0; i < NS; ++i) mma16816(t, f[i], pt[j][i][0], pt[j][i][1]);
      o[k][0] = fmaf(o[k][0], c0, t[0]);
      o[k][1] = fmaf(o[k][1], c1, t[1]);
      o[k][2] = fmaf(o[k][2], c0, t[2]);
      o[k][3] = fmaf(o[k][3], c1, t[3]);
    }
  }

  // The sums over all of the warp's keys and of the parts (the lanes hold shares of l, the columns
  // those of the outputs until here).  Column h < G then holds head h.
  __device__ void finish() {
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], d);
      l[1] += __shfl_xor_sync(0xffffffffu, l[1], d);
    }
    if constexpr (G < 8) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (G == 1 && (x & 1)) continue;
          float y = G == 1 ? o[k][x] + o[k][x + 1] : o[k][x];  // G = 1: columns 0 to 3, of lanes 0 and 1 of four
          if (G <= 2) y += __shfl_xor_sync(0xffffffffu, y, 1);
          if (G >= 2) y += __shfl_xor_sync(0xffffffffu, y, 2);
          o[k][x] = y;
        }
    }
  }
  // The result: rows out [G][D], lse [G] (or nullptr).
  __device__ void write(__nv_bfloat16* out, float* lse, int lane) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int hh = (lane & 3) * 2 + e;
      if (hh < G) {
        const float inv = inverse_sum(l[e]);
        if (lse && lane < 4) lse[hh] = log_sum(m[e], l[e]);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          out[hh * D + k * 16 + (lane >> 2)] = __float2bfloat16_rn(o[k][e] * inv);
          out[hh * D + k * 16 + 8 + (lane >> 2)] = __float2bfloat16_rn(o[k][2 + e] * inv);
        }
      }
    }
  }
  // The partial: so [G][D], ml [G].
  __device__ void leave(float* so, float2* ml, int lane) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int hh = (lane & 3) * 2 + e;
      if (hh < G) {
        if (lane < 4) ml[hh] = make_float2(m[e], l[e]);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          so[hh * D + k * 16 + (lane >> 2)] = o[k][e];
          so[hh * D + k * 16 + 8 + (lane >> 2)] = o[k][2 + e];
        }
      }
    }
  }
};

// fp32: CUDA cores.  For the scores lane l takes keys pr, pr + 8, ... of the unit, pr a
// permutation of l / 4 that keeps the swizzled 16-byte reads free of bank conflicts, and the
// quarter l % 4 of the head; each query read from shared memory serves all its keys.  With four
// heads or more the quarters' sums are scattered as they are reduced: lane l ends with the
// logits of heads l % 4, l % 4 + 4 and does the softmax of those alone.  For the output it owns
// D / 32 adjacent columns of every head.
template <int D, int G>
struct WarpStateF32 {
  static constexpr int kTile = DenseCfg<float, D, G>::kTile;
  static constexpr int NR = kTile / 8;             // keys of a lane
  static constexpr int NH = G >= 4 ? G / 4 : G;    // heads whose softmax it does
  static constexpr int kCpl = D / 32;
  float m[NH], l[NH], o[G][kCpl];

  static __device__ __forceinline__ int head(int j, int lane) { return G >= 4 ? (lane & 3) + 4 * j : j; }

  __device__ void start(const DenseArgs& a, int bi, int gi, float* sq, int lane) {
    const float* row = static_cast<const float*>(a.q) + ((size_t)bi * a.h + gi * G) * D;
    for (int x = lane; x < G * D; x += 32) sq[x] = row[x];
    __syncwarp();
#pragma unroll
    for (int j = 0; j < NH; ++j) {
      m[j] = -INFINITY;
      l[j] = 0.f;
    }
#pragma unroll
    for (int hh = 0; hh < G; ++hh)
#pragma unroll
      for (int x = 0; x < kCpl; ++x) o[hh][x] = 0.f;
  }

  // The sum over the quarters of one key's logits s, of the lane's heads.
  static __device__ __forceinline__ void reduce(const float (&s)[G], float (&x)[NH], int lane) {
    if constexpr (G >= 4) {
      // lanes 2 apart exchange the heads that the other keeps (bit 1 of the head), then 1 apart
      float y[G / 2];
#pragma unroll
      for (int j = 0; j < G / 2; ++j) {
        const int lo = (j >> 1) * 4 + (j & 1), hi = lo + 2;
        const float keep = lane & 2 ? s[hi] : s[lo], send = lane & 2 ? s[lo] : s[hi];
        y[j] = keep + __shfl_xor_sync(0xffffffffu, send, 2);
      }
#pragma unroll
      for (int j = 0; j < NH; ++j) {
        const float keep = lane & 1 ? y[2 * j + 1] : y[2 * j], send = lane & 1 ? y[2 * j] : y[2 * j + 1];
        x[j] = keep + __shfl_xor_sync(0xffffffffu, send, 1);
      }
    } else {
#pragma unroll
      for (int j = 0; j < NH; ++j) {
        x[j] = s[j] + __shfl_xor_sync(0xffffffffu, s[j], 1);
        x[j] += __shfl_xor_sync(0xffffffffu, x[j], 2);
      }
    }
  }

  // A unit with `valid` keys (> 0).  sp: [kTile][G] weights, then [G] factors.
  __device__ void consume(uint32_t sk, uint32_t sv, int valid, float scale, const float* sq, float* sp, int lane) {
    constexpr uint32_t kSub = DenseCfg<float, D, G>::kSub;
    const int rr = lane >> 2, c = lane & 3;
    const int pr = ((rr & 1) << 2) | (rr >> 1);
    float s[NR][G];
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int hh = 0; hh < G; ++hh) s[r][hh] = 0.f;
#pragma unroll 2
    for (int i = 0; i < D / 16; ++i) {
      const uint32_t base = sk + (i >> 1) * kSub, j = c + 4 * (i & 1);
      float4 k[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) k[r] = lds4(base + tc::sw128_chunk(8 * r + pr, j));
#pragma unroll
      for (int hh = 0; hh < G; ++hh) {
        const float4 q = *reinterpret_cast<const float4*>(sq + hh * D + (c + 4 * i) * 4);
#pragma unroll
        for (int r = 0; r < NR; ++r)
          s[r][hh] = fmaf(q.x, k[r].x, fmaf(q.y, k[r].y, fmaf(q.z, k[r].z, fmaf(q.w, k[r].w, s[r][hh]))));
      }
    }
    float x[NR][NH], f[NH];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      reduce(s[r], x[r], lane);
#pragma unroll
      for (int j = 0; j < NH; ++j) x[r][j] = 8 * r + pr < valid ? x[r][j] * scale : -INFINITY;
    }
    bool raised = false;
#pragma unroll
    for (int j = 0; j < NH; ++j) {
      float t = x[0][j], base;
#pragma unroll
      for (int r = 1; r < NR; ++r) t = fmaxf(t, x[r][j]);
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
      f[j] = raise_max(m[j], t, base);
      raised |= f[j] != 1.f;
      l[j] *= f[j];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float p = exp2f(x[r][j] - base);
        l[j] += p;
        if (G >= 4 || c == j) sp[(8 * r + pr) * G + head(j, lane)] = p;
      }
      if (rr == 0 && (G >= 4 || c == j)) sp[kTile * G + head(j, lane)] = f[j];
    }
    raised = __any_sync(0xffffffffu, raised);
    __syncwarp();
    if (raised) {
#pragma unroll
      for (int hh = 0; hh < G; ++hh) {
        const float g = sp[kTile * G + hh];
#pragma unroll
        for (int y = 0; y < kCpl; ++y) o[hh][y] *= g;
      }
    }
    const uint32_t piece = lane * kCpl / 4;
    const uint32_t vb = sv + (piece >> 3) * kSub + (lane * kCpl % 4) * 4;
#pragma unroll 4
    for (int j = 0; j < min(kTile, valid); ++j) {  // the values behind the last key are not read
      const uint32_t addr = vb + tc::sw128_chunk(j, piece & 7);
      float v[kCpl], p[G];
      if constexpr (kCpl == 4) {
        const float4 y = lds4(addr);
        v[0] = y.x; v[1] = y.y; v[2] = y.z; v[3] = y.w;
      } else {
        const float2 y = lds2(addr);
        v[0] = y.x; v[1] = y.y;
      }
      if constexpr (G >= 4) {
#pragma unroll
        for (int hh = 0; hh < G; hh += 4) {
          const float4 y = *reinterpret_cast<const float4*>(sp + j * G + hh);
          p[hh] = y.x; p[hh + 1] = y.y; p[hh + 2] = y.z; p[hh + 3] = y.w;
        }
      } else {
#pragma unroll
        for (int hh = 0; hh < G; ++hh) p[hh] = sp[j * G + hh];
      }
#pragma unroll
      for (int hh = 0; hh < G; ++hh)
#pragma unroll
        for (int y = 0; y < kCpl; ++y) o[hh][y] = fmaf(p[hh], v[y], o[hh][y]);
    }
    __syncwarp();
  }

  __device__ void finish() {
#pragma unroll
    for (int j = 0; j < NH; ++j)
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[j] += __shfl_xor_sync(0xffffffffu, l[j], d);
  }
  // m and l of head hh, from the lane that has them
  __device__ __forceinline__ float2 of(int hh) const {
    const int j = G >= 4 ? hh / 4 : hh, from = G >= 4 ? hh % 4 : 0;
    return make_float2(__shfl_sync(0xffffffffu, m[j], from), __shfl_sync(0xffffffffu, l[j], from));
  }
  __device__ void write(float* out, float* lse, int lane) {
#pragma unroll
    for (int hh = 0; hh < G; ++hh) {
      const float2 ml = of(hh);
      const float inv = inverse_sum(ml.y);
      if (lse && lane == 0) lse[hh] = log_sum(ml.x, ml.y);
#pragma unroll
      for (int x = 0; x < kCpl; ++x) out[hh * D + lane * kCpl + x] = o[hh][x] * inv;
    }
  }
  __device__ void leave(float* so, float2* ml, int lane) {
#pragma unroll
    for (int hh = 0; hh < G; ++hh) {
      const float2 y = of(hh);
      if (lane == 0) ml[hh] = y;
#pragma unroll
      for (int x = 0; x < kCpl; ++x) so[hh * D + lane * kCpl + x] = o[hh][x];
    }
  }
};

template <typename T, int D, int G> struct WarpState;
template <int D, int G> struct WarpState<__nv_bfloat16, D, G> : WarpStateBf16<D, G> {};
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

// Segment of units: one (sequence, KV head).
struct Segment {
  int bi, gi, nt;      // nt: its units
  unsigned lo, hi;     // [lo, hi)
};
// A segment that is cut between CTAs: its parts, the first of them that of CTA `first`.
struct Cut {
  Segment g;
  int first, n;        // n 0: there is none
};

template <typename T, int D, int G>
__global__ void __launch_bounds__(kDenseThreads, 1) decode_dense_kernel(const __grid_constant__ DenseKernelArgs ka) {
  using C = DenseCfg<T, D, G>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ unsigned s_prefix[kDenseSeqs + 1];  // units before each sequence
  __shared__ int s_len[kDenseSeqs];
  __shared__ unsigned s_own_prefix[kDenseWarps][33];  // the same of at most 32 sequences, one copy a warp
  __shared__ int s_own_len[kDenseWarps][32];
  __shared__ __align__(16) unsigned s_scan[kDenseWarps];
  __shared__ uint64_t s_full[kDenseWarps][C::kStages];
  __shared__ Segment s_seg[2 * kDenseWarps];     // the segment in each warp slot (nt 0: none)
  __shared__ Cut s_cut[2];                       // the segments of u0 and u1 - 1, where they are cut
  __shared__ float2 s_ml[2 * kDenseWarps][G];
  __shared__ float s_M[G], s_z[G];
  __shared__ int s_abort, s_last[2];
  static_assert(C::kSmem + sizeof(s_prefix) + sizeof(s_len) + sizeof(s_own_prefix) + sizeof(s_own_len) + sizeof(s_scan) +
                        sizeof(s_full) + sizeof(s_seg) + sizeof(s_cut) + sizeof(s_ml) + sizeof(s_M) + sizeof(s_z) +
                        sizeof(s_abort) + sizeof(s_last) + 12 * 16 <=
                    227 * 1024,
                "dynamic and static shared memory of a CTA, the gaps between variables among them");

  const DenseArgs& a = ka.a;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const uint32_t ring0 = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t ring = ring0 + warp * kDenseRing;
  float* s_ring = reinterpret_cast<float*>(smem_raw + (ring0 - tc::smem_u32(smem_raw)));
  float* s_heads = s_ring + C::kRings / 4;
  float* s_weights = s_heads + C::kHeads;
  float* s_sums = s_weights + C::kWeights;
  float* s_q = s_sums + C::kSums + warp * (C::kQ + C::kP);
  float* s_p = s_q + C::kQ;
  // A warp's slots: 2 w for the segment that began before its run, 2 w + 1 for the one that goes
  // on behind it.  The second is left when the warp's ring is no longer in use, and lies there.
  auto slot_of = [&](int x) { return x & 1 ? s_ring + (x >> 1) * (kDenseRing / 4) : s_heads + (x >> 1) * G * D; };

  if (lane == 0) {
    for (int s = 0; s < C::kStages; ++s) tc::mbar_init(tc::smem_u32(&s_full[warp][s]), 1);
    tc::mbar_fence_init();
    s_seg[2 * warp].nt = s_seg[2 * warp + 1].nt = 0;
  }
  if (t == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&ka.tmap_k) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&ka.tmap_v) : "memory");
    s_abort = 0;
  }
  wait_for_stream();
  // ---- units before each sequence
  const unsigned* prefix = s_prefix;
  const int* len = s_len;
  const long long cap = (long long)a.max_chunks * kChunk;
  auto length_of = [&](int b) {
    int L = b < a.b ? a.seq_lens[b] : 0;
    if (L > cap) {
      if (blockIdx.x == 0) set_error(a.err, kErrBadPage);
      L = (int)cap;
    }
    return L;
  };
  auto up_to = [&](unsigned x) {  // inclusive sum over the lanes
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    return x;
  };
  if (a.b <= 32) {  // each warp for itself, without barriers (7 sequences, window of 512: 9.0 -> 8.5 us a call)
    const int L = length_of(lane);
    s_own_len[warp][lane] = L;
    s_own_prefix[warp][lane + 1] = up_to((unsigned)n_tiles<C::kTile>(L, a.n_win) * (unsigned)a.g);
    if (lane == 0) s_own_prefix[warp][0] = 0;
    prefix = s_own_prefix[warp];
    len = s_own_len[warp];
    __syncwarp();
  } else {  // thread t counts sequences 4 t .. 4 t + 3
    constexpr int kPer = kDenseSeqs / kDenseThreads;
    unsigned mine[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int L = length_of(t * kPer + i);
      s_len[t * kPer + i] = L;
      sum += (unsigned)n_tiles<C::kTile>(L, a.n_win) * (unsigned)a.g;
      mine[i] = sum;
    }
    const unsigned inc = up_to(sum);
    if (lane == 31) s_scan[warp] = inc;
    sum = inc - sum;  // before this thread, within the warp
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kDenseWarps; ++w) sum += w < warp ? s_scan[w] : 0u;
#pragma unroll
    for (int i = 0; i < kPer; ++i) s_prefix[t * kPer + i + 1] = sum + mine[i];
    if (t == 0) s_prefix[0] = 0;
    __syncthreads();
  }
  const unsigned total = prefix[a.b];
  const unsigned per = max((unsigned)kDenseMinUnits, (total + kDenseCtas - 1) / kDenseCtas);
  const unsigned u0 = min(total, blockIdx.x * per), u1 = min(total, u0 + per);
  const unsigned per_warp = (u1 - u0 + kDenseWarps - 1) / kDenseWarps;
  const unsigned w0 = min(u1, u0 + warp * per_warp), w1 = min(u1, w0 + per_warp);
  auto segment_of = [&](int b, unsigned u) {  // the segment of unit u of sequence b
    Segment g;
    g.bi = b;
    g.nt = n_tiles<C::kTile>(len[b], a.n_win);
    g.gi = (int)(u - prefix[b]) / g.nt;
    g.lo = prefix[b] + (unsigned)g.gi * g.nt;
    g.hi = g.lo + g.nt;
    return g;
  };

  T* out = static_cast<T*>(a.out);
  // ---- the warp's run: units w0 + 0, 1, ...; lane j knows the place of number base + j (z: block
  // of the pool, -1 for a bad page; y: row in it) and of the 32 after those
  auto locate = [&](unsigned i, int& y, int& z) {
    const unsigned u = w0 + i;
    z = -1;
    y = 0;
    if (u >= w1) return;
    const int b = seq_of(prefix, a.b, u);
    const Segment g = segment_of(b, u);
    const int tile = first_tile<C::kTile>(len[b], a.n_win) + (int)(u - g.lo);
    const int page = a.block_table[(size_t)b * a.max_chunks + tile * C::kTile / kChunk];
    y = tile * C::kTile % kChunk;
    if (page >= 0 && page < a.n_pages) z = page * a.g + g.gi;
    else set_error(a.err, kErrBadPage);
  };
  const unsigned mine = w1 - w0;
  unsigned issued = 0, base = 0, bad = 0;  // bad: bit s, stage s has no page
  int y, z, yn = 0, zn = -1;
  locate(lane, y, z);
  if (mine > 32) locate(32 + lane, yn, zn);
  auto issue = [&]() {  // the next unit's copies (all lanes call it)
    if (issued - base == 32) {
      base += 32;
      y = yn;
      z = zn;
      if (base + 32 < mine) locate(base + 32 + lane, yn, zn);
    }
    const int yi = __shfl_sync(0xffffffffu, y, issued - base), zi = __shfl_sync(0xffffffffu, z, issued - base);
    const int st = (int)(issued % C::kStages);
    bad = zi < 0 ? bad | 1u << st : bad & ~(1u << st);
    if (lane == 0 && zi >= 0) {
      const uint32_t full = tc::smem_u32(&s_full[warp][st]), dst = ring + st * C::kStage;
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
  __syncthreads();  // s_abort is clear
  unsigned phases = 0;  // bit s: parity of the next fill of stage s to wait for

  if (t == 0) {  // for the end, while the first units are on their way
    s_cut[0].n = s_cut[1].n = 0;
    auto note = [&](int side, const Segment& g) {
      const int first = (int)(g.lo / per);
      s_cut[side] = Cut{g, first, (int)((g.hi - 1) / per) - first + 1};
    };
    if (u0 < u1) {
      const Segment first = segment_of(seq_of(prefix, a.b, u0), u0);
      if (first.lo < u0 || first.hi > u1) note(0, first);
      if (first.hi < u1) {
        const Segment last = segment_of(seq_of(prefix, a.b, u1 - 1), u1 - 1);
        if (last.hi > u1) note(1, last);
      }
    }
  }

  // sequences without keys
  for (int b = blockIdx.x; b < a.b; b += kDenseCtas) {
    if (len[b] > 0) continue;
    for (int x = t; x < a.h * D / 4; x += kDenseThreads)
      store4(out + (size_t)b * a.h * D + x * 4, make_float4(0.f, 0.f, 0.f, 0.f));
    if (a.lse)
      for (int x = t; x < a.h; x += kDenseThreads) a.lse[(size_t)b * a.h + x] = -INFINITY;
  }

  const float scale = a.scale * 1.4426950408889634f;  // logits in units of log 2
  bool failed = false;
  int bi = w0 < w1 ? seq_of(prefix, a.b, w0) : 0;
  unsigned u = w0;
  while (u < w1) {
    while (prefix[bi + 1] <= u) ++bi;
    const Segment g = segment_of(bi, u);
    const unsigned ue = min(w1, g.hi);
    const int first = first_tile<C::kTile>(len[bi], a.n_win);
    WarpState<T, D, G> w;
    w.start(a, bi, g.gi, s_q, lane);
    for (; u < ue; ++u) {
      const unsigned i = u - w0;
      const int st = (int)(i % C::kStages);
      if (!(bad >> st & 1u)) {
        failed = !__all_sync(0xffffffffu, tc::mbar_wait(tc::smem_u32(&s_full[warp][st]), phases >> st & 1u, a.poll));
        if (failed) break;
        phases ^= 1u << st;
        const uint32_t sk = ring + st * C::kStage;
        w.consume(sk, sk + C::kHalf, min(C::kTile, len[bi] - (first + (int)(u - g.lo)) * C::kTile), scale, s_q, s_p,
                  lane);
        __syncwarp();
      }
      if (issued < mine) issue();
    }
    if (failed) break;
    w.finish();
    if (g.lo >= w0 && g.hi <= w1) {
      const size_t row = (size_t)bi * a.h + g.gi * G;
      w.write(out + row * D, a.lse ? a.lse + row : nullptr, lane);
    } else {
      const int x = 2 * warp + (g.lo >= w0 ? 1 : 0);
      w.leave(slot_of(x), s_ml[x], lane);
      if (lane == 0) s_seg[x] = g;
    }
  }
  if (failed) {
    // the copies in flight (units u .. w0 + issued - 1) land before the CTA can end
    for (unsigned i = u - w0; i < issued; ++i) {
      const int st = (int)(i % C::kStages);
      if (!(bad >> st & 1u)) tc::mbar_wait(tc::smem_u32(&s_full[warp][st]), phases >> st & 1u, kDrainPolls);
    }
    if (lane == 0) {
      set_error(a.err, kErrTimeout);
      s_abort = 1;
    }
  }
  __syncthreads();
  if (u0 == u1) return;
  const bool aborted = s_abort != 0;

  // ---- the cut segments of the CTA: a chain of slots begins with slot 0 or an odd one and goes
  // on with the even slots of the warps behind it
  auto write_row = [&](int b, int gi, int x, float4 acc, float M, float z) {  // float4 column x of [G][D]
    const size_t row = (size_t)b * a.h + gi * G + x * 4 / D;
    const float inv = inverse_sum(z);
    acc.x *= inv; acc.y *= inv; acc.z *= inv; acc.w *= inv;
    store4(out + row * D + x * 4 % D, acc);
    if (a.lse && x * 4 % D == 0) a.lse[row] = log_sum(M, z);
  };
  // kNp threads share a float4 column: they take every kNp-th chain, or part
  constexpr int kNp = kDenseThreads / C::kVec;
  const int v = t % C::kVec, np = t / C::kVec, hv = v * 4 / D;
  auto first_slot = [](int c) { return c == 0 ? 0 : 2 * c - 1; };
  unsigned chains = __ballot_sync(0xffffffffu, lane <= kDenseWarps && s_seg[first_slot(min(lane, kDenseWarps))].nt != 0);
  for (int k = 0; chains; chains &= chains - 1, ++k) {
    if (k % kNp != np) continue;
    const int x0 = first_slot(__ffs(chains) - 1), w_next = x0 / 2 + 1;
    const Segment g = s_seg[x0];
    int n = 1;  // slots of the chain: x0, then slots 2 w of the warps behind
    while (w_next + n - 1 < kDenseWarps && s_seg[2 * (w_next + n - 1)].nt != 0 && s_seg[2 * (w_next + n - 1)].lo == g.lo) ++n;
    auto member = [&](int i) { return i == 0 ? x0 : 2 * (w_next + i - 1); };
    float M = -INFINITY, sum = 0.f;
    for (int i = 0; i < n; ++i) M = fmaxf(M, s_ml[member(i)][hv].x);
    const float top = M == -INFINITY ? 0.f : M;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < n; ++i) {
      const float2 ml = s_ml[member(i)][hv];
      const float e = exp2f(ml.x - top);
      const float4 p = reinterpret_cast<const float4*>(slot_of(member(i)))[v];
      sum = fmaf(e, ml.y, sum);
      acc.x = fmaf(e, p.x, acc.x); acc.y = fmaf(e, p.y, acc.y);
      acc.z = fmaf(e, p.z, acc.z); acc.w = fmaf(e, p.w, acc.w);
    }
    if (g.lo >= u0 && g.hi <= u1) {
      if (!aborted) write_row(g.bi, g.gi, v, acc, M, sum);
    } else {
      const int slot = 2 * blockIdx.x + (g.lo >= u0 ? 1 : 0);
      __stcg(reinterpret_cast<float4*>(ka.part + (size_t)slot * G * D) + v, acc);
      if (v * 4 % D == 0) __stcg(ka.part_ml + (size_t)slot * G + hv, make_float2(M, sum));
    }
  }
  if (aborted) {  // NaN as a maximum (which is never one) marks the parts that were given up
    __syncthreads();
    if (t < 2 * G) __stcg(ka.part_ml + (size_t)(2 * blockIdx.x + t / G) * G + t % G, make_float2(NAN, 0.f));
  }
  __syncthreads();

  // ---- segments cut between CTAs: the one of u0, and the one of u1 - 1
  // Joins parts j0, j0 + step, ... (n <= kJoinMost) of the segment that begins in CTA `first`:
  // the sum of the float4 column in the threads t < kVec, the rest in s_M and s_z.  Slot 1 of a CTA
  // holds the part of a segment that begins there, slot 0 that of one that began before.
  auto join = [&](int first, int j0, int step, int n) {
    auto slot = [&](int j) { return (size_t)(2 * (first + j0 + j * step) + (j0 + j * step == 0 ? 1 : 0)); };
    auto part_at = [&](int j) { return __ldcg(reinterpret_cast<const float4*>(ka.part + slot(j) * G * D) + v); };
    constexpr int kFirst = 8;  // parts on their way while the weights are computed
    float4 x[kFirst];
#pragma unroll
    for (int i = 0; i < kFirst; ++i)
      x[i] = np + i * kNp < n ? part_at(np + i * kNp) : make_float4(0.f, 0.f, 0.f, 0.f);
    if (warp < G) {
      const float2 ml = lane < n ? __ldcg(ka.part_ml + slot(lane) * G + warp) : make_float2(-INFINITY, 0.f);
      if (ml.x != ml.x) s_abort = 1;
      const float M = warp_max(ml.x), e = exp2f(ml.x - (M == -INFINITY ? 0.f : M));
      const float sum = warp_sum(e * ml.y);
      s_weights[warp * kJoinMost + lane] = e;
      if (lane == 0) {
        s_M[warp] = M;
        s_z[warp] = sum;
      }
    }
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4& p, int j) {
      const float e = s_weights[hv * kJoinMost + j];
      acc.x = fmaf(e, p.x, acc.x); acc.y = fmaf(e, p.y, acc.y);
      acc.z = fmaf(e, p.z, acc.z); acc.w = fmaf(e, p.w, acc.w);
    };
#pragma unroll
    for (int i = 0; i < kFirst; ++i)
      if (np + i * kNp < n) add(x[i], np + i * kNp);
#pragma unroll 8
    for (int j = np + kFirst * kNp; j < n; j += kNp) add(part_at(j), j);
    if constexpr (kNp > 1) {
      float4* sums = reinterpret_cast<float4*>(s_sums);
      sums[np * C::kVec + v] = acc;
      __syncthreads();
      if (np == 0) {
#pragma unroll
        for (int k = 1; k < kNp; ++k) {
          const float4 p = sums[k * C::kVec + v];
          acc.x += p.x; acc.y += p.y; acc.z += p.z; acc.w += p.w;
        }
      }
    }
    return acc;
  };
  // Takes a ticket of n; true for the last.  The counter runs to n - 1 and starts again at 0: ready
  // for the next call.  (One thread: release and acquire cover what the CTA's barriers order.)
  auto take = [](unsigned* counter, int n) {
    unsigned old;
    asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(old) : "l"(counter), "r"(n - 1) : "memory");
    return old == (unsigned)(n - 1);
  };
  // parts are joined at once, or in blocks first: the CTA's block, its slot and its parts
  auto block_of = [&](const Cut& c, size_t& slot, int& j0) {
    j0 = ((int)blockIdx.x - c.first) / kJoinBlock * kJoinBlock;
    slot = 2 * (c.first + j0) + (j0 == 0 ? 1 : 0);
    return min(kJoinBlock, c.n - j0);
  };
  if (lane == 0 && warp < 2 && s_cut[warp].n) {  // both tickets at once
    const Cut c = s_cut[warp];
    if (c.n <= kJoinMost) {
      s_last[warp] = take(ka.ticket + (size_t)c.g.bi * a.g + c.g.gi, c.n);
    } else {
      size_t slot;
      int j0;
      const int members = block_of(c, slot, j0);
      s_last[warp] = take(ka.block_ticket + slot, members);
    }
  }
  __syncthreads();
  for (int side = 0; side < 2; ++side) {
    const Cut c = s_cut[side];
    if (c.n == 0 || !s_last[side]) continue;
    int step = 1, count = c.n;
    if (c.n > kJoinMost) {
      size_t slot;
      int j0;
      const int members = block_of(c, slot, j0);
      const float4 acc = join(c.first, j0, 1, members);
      // the block's sum takes the place of its first part, which has been read
      if (t < C::kVec) {
        __stcg(reinterpret_cast<float4*>(ka.part + slot * G * D) + v, acc);
        if (v * 4 % D == 0) __stcg(ka.part_ml + slot * G + hv, make_float2(s_abort ? NAN : s_M[hv], s_z[hv]));
      }
      __syncthreads();
      step = kJoinBlock;
      count = (c.n + kJoinBlock - 1) / kJoinBlock;
      if (t == 0) s_last[side] = take(ka.ticket + (size_t)c.g.bi * a.g + c.g.gi, count);
      __syncthreads();
      if (!s_last[side]) continue;
    }
    const float4 acc = join(c.first, 0, step, count);
    if (t < C::kVec && !s_abort) write_row(c.g.bi, c.g.gi, v, acc, s_M[hv], s_z[hv]);
    __syncthreads();
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
  return launch_overlapped(decode_dense_kernel<T, D, G>, kDenseCtas, kDenseThreads, C::kSmem, st, ka);
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
  s.block_ticket = s.part_ml + 2ull * kDenseCtas * G * 8;
  s.ticket = s.block_ticket + 2ull * kDenseCtas * 4;
  s.total = s.ticket + 4ull * (b < kDenseSeqs ? b : kDenseSeqs) * g;
  return s;
}

cudaError_t run_decode_dense(const DenseArgs& a, void* scratch, cudaStream_t st) {
  const DenseScratch S = decode_dense_scratch(a.b, a.h, a.g, a.d);
  const size_t es = a.bf16 ? 2 : 4;
  DenseKernelArgs ka;
  const int rows = 8192 / (int)(a.d * es);  // kTile
  if (!encode_pages_map(&ka.tmap_k, a.k_pages, a.d, (long long)a.n_pages * a.g, a.bf16, rows) ||
      !encode_pages_map(&ka.tmap_v, a.v_pages, a.d, (long long)a.n_pages * a.g, a.bf16, rows))
    return cudaErrorInvalidValue;
  char* w = static_cast<char*>(scratch);
  ka.part = reinterpret_cast<float*>(w + S.part);
  ka.part_ml = reinterpret_cast<float2*>(w + S.part_ml);
  ka.block_ticket = reinterpret_cast<unsigned*>(w + S.block_ticket);
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
