// Position rotation (the schemes HiLS notes section 5.4 leaves to the model) of rows of
// queries and keys, and the append of new tokens' keys and values to the paged chunk cache
// with that rotation on the way.
//
// Pair f of a row at position p is turned by the angle p w_f:
//   (x, y) -> (x cos - y sin, y cos + x sin);
// the inverse (the transpose: the gradient) takes -sin.  The angle is reduced in fp64 --
// p w_f / 2 pi less its nearest integer, where the fp32 product would be off by whole
// radians at the positions of a long cache -- and only its remainder, at most half a turn,
// is rounded to fp32 for sincospif.
//
// Both kernels are bound by HBM: every element is read once and written once.  A CTA takes a
// tile of tokens and a block of heads, computes the tile's cosines and sines once into
// shared memory (all its heads use them), and then moves 32 bytes a thread and step: a unit
// is 2 E elements (E = 16 bytes' worth), either E adjacent pairs, or E elements of the
// first half of the rotated part with their E partners, or 2 E elements that are copied.
#include "common.cuh"
#include "kernels.cuh"

namespace hils {

namespace {

constexpr int kRotThreads = 256;
constexpr int kRotTile = 32;      // tokens per CTA, at most
constexpr int kRotUnits = 4;      // units a thread loads before it stores the first
constexpr int kRotCtas = 4 * 148; // CTAs wanted before tiles are made smaller

__device__ __forceinline__ float2 turn_of(int pos, float w) {
  double t = (double)pos * (double)w * 0.15915494309189533577;  // 1 / (2 pi)
  t -= rint(t);
  float s, c;
  sincospif((float)(2.0 * t), &s, &c);
  return make_float2(c, s);
}

template <typename T> struct Unit { static constexpr int E = 16 / (int)sizeof(T); };

// E elements as 16 raw bytes.
template <typename T>
__device__ __forceinline__ void unpack(const uint4& r, float (&f)[Unit<T>::E]) {
  if constexpr (sizeof(T) == 2) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = __bfloat1622float2(h[i]);
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
  } else {
    f[0] = __uint_as_float(r.x); f[1] = __uint_as_float(r.y);
    f[2] = __uint_as_float(r.z); f[3] = __uint_as_float(r.w);
  }
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Stores N adjacent elements, rounded once.
template <typename T, int N>
__device__ __forceinline__ void store(T* dst, const float (&f)[N]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<float4*>(dst + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
  } else if constexpr (N == 4) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]));
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 8)
      *reinterpret_cast<uint4*>(dst + i) =
          make_uint4(bf16_pair(f[i], f[i + 1]), bf16_pair(f[i + 2], f[i + 3]), bf16_pair(f[i + 4], f[i + 5]),
                     bf16_pair(f[i + 6], f[i + 7]));
  }
}

// Where the two 16-byte pieces of unit u lie in a row whose first `rot` elements are rotated.
template <int E>
__device__ __forceinline__ void unit_offsets(int u, int rot, bool interleaved, int& o0, int& o1) {
  const bool halves = !interleaved && u < rot / (2 * E);
  o0 = halves ? u * E : u * 2 * E;
  o1 = halves ? o0 + rot / 2 : o0 + E;
}

// Turns one unit and stores it.  cs: the token's (cos, sin) by frequency.
template <typename Tin, typename Tout>
__device__ __forceinline__ void turn_unit(const uint4& r0, const uint4& r1, int u, int rot, bool interleaved,
                                          const float2* cs, Tout* row) {
  constexpr int E = Unit<Tin>::E;
  int o0, o1;
  unit_offsets<E>(u, rot, interleaved, o0, o1);
  float a[E], b[E];
  unpack<Tin>(r0, a);
  unpack<Tin>(r1, b);
  if (u < rot / (2 * E)) {
    if (interleaved) {
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        const float2 w0 = cs[u * E + i / 2], w1 = cs[u * E + E / 2 + i / 2];
        const float x0 = a[i], y0 = a[i + 1], x1 = b[i], y1 = b[i + 1];
        a[i] = x0 * w0.x - y0 * w0.y;
        a[i + 1] = y0 * w0.x + x0 * w0.y;
        b[i] = x1 * w1.x - y1 * w1.y;
        b[i + 1] = y1 * w1.x + x1 * w1.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float2 w = cs[u * E + i];
        const float x = a[i], y = b[i];
        a[i] = x * w.x - y * w.y;
        b[i] = y * w.x + x * w.y;
      }
    }
  }
  store<Tout>(row + o0, a);
  store<Tout>(row + o1, b);
}

// Tokens of a tile and heads of a block so that about kRotCtas CTAs have work: long inputs
// get full tiles and every head (the cosines are computed once); few tokens are spread over
// the SMs, tokens first, then heads.
void pick_tile(long long tokens, int heads, int* tile, int* head_block) {
  int t = kRotTile, hb = heads;
  while (t > 1 && (tokens + t - 1) / t < kRotCtas) t >>= 1;
  while (hb > 1 && (tokens + t - 1) / t * ((heads + hb - 1) / hb) < kRotCtas && (long long)t * hb > 8) hb = (hb + 1) / 2;
  *tile = t;
  *head_block = hb;
}

}  // namespace

// ---- hils_rotate ------------------------------------------------------------
template <typename Tin, typename Tout, int D>
__global__ void __launch_bounds__(kRotThreads) rotate_kernel(RotateArgs a) {
  constexpr int E = Unit<Tin>::E;
  constexpr int U = D / (2 * E);  // units per row
  __shared__ float2 s_cs[kRotTile][D / 2];
  const int t = threadIdx.x;
  const int heads = a.heads[0] + a.heads[1];
  const int n_hb = (heads + a.head_block - 1) / a.head_block;
  const int n_tile = (a.n + a.tile - 1) / a.tile;
  const int h0 = (int)(blockIdx.x % n_hb) * a.head_block;
  const int ti = (int)(blockIdx.x / n_hb) % n_tile;
  const int bi = (int)(blockIdx.x / n_hb) / n_tile;
  const int t0 = ti * a.tile, nt = min(a.tile, a.n - t0), nh = min(a.head_block, heads - h0);
  const int nf = a.rot / 2;
  for (int x = t; x < nt * nf; x += kRotThreads) {
    const int tok = x / nf, f = x % nf;
    const int pos = a.positions ? a.positions[bi * a.position_stride + t0 + tok] : t0 + tok;
    float2 w = turn_of(pos, a.inv_freq[f]);
    if (a.inverse) w.y = -w.y;
    s_cs[tok][f] = w;
  }
  __syncthreads();
  const int total = nh * a.tile * U;
  for (int x0 = t; x0 < total; x0 += kRotThreads * kRotUnits) {
    uint4 r0[kRotUnits], r1[kRotUnits];
#pragma unroll
    for (int k = 0; k < kRotUnits; ++k) {
      const int x = x0 + k * kRotThreads;
      const int u = x % U, tok = x / U % a.tile, hh = h0 + x / U / a.tile;
      if (x < total && tok < nt) {
        const int which = hh >= a.heads[0];
        const Rows& R = a.in[which];
        const Tin* row = static_cast<const Tin*>(R.data) + bi * R.batch_stride +
                         (hh - which * a.heads[0]) * R.head_stride + (t0 + tok) * R.token_stride;
        int o0, o1;
        unit_offsets<E>(u, a.rot, a.interleaved, o0, o1);
        r0[k] = *reinterpret_cast<const uint4*>(row + o0);
        r1[k] = *reinterpret_cast<const uint4*>(row + o1);
      }
    }
#pragma unroll
    for (int k = 0; k < kRotUnits; ++k) {
      const int x = x0 + k * kRotThreads;
      const int u = x % U, tok = x / U % a.tile, hh = h0 + x / U / a.tile;
      if (x < total && tok < nt) {
        const int which = hh >= a.heads[0];
        const Rows& R = a.out[which];
        Tout* row = static_cast<Tout*>(R.data) + bi * R.batch_stride + (hh - which * a.heads[0]) * R.head_stride +
                    (t0 + tok) * R.token_stride;
        turn_unit<Tin, Tout>(r0[k], r1[k], u, a.rot, a.interleaved, s_cs[tok], row);
      }
    }
  }
}

template <typename Tin, typename Tout>
static cudaError_t launch_rotate(const RotateArgs& a, cudaStream_t st) {
  const int heads = a.heads[0] + a.heads[1];
  const long long blocks =
      (long long)a.b * ((a.n + a.tile - 1) / a.tile) * ((heads + a.head_block - 1) / a.head_block);
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  if (a.d == 64) rotate_kernel<Tin, Tout, 64><<<(unsigned)blocks, kRotThreads, 0, st>>>(a);
  else rotate_kernel<Tin, Tout, 128><<<(unsigned)blocks, kRotThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t run_rotate(RotateArgs a, cudaStream_t st) {
  pick_tile((long long)a.b * a.n, a.heads[0] + a.heads[1], &a.tile, &a.head_block);
  if (a.in_bf16)
    return a.out_bf16 ? launch_rotate<__nv_bfloat16, __nv_bfloat16>(a, st) : launch_rotate<__nv_bfloat16, float>(a, st);
  return a.out_bf16 ? launch_rotate<float, __nv_bfloat16>(a, st) : launch_rotate<float, float>(a, st);
}

// ---- hils_append_paged ------------------------------------------------------
namespace {

// What a CTA knows of a token of its tile.
struct Token {
  int live;        // 0: padding, or a token that cannot be placed
  int bi, i;       // sequence, and token within it
  int pos;         // position in the cache
  int page;        // -1: not written to the pages
};

// The sequence b with cu[b] <= t < cu[b + 1] (the last one with cu[b] <= t; in [0, n) for
// any values).
__device__ __forceinline__ int find_seq(const int32_t* cu, int n, int t) {
  int lo = 0, hi = n;  // cu[lo] <= t < cu[hi], in the sense of a sorted cu
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace

template <typename T, int D>
__global__ void __launch_bounds__(kRotThreads) append_kernel(AppendArgs a, int n_work, int n_tile) {
  constexpr int E = Unit<T>::E;
  constexpr int U = D / (2 * E);
  __shared__ float2 s_cs[kRotTile][D / 2];
  __shared__ Token s_tok[kRotTile];
  const int t = threadIdx.x;
  const bool packed = a.cu_new != nullptr;

  if ((int)blockIdx.x >= n_work) {
    // the list of filled pages: entry s belongs to the sequence b with P_b <= s < P_{b+1},
    // P_b = b + start_b / B; that is room for every page the sequence's tokens can fill
    const int s = ((int)blockIdx.x - n_work) * kRotThreads + t;
    if (s >= a.n_slots) return;
    auto start = [&](int b) { return packed ? (long long)a.cu_new[b] : (long long)b * a.n_new; };
    int lo = 0, hi = a.b;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (mid + start(mid) / kChunk <= s) lo = mid;
      else hi = mid;
    }
    int n = packed ? a.cu_new[lo + 1] - a.cu_new[lo] : a.new_lens ? min(a.new_lens[lo], a.n_new) : a.n_new;
    const long long L = a.seq_lens[lo];
    const long long pos0 = L - n;
    const long long c = (pos0 < 0 ? 0 : pos0) / kChunk + (s - lo - start(lo) / kChunk);
    int page = -1;
    if (n > 0 && s >= lo + start(lo) / kChunk && c * kChunk + kChunk - 1 < L && c < a.max_chunks) {
      page = a.block_table[(size_t)lo * a.max_chunks + c];
      if (page < 0 || page >= a.n_pages) page = -1;
    }
    a.full_pages[s] = page;
    return;
  }

  const int heads = a.h + 2 * a.g;
  const int n_hb = (heads + a.head_block - 1) / a.head_block;
  const int h0 = (int)(blockIdx.x % n_hb) * a.head_block;
  const int ti = (int)(blockIdx.x / n_hb) % n_tile;
  const int row0 = ti * a.tile;  // first token of the tile: a row, or a token of sequence bz
  const int bz = (int)(blockIdx.x / n_hb) / n_tile;
  const int nt = min(a.tile, a.n_new - row0), nh = min(a.head_block, heads - h0);
  const int nf = a.rot / 2;
  if (t < nt) {
    Token k;
    int n;
    if (packed) {
      k.bi = find_seq(a.cu_new, a.b, row0 + t);
      n = a.cu_new[k.bi + 1] - a.cu_new[k.bi];
      k.i = row0 + t - a.cu_new[k.bi];
    } else {
      k.bi = bz;
      n = a.new_lens ? min(a.new_lens[bz], a.n_new) : a.n_new;
      k.i = row0 + t;
    }
    const long long pos = (long long)a.seq_lens[k.bi] - n + k.i;
    k.live = k.i >= 0 && k.i < n;
    k.pos = (int)pos;
    k.page = -1;
    if (k.live) {
      if (pos >= 0 && pos < (long long)a.max_chunks * kChunk)
        k.page = a.block_table[(size_t)k.bi * a.max_chunks + k.pos / kChunk];
      if (k.page < 0 || k.page >= a.n_pages) {
        k.page = -1;
        set_error(a.err, kErrBadPage);
      }
      if (pos < 0) k.live = 0;
    }
    s_tok[t] = k;
  }
  __syncthreads();
  if (a.inv_freq && h0 < a.h + a.g) {
    for (int x = t; x < nt * nf; x += kRotThreads) {
      const int tok = x / nf, f = x % nf;
      if (s_tok[tok].live) s_cs[tok][f] = turn_of(s_tok[tok].pos, a.inv_freq[f]);
    }
    __syncthreads();
  }
  const int total = nh * a.tile * U;
  for (int x0 = t; x0 < total; x0 += kRotThreads * kRotUnits) {
    uint4 r0[kRotUnits], r1[kRotUnits];
    T* dst[kRotUnits];
#pragma unroll
    for (int k = 0; k < kRotUnits; ++k) {
      const int x = x0 + k * kRotThreads;
      const int u = x % U, tok = x / U % a.tile, hh = h0 + x / U / a.tile;
      dst[k] = nullptr;
      if (x < total && tok < nt) {
        const Token& w = s_tok[tok];
        // virtual heads: the h query heads, the g key heads, the g value heads
        const bool is_q = hh < a.h, is_k = !is_q && hh < a.h + a.g;
        const int head = is_q ? hh : is_k ? hh - a.h : hh - a.h - a.g;
        if (w.live && (is_q || w.page >= 0)) {
          const long long b_row = packed ? 0 : w.bi, i_row = packed ? row0 + tok : w.i;
          const Rows& R = is_q ? a.q : is_k ? a.k : a.v;
          const T* row = static_cast<const T*>(R.data) + b_row * R.batch_stride + head * R.head_stride +
                         i_row * R.token_stride;
          if (is_q)
            dst[k] = static_cast<T*>(a.q_out.data) + b_row * a.q_out.batch_stride + head * a.q_out.head_stride +
                     i_row * a.q_out.token_stride;
          else
            dst[k] = static_cast<T*>(is_k ? a.k_pages : a.v_pages) +
                     (((size_t)w.page * a.g + head) * kChunk + w.pos % kChunk) * D;
          int o0, o1;
          unit_offsets<E>(u, is_q || is_k ? a.rot : 0, a.interleaved, o0, o1);
          r0[k] = *reinterpret_cast<const uint4*>(row + o0);
          r1[k] = *reinterpret_cast<const uint4*>(row + o1);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kRotUnits; ++k) {
      const int x = x0 + k * kRotThreads;
      const int u = x % U, tok = x / U % a.tile, hh = h0 + x / U / a.tile;
      if (dst[k]) turn_unit<T, T>(r0[k], r1[k], u, hh < a.h + a.g ? a.rot : 0, a.interleaved, s_cs[tok], dst[k]);
    }
  }
}

cudaError_t run_append(AppendArgs a, cudaStream_t st) {
  const bool packed = a.cu_new != nullptr;
  const int heads = a.h + 2 * a.g;
  const long long tokens = packed ? a.n_new : (long long)a.b * a.n_new;
  long long n_work = 0, n_tile = 0;
  if (tokens > 0) {
    pick_tile(tokens, heads, &a.tile, &a.head_block);
    n_tile = (a.n_new + a.tile - 1) / a.tile;
    n_work = n_tile * (packed ? 1 : a.b) * ((heads + a.head_block - 1) / a.head_block);
  }
  const long long blocks = n_work + (a.n_slots + kRotThreads - 1) / kRotThreads;
  if (blocks == 0) return cudaSuccess;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  if (a.bf16) {
    if (a.d == 64) append_kernel<__nv_bfloat16, 64><<<(unsigned)blocks, kRotThreads, 0, st>>>(a, (int)n_work, (int)n_tile);
    else append_kernel<__nv_bfloat16, 128><<<(unsigned)blocks, kRotThreads, 0, st>>>(a, (int)n_work, (int)n_tile);
  } else {
    if (a.d == 64) append_kernel<float, 64><<<(unsigned)blocks, kRotThreads, 0, st>>>(a, (int)n_work, (int)n_tile);
    else append_kernel<float, 128><<<(unsigned)blocks, kRotThreads, 0, st>>>(a, (int)n_work, (int)n_tile);
  }
  return cudaGetLastError();
}

}  // namespace hils
