// Position rotation (the schemes HiLS notes section 5.4 leaves to the model) of rows of
// queries and keys, and the append of new tokens' keys and values to the paged chunk cache
// with that rotation on the way.
//
// Pair f of a row at position p is turned by the angle p w_f:
//   (x, y) -> (x cos - y sin, y cos + x sin);
// the inverse (the transpose: the gradient) takes -sin.  The angle is reduced in fp64: p w_f / 2 pi
// less its nearest integer, where the fp32 product is off by up to 0.03 radians at position 512K
// and 0.25 at 4M.  Only the remainder, at most half a turn, is rounded to fp32 for sincospif.
//
// Both kernels are bound by HBM: every element is read once and written once.  A thread owns
// one unit of one token -- 2 E elements of its row (E = 16 bytes' worth): E pairs, or 2 E
// elements that are copied -- in every head of its block.  It computes the cosines and sines
// of its pairs once, keeps them in registers, and walks the heads, so that a head costs two
// loads, the products and two stores.  The tokens of the whole batch are numbered in a row, and
// a CTA takes kRotThreads / (units per row) of them: short sequences fill it as long ones do.
// Loads and stores are marked as streaming (nothing is read twice): reads that stayed in L2
// pushed half-written output lines out of it (345M prefill shape: 55 -> 47 us).  Measured:
// q and k of the 345M prefill shape, slices of a fused projection, 44 us (268 MB, 6.2 TB/s), to
// fp32 72 us (403 MB, 5.6 TB/s), from fp32 to bf16 63 us (6.4 TB/s); fp32 gradients of the 16K
// training shape 164 us (1.07 GB, 6.6 TB/s); 20K prompt tokens of the 7B shape appended in 80 us
// (490 MB, 6.1 TB/s); one token for each of 64 sequences 3.7 us.
#include "common.cuh"
#include "kernels.cuh"

namespace hils {

namespace {

constexpr int kRotThreads = 128;
constexpr int kRotHeads = 4;       // heads whose loads a thread issues before it stores the first
constexpr int kRotMany = 32 * 148; // CTAs wanted: several waves, so that the last one costs little ...
constexpr int kRotBlock = 8;       // ... but blocks of this many heads (the angles are computed per block) ...
constexpr int kRotFew = 2 * 148;   // ... unless that leaves fewer CTAs than this: then down to one head each
constexpr int kRotSeqs = 1024;     // sequences whose row offsets fit shared memory

__device__ __forceinline__ float2 turn_of(int pos, float w) {
  // a + e is p w (31 + 24 bits, two more than a double has), kInv + kInvLow is 1 / 2 pi: the
  // remainder is right to 2^-53 of a turn (one double each: 4e-7 radians off at position 2^31)
  constexpr double kInv = 0.15915494309189535, kInvLow = -9.839338337591243e-18;
  const double a = (double)pos * (double)w, e = fma((double)pos, (double)w, -a);
  const double t = fma(a, kInv, -rint(a * kInv)) + fma(a, kInvLow, e * kInv);
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
      __stcs(reinterpret_cast<float4*>(dst + i), make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]));
  } else if constexpr (N == 4) {
    __stcs(reinterpret_cast<uint2*>(dst), make_uint2(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3])));
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 8)
      __stcs(reinterpret_cast<uint4*>(dst + i),
             make_uint4(bf16_pair(f[i], f[i + 1]), bf16_pair(f[i + 2], f[i + 3]), bf16_pair(f[i + 4], f[i + 5]),
                        bf16_pair(f[i + 6], f[i + 7])));
  }
}

// Where the two 16-byte pieces of unit u lie in a row whose first `rot` elements are rotated.
template <int E>
__device__ __forceinline__ void unit_offsets(int u, int rot, bool interleaved, int& o0, int& o1) {
  const bool halves = !interleaved && u < rot / (2 * E);
  o0 = halves ? u * E : u * 2 * E;
  o1 = halves ? o0 + rot / 2 : o0 + E;
}

// The cosines and sines of one unit's pairs, and how its pieces pair up.
enum { kCopied = 0, kHalves = 1, kAdjacent = 2 };
template <int E>
struct Turns {
  float2 w[E];
  int how;
  __device__ __forceinline__ void set(int pos, const float* inv_freq, int u, int rot, bool interleaved, bool inverse) {
    how = u >= rot / (2 * E) ? kCopied : interleaved ? kAdjacent : kHalves;
    if (how == kCopied) return;
#pragma unroll
    for (int i = 0; i < E; ++i) {  // pair u E + i, whichever way the pairs are laid out
      w[i] = turn_of(pos, inv_freq[u * E + i]);
      if (inverse) w[i].y = -w[i].y;
    }
  }
};

// Turns one unit's two pieces and stores them.
template <typename Tin, typename Tout, int E = Unit<Tin>::E>
__device__ __forceinline__ void turn_unit(const uint4& r0, const uint4& r1, const Turns<E>& t, int how, Tout* d0,
                                          Tout* d1) {
  if (sizeof(Tin) == sizeof(Tout) && how == kCopied) {  // bit for bit
    __stcs(reinterpret_cast<uint4*>(d0), r0);
    __stcs(reinterpret_cast<uint4*>(d1), r1);
    return;
  }
  float a[E], b[E];
  unpack<Tin>(r0, a);
  unpack<Tin>(r1, b);
  if (how == kAdjacent) {
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const float2 w0 = t.w[i / 2], w1 = t.w[E / 2 + i / 2];
      const float x0 = a[i], y0 = a[i + 1], x1 = b[i], y1 = b[i + 1];
      a[i] = x0 * w0.x - y0 * w0.y;
      a[i + 1] = y0 * w0.x + x0 * w0.y;
      b[i] = x1 * w1.x - y1 * w1.y;
      b[i + 1] = y1 * w1.x + x1 * w1.y;
    }
  } else if (how == kHalves) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float x = a[i], y = b[i];
      a[i] = x * t.w[i].x - y * t.w[i].y;
      b[i] = y * t.w[i].x + x * t.w[i].y;
    }
  }
  store<Tout>(d0, a);
  store<Tout>(d1, b);
}

// One unit of n heads: head k lies at src + k ss and goes to dst + k ds.
template <typename Tin, typename Tout, int E = Unit<Tin>::E>
__device__ __forceinline__ void turn_heads(const Tin* src, long long ss, Tout* dst, long long ds, int n, int o0, int o1,
                                           const Turns<E>& t, int how) {
  src += o0;
  dst += o0;
  const int step = o1 - o0;
  for (; n > 0; n -= kRotHeads, src += kRotHeads * ss, dst += kRotHeads * ds) {
    uint4 r0[kRotHeads], r1[kRotHeads];
#pragma unroll
    for (int k = 0; k < kRotHeads; ++k) {
      if (k < n) {
        r0[k] = __ldcs(reinterpret_cast<const uint4*>(src + k * ss));
        r1[k] = __ldcs(reinterpret_cast<const uint4*>(src + k * ss + step));
      }
    }
#pragma unroll
    for (int k = 0; k < kRotHeads; ++k)
      if (k < n) turn_unit<Tin, Tout>(r0[k], r1[k], t, how, dst + k * ds, dst + k * ds + step);
  }
}

// Heads per CTA.  One block of all heads computes the angles once but leaves few waves of CTAs: at
// the 345M prefill shape 46 us with blocks of 16 heads, 44 with 8, and with 8 waves wanted instead
// of 32 45 us there and 88 instead of 80 for 20K prompt tokens.  Halves that are not below
// kRotBlock are tried first, then kRotBlock itself: 48 heads of those prompts take blocks of 12
// (80.5 us, 81.8 with 8), 40 heads of a 2K prompt blocks of 8 (8.1 us; halved on to 5 9.2), 48
// heads of four prompts 8.3 us (6: 10.7).  Few tokens are spread further, down to one head a CTA:
// one token for each of 64 sequences 3.6 us, 4.0 with all heads in one block.
int pick_heads(long long token_blocks, int heads) {
  int hb = heads;
  auto ctas = [&] { return token_blocks * ((heads + hb - 1) / hb); };
  while ((hb + 1) / 2 >= kRotBlock && ctas() < kRotMany) hb = (hb + 1) / 2;
  if (hb > kRotBlock && ctas() < kRotMany) hb = kRotBlock;
  while (hb > 1 && ctas() < kRotFew) hb = (hb + 1) / 2;
  return hb;
}

}  // namespace

// ---- hils_rotate ------------------------------------------------------------
template <typename Tin, typename Tout, int D>
__global__ void __launch_bounds__(kRotThreads) rotate_kernel(RotateArgs a) {
  constexpr int E = Unit<Tin>::E;
  constexpr int U = D / (2 * E);  // units per row
  wait_for_stream();
  const int heads = a.heads[0] + a.heads[1];
  const int n_hb = (heads + a.head_block - 1) / a.head_block;
  const int h0 = (int)(blockIdx.x % n_hb) * a.head_block, h1 = min(heads, h0 + a.head_block);
  const int u = threadIdx.x % U;
  const unsigned row = blockIdx.x / n_hb * (kRotThreads / U) + threadIdx.x / U;  // b n < 2^31
  if (row >= (unsigned)a.b * (unsigned)a.n) return;
  const int bi = (int)(row / (unsigned)a.n), i = (int)(row % (unsigned)a.n);
  int o0, o1;
  unit_offsets<E>(u, a.rot, a.interleaved, o0, o1);
  const int pos = a.positions ? a.positions[bi * a.position_stride + i] : i;
  Turns<E> t;
  t.set(pos, a.inv_freq, u, a.rot, a.interleaved, a.inverse);
#pragma unroll 1
  for (int w = 0; w < 2; ++w) {  // the block's heads of q, then those of k
    const int lo = max(h0 - (w ? a.heads[0] : 0), 0), hi = min(h1 - (w ? a.heads[0] : 0), a.heads[w]);
    if (lo >= hi) continue;
    const Rows& in = a.in[w];
    const Rows& out = a.out[w];
    turn_heads<Tin, Tout>(
        static_cast<const Tin*>(in.data) + bi * in.batch_stride + i * in.token_stride + lo * in.head_stride,
        in.head_stride,
        static_cast<Tout*>(out.data) + bi * out.batch_stride + i * out.token_stride + lo * out.head_stride,
        out.head_stride, hi - lo, o0, o1, t, t.how);
  }
}

template <typename Tin, typename Tout, int D>
static cudaError_t launch_rotate_d(RotateArgs a, cudaStream_t st) {
  constexpr int kRows = kRotThreads / (D / (2 * Unit<Tin>::E));
  const int heads = a.heads[0] + a.heads[1];
  const long long token_blocks = ((long long)a.b * a.n + kRows - 1) / kRows;
  a.head_block = pick_heads(token_blocks, heads);
  const long long blocks = token_blocks * ((heads + a.head_block - 1) / a.head_block);
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  return launch_overlapped(rotate_kernel<Tin, Tout, D>, (unsigned)blocks, kRotThreads, 0, st, a);
}
template <typename Tin, typename Tout>
static cudaError_t launch_rotate(const RotateArgs& a, cudaStream_t st) {
  return a.d == 64 ? launch_rotate_d<Tin, Tout, 64>(a, st) : launch_rotate_d<Tin, Tout, 128>(a, st);
}

cudaError_t run_rotate(const RotateArgs& a, cudaStream_t st) {
  if (a.in_bf16)
    return a.out_bf16 ? launch_rotate<__nv_bfloat16, __nv_bfloat16>(a, st) : launch_rotate<__nv_bfloat16, float>(a, st);
  return a.out_bf16 ? launch_rotate<float, __nv_bfloat16>(a, st) : launch_rotate<float, float>(a, st);
}

// ---- hils_append_paged ------------------------------------------------------
namespace {

// The last b < n with cu[b] <= t (0 where there is none): the sequence of row t.
__device__ __forceinline__ int find_seq(const int32_t* cu, int n, int t) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace

// The CTAs from n_work on write the list of filled pages.
template <typename T, int D>
__global__ void __launch_bounds__(kRotThreads) append_kernel(AppendArgs a, int n_work) {
  constexpr int E = Unit<T>::E;
  constexpr int U = D / (2 * E);
  __shared__ int32_t s_cu[kRotSeqs + 1];
  wait_for_stream();
  const int t = threadIdx.x;
  const bool packed = a.cu_new != nullptr;
  const int32_t* cu = a.cu_new;
  if (packed && a.b <= kRotSeqs) {  // the search below reads the offsets one after another
    for (int x = t; x <= a.b; x += kRotThreads) s_cu[x] = a.cu_new[x];
    __syncthreads();
    cu = s_cu;
  }

  if ((int)blockIdx.x >= n_work) {
    // entry s belongs to the sequence b with P_b <= s < P_{b+1}, P_b = b + start_b / B: that
    // is room for every page the sequence's tokens can fill
    const int s = ((int)blockIdx.x - n_work) * kRotThreads + t;
    if (s >= a.n_slots) return;
    auto start = [&](int b) { return packed ? (long long)cu[b] : (long long)b * a.n_new; };
    int lo = 0, hi = a.b;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (mid + start(mid) / kChunk <= s) lo = mid;
      else hi = mid;
    }
    const int n = packed ? cu[lo + 1] - cu[lo] : a.new_lens ? min(a.new_lens[lo], a.n_new) : a.n_new;
    const long long L = a.seq_lens[lo], pos0 = L - n;
    const long long j = s - lo - start(lo) / kChunk;
    const long long c = (pos0 < 0 ? 0 : pos0) / kChunk + j;
    int page = -1;
    if (n > 0 && j >= 0 && c * kChunk + kChunk - 1 < L && c < a.max_chunks) {
      page = a.block_table[(size_t)lo * a.max_chunks + c];
      if (page < 0 || page >= a.n_pages) page = -1;
    }
    a.full_pages[s] = page;
    return;
  }

  const int heads = a.h + 2 * a.g;  // the query heads, the key heads, the value heads
  const int n_hb = (heads + a.head_block - 1) / a.head_block;
  const int h0 = (int)(blockIdx.x % n_hb) * a.head_block, h1 = min(heads, h0 + a.head_block);
  const int u = t % U;
  const unsigned row = blockIdx.x / n_hb * (kRotThreads / U) + t / U;  // fewer than 2^31 rows
  if (row >= (packed ? (unsigned)a.n_new : (unsigned)a.b * (unsigned)a.n_new)) return;
  const int bi = packed ? find_seq(cu, a.b, (int)row) : (int)(row / (unsigned)a.n_new);
  const int i = packed ? (int)row - cu[bi] : (int)(row % (unsigned)a.n_new);
  const int n = packed ? cu[bi + 1] - cu[bi] : a.new_lens ? min(a.new_lens[bi], a.n_new) : a.n_new;
  if (i < 0 || i >= n) return;  // padding
  const long long pos = (long long)a.seq_lens[bi] - n + i;
  int page = -1;
  if (pos >= 0 && pos < (long long)a.max_chunks * kChunk)
    page = a.block_table[(size_t)bi * a.max_chunks + pos / kChunk];
  if (page < 0 || page >= a.n_pages) {
    if (u == 0) set_error(a.err, kErrBadPage);
    page = -1;
  }
  if (pos < 0) return;

  const long long bs = packed ? 0 : bi, is = packed ? (long long)row : i;
  const int rot = h0 < a.h + a.g ? a.rot : 0;  // a block of values needs no angles
  Turns<E> w;
  w.set((int)pos, a.inv_freq, u, rot, a.interleaved, false);
  int o0, o1;
  unit_offsets<E>(u, a.rot, a.interleaved, o0, o1);
  const size_t cell = ((size_t)(page < 0 ? 0 : page) * a.g * kChunk + (size_t)(pos % kChunk)) * D;  // of head 0
#pragma unroll 1
  for (int part = 0; part < 3; ++part) {  // the block's heads of q, of k and of v
    const int base = part == 0 ? 0 : part == 1 ? a.h : a.h + a.g, count = part == 0 ? a.h : a.g;
    const int lo = max(h0 - base, 0), hi = min(h1 - base, count);
    if (lo >= hi || (part > 0 && page < 0)) continue;
    const Rows& in = part == 0 ? a.q : part == 1 ? a.k : a.v;
    const T* src = static_cast<const T*>(in.data) + bs * in.batch_stride + is * in.token_stride + lo * in.head_stride;
    T* dst;
    long long ds;
    if (part == 0) {
      dst = static_cast<T*>(a.q_out.data) + bs * a.q_out.batch_stride + is * a.q_out.token_stride +
            lo * a.q_out.head_stride;
      ds = a.q_out.head_stride;
    } else {
      dst = static_cast<T*>(part == 1 ? a.k_pages : a.v_pages) + cell + (size_t)lo * kChunk * D;
      ds = kChunk * D;
    }
    turn_heads<T, T>(src, in.head_stride, dst, ds, hi - lo, o0, o1, w, part == 2 ? (int)kCopied : w.how);
  }
}

template <typename T, int D>
static cudaError_t launch_append(AppendArgs a, cudaStream_t st) {
  constexpr int kRows = kRotThreads / (D / (2 * Unit<T>::E));
  const int heads = a.h + 2 * a.g;
  const long long tokens = a.cu_new ? a.n_new : (long long)a.b * a.n_new;
  const long long token_blocks = (tokens + kRows - 1) / kRows;
  a.head_block = pick_heads(token_blocks, heads);
  const long long n_work = token_blocks * ((heads + a.head_block - 1) / a.head_block);
  const long long blocks = n_work + (a.n_slots + kRotThreads - 1) / kRotThreads;
  if (blocks == 0) return cudaSuccess;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  return launch_overlapped(append_kernel<T, D>, (unsigned)blocks, kRotThreads, 0, st, a, (int)n_work);
}

cudaError_t run_append(const AppendArgs& a, cudaStream_t st) {
  if (a.bf16) return a.d == 64 ? launch_append<__nv_bfloat16, 64>(a, st) : launch_append<__nv_bfloat16, 128>(a, st);
  return a.d == 64 ? launch_append<float, 64>(a, st) : launch_append<float, 128>(a, st);
}

}  // namespace hils
