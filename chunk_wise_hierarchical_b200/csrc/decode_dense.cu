// Attention of one new token per sequence over every key of its paged cache:
//   s_j = q.k_j scale,  out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  m = max_j s_j,
// over the keys j of the sequence (or of its last window of chunks), and log sum_j exp(s_j).
//
// One CTA per (sequence, KV head); its warps take the keys in turn, each with its own
// running maximum, sum and output, joined at the end in shared memory.
#include "common.cuh"
#include "kernels.cuh"

namespace hils {

namespace {
constexpr int kDenseWarps = 8;
}

template <typename T, int D, int G>
__global__ void __launch_bounds__(kDenseWarps * 32) decode_dense_kernel(DenseArgs a) {
  constexpr int CPL = D / 32;
  __shared__ float s_o[kDenseWarps][G][D];
  __shared__ float s_m[kDenseWarps][G], s_l[kDenseWarps][G];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gi = blockIdx.x % a.g, bi = blockIdx.x / a.g;
  const long long cap = (long long)a.max_chunks * kChunk;
  long long L = a.seq_lens[bi];
  if (L > cap) {
    if (threadIdx.x == 0) set_error(a.err, kErrBadPage);
    L = cap;
  }
  const long long first = a.n_win ? max(0ll, ((L > 0 ? L - 1 : 0) / kChunk + 1 - a.n_win) * kChunk) : 0;
  float q[G][CPL], o[G][CPL], m[G], l[G];
#pragma unroll
  for (int hh = 0; hh < G; ++hh) {
    m[hh] = -INFINITY;
    l[hh] = 0.f;
#pragma unroll
    for (int x = 0; x < CPL; ++x) {
      q[hh][x] = to_f(static_cast<const T*>(a.q)[((size_t)bi * a.h + gi * G + hh) * D + lane * CPL + x]);
      o[hh][x] = 0.f;
    }
  }
  for (long long j = first + warp; j < L; j += kDenseWarps) {
    const int p = a.block_table[(size_t)bi * a.max_chunks + j / kChunk];
    if (p < 0 || p >= a.n_pages) {
      if (lane == 0) set_error(a.err, kErrBadPage);
      continue;
    }
    const size_t row = (((size_t)p * a.g + gi) * kChunk + j % kChunk) * D + lane * CPL;
    float k[CPL], v[CPL];
#pragma unroll
    for (int x = 0; x < CPL; ++x) {
      k[x] = to_f(static_cast<const T*>(a.k_pages)[row + x]);
      v[x] = to_f(static_cast<const T*>(a.v_pages)[row + x]);
    }
#pragma unroll
    for (int hh = 0; hh < G; ++hh) {
      float s = 0.f;
#pragma unroll
      for (int x = 0; x < CPL; ++x) s = fmaf(q[hh][x], k[x], s);
      s = warp_sum(s) * a.scale;
      const float mn = fmaxf(m[hh], s), base = mn == -INFINITY ? 0.f : mn;
      const float c = expf(m[hh] - base), e = expf(s - base);
      m[hh] = mn;
      l[hh] = l[hh] * c + e;
#pragma unroll
      for (int x = 0; x < CPL; ++x) o[hh][x] = o[hh][x] * c + e * v[x];
    }
  }
#pragma unroll
  for (int hh = 0; hh < G; ++hh) {
    s_m[warp][hh] = m[hh];
    s_l[warp][hh] = l[hh];
#pragma unroll
    for (int x = 0; x < CPL; ++x) s_o[warp][hh][lane * CPL + x] = o[hh][x];
  }
  __syncthreads();
  for (int x = threadIdx.x; x < G * D; x += kDenseWarps * 32) {
    const int hh = x / D, col = x % D;
    float M = -INFINITY, z = 0.f, acc = 0.f;
    for (int w = 0; w < kDenseWarps; ++w) M = fmaxf(M, s_m[w][hh]);
    const float base = M == -INFINITY ? 0.f : M;
    for (int w = 0; w < kDenseWarps; ++w) {
      const float e = expf(s_m[w][hh] - base);
      z += s_l[w][hh] * e;
      acc += s_o[w][hh][col] * e;
    }
    const size_t row = (size_t)bi * a.h + gi * G + hh;
    static_cast<T*>(a.out)[row * D + col] = from_f<T>(z == 0.f ? 0.f : acc / z);
    if (a.lse && col == 0) a.lse[row] = z == 0.f ? -INFINITY : M + logf(z);
  }
}

template <typename T, int D>
static cudaError_t launch_dense(const DenseArgs& a, cudaStream_t st) {
  const unsigned blocks = (unsigned)a.b * a.g;
  switch (a.h / a.g) {
    case 1: decode_dense_kernel<T, D, 1><<<blocks, kDenseWarps * 32, 0, st>>>(a); break;
    case 2: decode_dense_kernel<T, D, 2><<<blocks, kDenseWarps * 32, 0, st>>>(a); break;
    case 4: decode_dense_kernel<T, D, 4><<<blocks, kDenseWarps * 32, 0, st>>>(a); break;
    case 8: decode_dense_kernel<T, D, 8><<<blocks, kDenseWarps * 32, 0, st>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

cudaError_t run_decode_dense(DenseArgs a, cudaStream_t st) {
  if (a.bf16) return a.d == 64 ? launch_dense<__nv_bfloat16, 64>(a, st) : launch_dense<__nv_bfloat16, 128>(a, st);
  return a.d == 64 ? launch_dense<float, 64>(a, st) : launch_dense<float, 128>(a, st);
}

}  // namespace hils
