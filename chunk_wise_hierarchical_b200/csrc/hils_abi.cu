// C ABI of libhils.so: argument validation, workspace layout and dispatch.
// Every entry point checks its arguments on the host, then enqueues kernels on
// the caller's stream; nothing here allocates device memory or synchronises
// (except hils_device_status).
#include <algorithm>
#include <cmath>
#include <cstring>
#include <atomic>
#include <mutex>
#include <utility>

#include "../../include/hils.h"
#include "common.cuh"
#include "kernels.cuh"

namespace {

// Polls of an ordinary bounded wait in the tensor-core kernels (hils_set_wait_limit).
std::atomic<uint32_t> g_wait_limit{HILS_DEFAULT_WAIT_LIMIT};

constexpr size_t kAlign = 256;
constexpr size_t kHeader = 256;  // error word + reserved
constexpr int kMaxWindow = 64 * 128;  // local branch of at most 128 chunks
constexpr int kMaxDecodeLocal = 16;   // ... and of at most 16 in a decode step
constexpr int kAnyWindow = 0x7fffffff;  // dense decode: a window only says where it begins

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

hils_status check_shape(const hils_shape* s, bool need_seq, int max_window = kMaxWindow) {
  if (!s) return HILS_ERR_INVALID_ARG;
  if (s->batch < 0 || s->heads_q <= 0 || s->heads_kv <= 0 || s->head_dim <= 0 || s->seq_len < 0 ||
      s->chunk <= 0 || s->top_k < 0)
    return HILS_ERR_INVALID_ARG;
  if (s->heads_q % s->heads_kv != 0) return HILS_ERR_INVALID_ARG;
  if (!std::isfinite(s->scale)) return HILS_ERR_INVALID_ARG;
  if (s->dtype != HILS_F32 && s->dtype != HILS_BF16) return HILS_ERR_INVALID_ARG;
  const int grp = s->heads_q / s->heads_kv;
  if (grp != 1 && grp != 2 && grp != 4 && grp != 8) return HILS_ERR_UNSUPPORTED;
  if (s->head_dim != 64 && s->head_dim != 128) return HILS_ERR_UNSUPPORTED;
  if (s->chunk != hils::kChunk) return HILS_ERR_UNSUPPORTED;
  if (s->top_k > hils::kMaxTopK) return HILS_ERR_UNSUPPORTED;
  if (s->window < 0 || s->window % s->chunk != 0) return HILS_ERR_INVALID_ARG;
  if (s->window > max_window) return HILS_ERR_UNSUPPORTED;
  (void)need_seq;
  return HILS_OK;
}

// Chunks in the local branch: the own chunk (window 0 or B) or window / B.
int n_local(const hils_shape* s) { return s->window <= s->chunk ? 1 : s->window / s->chunk; }

float eff_scale(const hils_shape* s) {
  return s->scale == 0.f ? 1.0f / std::sqrt((float)s->head_dim) : s->scale;
}

// Whether prefill attention takes the chunk-major tensor-core path for this shape (its
// scratch is then part of the workspace); the kernel's register check comes at launch.
bool cm_applies(const hils_shape* s) {
  if (s->dtype != HILS_BF16 || s->heads_kv <= 0) return false;
  const int G = s->heads_q / s->heads_kv;
  if (!hils::cm_shape_supported(s->head_dim, G, s->top_k, s->seq_len, n_local(s))) return false;
  const hils::CmScratch S = hils::cm_scratch(s->batch, s->heads_q, s->heads_kv, s->seq_len, s->head_dim,
                                             s->top_k, n_local(s));
  // partial rows and selection indices are 32-bit
  return ((size_t)S.n_lt + S.max_sel) * 128 < (1ull << 31) &&
         (size_t)s->batch * s->heads_kv * s->seq_len * s->top_k < (1ull << 31) &&
         (size_t)s->batch * s->heads_q * s->seq_len < (1ull << 31);
}
size_t cm_bytes(const hils_shape* s) {
  if (!cm_applies(s)) return 0;
  return hils::cm_scratch(s->batch, s->heads_q, s->heads_kv, s->seq_len, s->head_dim, s->top_k, n_local(s)).total;
}

// Whether selection takes the grouped tensor-core path (its split summaries are then
// part of the workspace): bf16, G in {2, 4, 8}, at least one full tile of chunks and of
// queries.
bool gtc_applies(const hils_shape* s) {
  if (s->dtype != HILS_BF16 || s->heads_kv <= 0) return false;
  const int G = s->heads_q / s->heads_kv;
  return hils::select_gtc_supported(s->head_dim, G, s->top_k, true) && s->seq_len / s->chunk >= 64 &&
         s->seq_len >= 128;
}
size_t gtc_bytes(const hils_shape* s) {
  if (!gtc_applies(s)) return 0;
  return 2 * align_up(hils::gtc_split_bytes(s->batch, s->heads_q, s->seq_len / s->chunk, s->head_dim));
}

struct AttendLayout {
  size_t kbar, hbias, idx, ssel, gtc, cm, total;
};
AttendLayout attend_layout(const hils_shape* s) {
  const size_t b = s->batch, h = s->heads_q, g = s->heads_kv, n = s->seq_len, d = s->head_dim;
  const size_t C = n / s->chunk, K = s->top_k;
  AttendLayout L;
  size_t off = kHeader;
  L.kbar = off; off = align_up(off + b * h * C * d * 4);
  L.hbias = off; off = align_up(off + b * h * C * 4);
  L.idx = off; off = align_up(off + b * g * n * K * 4);
  L.ssel = off; off = align_up(off + b * h * n * K * 4);
  L.gtc = off; off = align_up(off + gtc_bytes(s));
  L.cm = off; off = align_up(off + cm_bytes(s));
  L.total = off;
  return L;
}

struct BackwardLayout {
  size_t drow, list_off, list, total;
};
BackwardLayout backward_layout(const hils_shape* s) {
  const size_t b = s->batch, h = s->heads_q, g = s->heads_kv, n = s->seq_len, K = s->top_k;
  const size_t C = n / s->chunk;
  BackwardLayout L;
  size_t off = kHeader;
  L.drow = off; off = align_up(off + b * h * n * 4);
  L.list_off = off; off = align_up(off + b * g * (C + 1) * 4);
  L.list = off; off = align_up(off + b * g * n * K * 4);
  L.total = off;
  return L;
}

struct DecodeLayout {
  size_t part_keys, part_att, scan_ticket, att_ticket, idx, sel_page, ssel, total;
};
DecodeLayout decode_layout(const hils_shape* s) {
  const size_t b = s->batch, h = s->heads_q, g = s->heads_kv, K = s->top_k, d = s->head_dim;
  const size_t G = h / g;
  const int cmax = (s->seq_len + s->chunk - 1) / s->chunk;
  const size_t nsplit = hils::decode_splits(s->batch, cmax);
  DecodeLayout L;
  size_t off = kHeader;
  L.part_keys = off; off = align_up(off + b * g * nsplit * K * 8);
  L.part_att = off; off = align_up(off + b * g * 2 * (K + n_local(s)) * G * (d + 2) * 4);  // half-chunk partials
  L.scan_ticket = off; off = align_up(off + b * g * 4);
  L.att_ticket = off; off = align_up(off + b * g * 4);
  L.idx = off; off = align_up(off + b * g * K * 4);
  L.sel_page = off; off = align_up(off + b * g * K * 4);
  L.ssel = off; off = align_up(off + b * h * K * 4);
  L.total = off;
  return L;
}

hils_status cuda_status(cudaError_t e) { return e == cudaSuccess ? HILS_OK : HILS_ERR_CUDA; }

// Prefill attention + fusion for a selection: the chunk-major tcgen05 path for bf16
// inputs (scratch at `cm_ws`, 256-byte aligned), else the row-owner tcgen05 kernels
// where they fit the shape, else the row kernel.
cudaError_t run_prefill_attention(const hils_shape* s, const void* q, const void* k, const void* v,
                                  const int32_t* idx, const float* ssel, void* out, float* lse,
                                  unsigned* err, void* cm_ws, cudaStream_t cs) {
  const bool bf16 = s->dtype == HILS_BF16;
  const int G = s->heads_q / s->heads_kv;
  // d = 64 with the own-chunk branch stays on the row-owner kernel, measured faster there;
  // every other bf16 shape the chunk-major path covers takes it
  const bool row_owner_d64 = bf16 && n_local(s) == 1 && s->head_dim == 64 &&
                             hils::attend_tc3_supported(64, G, s->top_k, s->seq_len);
  if (!row_owner_d64 && cm_ws && cm_applies(s) && hils::cm_kernel_ready(s->head_dim, G)) {
    const hils::CmScratch S = hils::cm_scratch(s->batch, s->heads_q, s->heads_kv, s->seq_len, s->head_dim,
                                               s->top_k, n_local(s));
    char* w = static_cast<char*>(cm_ws);
    hils::CmArgs a{};
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.idx = idx; a.ssel = ssel; a.out = static_cast<__nv_bfloat16*>(out); a.lse = lse; a.err = err;
    a.cnt = reinterpret_cast<int*>(w + S.cnt);
    a.cur = reinterpret_cast<int*>(w + S.cur);
    a.toff = reinterpret_cast<int*>(w + S.toff);
    a.n_sel = reinterpret_cast<int*>(w + S.n_sel);
    a.abort_flag = reinterpret_cast<int*>(w + S.abort_flag);
    a.desc = reinterpret_cast<int4*>(w + S.desc);
    a.ent_q = reinterpret_cast<int*>(w + S.ent_q);
    a.pos = reinterpret_cast<int*>(w + S.pos);
    a.part = reinterpret_cast<__nv_bfloat16*>(w + S.part);
    a.plse = reinterpret_cast<float*>(w + S.plse);
    a.b = s->batch; a.h = s->heads_q; a.g = s->heads_kv; a.n = s->seq_len; a.d = s->head_dim;
    a.top_k = s->top_k; a.n_local = n_local(s);
    a.c_sel = S.c_sel; a.c_all = S.c_all; a.tl = S.tl; a.n_lt = S.n_lt; a.max_sel = S.max_sel;
    a.scale = eff_scale(s);
    a.poll = g_wait_limit.load();
    return hils::run_attend_cm(a, cs);
  }
  if (bf16 && n_local(s) == 1 && hils::attend_tc_supported(s->head_dim, G, s->top_k, s->seq_len)) {
    hils::TcAttendArgs ta{};
    ta.q = static_cast<const __nv_bfloat16*>(q);
    ta.k = static_cast<const __nv_bfloat16*>(k);
    ta.v = static_cast<const __nv_bfloat16*>(v);
    ta.idx = idx; ta.ssel = ssel; ta.out = static_cast<__nv_bfloat16*>(out); ta.lse = lse; ta.err = err;
    ta.b = s->batch; ta.h = s->heads_q; ta.g = s->heads_kv; ta.n = s->seq_len; ta.top_k = s->top_k;
    ta.scale = eff_scale(s);
    ta.poll = g_wait_limit.load();
    return hils::run_attend_tc(ta, s->head_dim, cs);
  }
  hils::AttendRowsArgs ar{};
  ar.q = q; ar.k = k; ar.v = v; ar.idx = idx; ar.ssel = ssel; ar.out = out; ar.lse = lse;
  ar.block_table = nullptr; ar.seq_lens = nullptr; ar.err = err;
  ar.b = s->batch; ar.h = s->heads_q; ar.g = s->heads_kv; ar.n = s->seq_len; ar.d = s->head_dim;
  ar.top_k = s->top_k; ar.max_chunks = 0; ar.n_pages = 0; ar.scale = eff_scale(s); ar.bf16 = bf16;
  ar.paged = false; ar.n_local = n_local(s);
  return hils::run_attend_rows(ar, cs);
}

// Rows of (nb, nh, nt) x d elements that 16-byte loads and stores can take (the stride of a
// dimension with one entry is not looked at).
hils_status check_rows(const hils_rows* r, long long nb, long long nh, long long nt, size_t elem) {
  if (!r || !r->data || !aligned16(r->data)) return HILS_ERR_INVALID_ARG;
  const long long n[3] = {nb, nh, nt}, st[3] = {r->batch_stride, r->head_stride, r->token_stride};
  for (int i = 0; i < 3; ++i)  // (and no stride beyond an address space, so that the sums below fit)
    if (n[i] > 1 && (st[i] < 0 || st[i] > (1ll << 56) / (long long)elem / (n[i] - 1) || st[i] * (long long)elem % 16 != 0))
      return HILS_ERR_INVALID_ARG;
  return HILS_OK;
}
// Bytes [lo, hi) that rows of (nb, nh, nt) x d elements lie in.
struct Span {
  uintptr_t lo, hi;
};
Span span_of(const hils_rows* r, long long nb, long long nh, long long nt, int d, size_t elem) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(r->data);
  if (nb == 0 || nh == 0 || nt == 0) return {p, p};
  return {p, p + (size_t)((nb - 1) * r->batch_stride + (nh - 1) * r->head_stride + (nt - 1) * r->token_stride + d) * elem};
}
bool overlap(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }
// Rows as sharing() compares them: strides and row length in bytes.
struct RowSet {
  long long data, n[3], stride[3], row;
};
RowSet row_set(const hils_rows* r, long long nb, long long nh, long long nt, int d, size_t elem) {
  const long long e = (long long)elem;
  return {(long long)reinterpret_cast<uintptr_t>(r->data), {nb, nh, nt},
          {r->batch_stride * e, r->head_stride * e, r->token_stride * e}, d * e};
}
// Whether some row of a and some row of b share a byte.  A dimension that both step by the same
// stride moves their distance by whole strides: those are searched, the widest first, and only
// the few steps that can bring the rows together (three where the strides nest).  One that they
// step by different strides is taken as filled.  So slices of one fused tensor are told apart
// exactly; other sets whose spans meet may be taken to share where they only interleave.
bool sharing(const RowSet& a, const RowSet& b) {
  long long end_a = a.row, end_b = b.row;  // rows meet at distances in (-end_b, end_a)
  struct Dim {
    long long s, lo, hi;
  } dim[3];
  int nd = 0;
  for (int i = 0; i < 3; ++i) {
    if (a.n[i] == 0 || b.n[i] == 0) return false;
    const long long s = a.n[i] == 1 ? b.stride[i] : a.stride[i];
    if (a.n[i] > 1 && b.n[i] > 1 && a.stride[i] != b.stride[i]) {
      end_a += (a.n[i] - 1) * a.stride[i];
      end_b += (b.n[i] - 1) * b.stride[i];
    } else if ((a.n[i] > 1 || b.n[i] > 1) && s > 0) {
      dim[nd++] = {s, -(a.n[i] - 1), b.n[i] - 1};
    }
  }
  for (int i = 0; i < nd; ++i)
    for (int j = i + 1; j < nd; ++j)
      if (dim[j].s > dim[i].s) std::swap(dim[i], dim[j]);
  int steps = 0;
  auto floor_div = [](long long x, long long y) { return x / y - (x % y < 0); };
  auto meet = [&](auto& self, int i, long long off) -> bool {
    if (i == nd) return -end_b < off && off < end_a;
    long long lo = 0, hi = 0;  // what the dimensions behind this one can add
    for (int j = i + 1; j < nd; ++j) {
      lo += dim[j].lo * dim[j].s;
      hi += dim[j].hi * dim[j].s;
    }
    const long long x0 = std::max(dim[i].lo, floor_div(-end_b - off - hi, dim[i].s) + 1);
    const long long x1 = std::min(dim[i].hi, -floor_div(-(end_a - off - lo), dim[i].s) - 1);
    for (long long x = x0; x <= x1; ++x)
      if (++steps > 100 || self(self, i + 1, off + x * dim[i].s)) return true;
    return false;
  };
  return meet(meet, 0, b.data - a.data);
}
// Whether no two rows of a written tensor share an element: by ascending stride, each
// dimension steps over all that the dimensions below it cover.
bool rows_apart(const hils_rows* r, long long nb, long long nh, long long nt, int d) {
  long long n[3] = {nb, nh, nt}, st[3] = {r->batch_stride, r->head_stride, r->token_stride}, extent = d;
  for (int i = 0; i < 2; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (st[j] < st[i]) {
        std::swap(st[i], st[j]);
        std::swap(n[i], n[j]);
      }
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (st[i] < extent) return false;
    extent += st[i] * (n[i] - 1);
  }
  return true;
}
// Whether out is in's own memory, element for element.
bool in_place(const hils_rows* out, const hils_rows* in, long long nb, long long nh, long long nt) {
  return out->data == in->data && (nb <= 1 || out->batch_stride == in->batch_stride) &&
         (nh <= 1 || out->head_stride == in->head_stride) && (nt <= 1 || out->token_stride == in->token_stride);
}
hils_status check_rope(const hils_rope* r, int head_dim) {
  if (!r || !r->inv_freq || !aligned4(r->inv_freq)) return HILS_ERR_INVALID_ARG;
  if (r->rotary_dim <= 0 || r->rotary_dim > head_dim || (r->interleaved != 0 && r->interleaved != 1))
    return HILS_ERR_INVALID_ARG;
  return r->rotary_dim % 16 == 0 ? HILS_OK : HILS_ERR_UNSUPPORTED;
}
size_t dense_bytes(const hils_shape* s) {
  return kHeader + align_up(hils::decode_dense_scratch(s->batch, s->heads_q, s->heads_kv, s->head_dim).total);
}
hils::Rows rows_of(const hils_rows* r) { return {r->data, r->batch_stride, r->head_stride, r->token_stride}; }
size_t elem_size(int32_t dtype) { return dtype == HILS_BF16 ? 2 : 4; }

}  // namespace

extern "C" {

const char* hils_status_string(int status) {
  switch (status) {
    case HILS_OK: return "ok";
    case HILS_ERR_INVALID_ARG: return "invalid argument";
    case HILS_ERR_UNSUPPORTED: return "unsupported shape or dtype";
    case HILS_ERR_WORKSPACE: return "workspace missing or too small";
    case HILS_ERR_CUDA: return "CUDA error";
    case HILS_ERR_DEVICE_CHECK: return "device-side index check failed";
    case HILS_ERR_DEVICE_TIMEOUT: return "device-side wait timed out";
  }
  return "unknown status";
}

int32_t hils_abi_version(void) { return 3; }

uint32_t hils_set_wait_limit(uint32_t polls) { return g_wait_limit.exchange(polls); }

hils_status hils_workspace_size(const hils_shape* s, int32_t op, size_t* bytes) {
  if (!bytes) return HILS_ERR_INVALID_ARG;
  hils_status st = check_shape(s, true, op == HILS_OP_DECODE_DENSE ? kAnyWindow : kMaxWindow);
  if (st != HILS_OK) return st;
  switch (op) {
    case HILS_OP_SELECT: *bytes = kHeader + gtc_bytes(s); return HILS_OK;
    case HILS_OP_ATTEND: *bytes = attend_layout(s).total; return HILS_OK;
    case HILS_OP_DECODE: *bytes = decode_layout(s).total; return HILS_OK;
    case HILS_OP_ATTEND_SELECTED: *bytes = kHeader + cm_bytes(s); return HILS_OK;
    case HILS_OP_BACKWARD: *bytes = backward_layout(s).total; return HILS_OK;
    case HILS_OP_DECODE_DENSE: *bytes = dense_bytes(s); return HILS_OK;
    case HILS_OP_APPEND: *bytes = kHeader; return HILS_OK;
  }
  return HILS_ERR_INVALID_ARG;
}

hils_status hils_summarize(const hils_shape* s, const void* k, const void* landmark_q, float* kbar,
                           float* hbias, void* stream) {
  hils_status st = check_shape(s, true);
  if (st != HILS_OK) return st;
  const int C = s->seq_len / s->chunk;
  if ((size_t)s->batch * C == 0) return HILS_OK;
  if (!k || !landmark_q || !kbar || !hbias) return HILS_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(landmark_q) || !aligned16(kbar)) return HILS_ERR_INVALID_ARG;
  hils::SummarizeArgs a{};
  a.k = k; a.lm = landmark_q; a.kbar = kbar; a.hbias = hbias;
  a.b = s->batch; a.h = s->heads_q; a.g = s->heads_kv; a.n = s->seq_len; a.d = s->head_dim;
  a.n_chunks = C; a.scale = eff_scale(s); a.bf16 = s->dtype == HILS_BF16;
  a.page_ids = nullptr;
  return cuda_status(hils::run_summarize(a, (cudaStream_t)stream));
}

hils_status hils_summarize_paged(const hils_shape* s, const void* k_pages, const void* landmark_pages,
                                 const int32_t* page_ids, int32_t n_listed, int32_t n_pages,
                                 float* kbar_pages, float* hbias_pages, void* stream) {
  return hils_summarize_paged_ex(s, k_pages, landmark_pages, page_ids, n_listed, n_pages, kbar_pages, HILS_F32,
                                 hbias_pages, stream);
}

hils_status hils_summarize_paged_ex(const hils_shape* s, const void* k_pages, const void* landmark_pages,
                                    const int32_t* page_ids, int32_t n_listed, int32_t n_pages,
                                    void* kbar_pages, int32_t summary_dtype, float* hbias_pages, void* stream) {
  hils_status st = check_shape(s, false);
  if (st != HILS_OK) return st;
  if (summary_dtype != HILS_F32 && summary_dtype != HILS_BF16) return HILS_ERR_INVALID_ARG;
  if (summary_dtype == HILS_BF16 && s->dtype != HILS_BF16) return HILS_ERR_UNSUPPORTED;
  if (n_listed < 0 || n_pages < 0) return HILS_ERR_INVALID_ARG;
  if (n_listed == 0) return HILS_OK;
  if (!k_pages || !landmark_pages || !page_ids || !kbar_pages || !hbias_pages) return HILS_ERR_INVALID_ARG;
  if (!aligned16(k_pages) || !aligned16(landmark_pages) || !aligned16(kbar_pages)) return HILS_ERR_INVALID_ARG;
  hils::SummarizeArgs a{};
  a.k = k_pages; a.lm = landmark_pages; a.kbar = kbar_pages; a.hbias = hbias_pages;
  a.b = 0; a.h = s->heads_q; a.g = s->heads_kv; a.n = 0; a.d = s->head_dim; a.n_chunks = 0;
  a.scale = eff_scale(s); a.bf16 = s->dtype == HILS_BF16;
  a.page_ids = page_ids; a.n_listed = n_listed; a.n_pages = n_pages;
  a.kbar_bf16 = summary_dtype == HILS_BF16;
  return cuda_status(hils::run_summarize(a, (cudaStream_t)stream));
}

// Scores + Top-K: the tensor-core kernel where it applies (bf16, G = 1), else SIMT.
// gtc_ws: the split-summary scratch (gtc_bytes), or nullptr where the grouped path does
// not apply.
static cudaError_t run_select(const hils::SelectArgs& a, void* gtc_ws, cudaStream_t st) {
  if (hils::select_tc_supported(a.d, a.h / a.g, a.top_k, a.bf16)) {
    hils::SelectArgs t = a;
    t.poll = g_wait_limit.load();
    return hils::run_select_tc(t, st);
  }
  if (gtc_ws) {
    hils::GtcArgs g{};
    g.q = static_cast<const __nv_bfloat16*>(a.q);
    g.kbar = a.kbar; g.hbias = a.hbias; g.idx = a.idx; g.score = a.score; g.err = a.err;
    const size_t half = align_up(hils::gtc_split_bytes(a.b, a.h, a.n_chunks, a.d));
    g.kbar_hi = static_cast<__nv_bfloat16*>(gtc_ws);
    g.kbar_lo = reinterpret_cast<__nv_bfloat16*>(static_cast<char*>(gtc_ws) + half);
    g.b = a.b; g.h = a.h; g.g = a.g; g.n = a.n; g.d = a.d; g.n_chunks = a.n_chunks; g.top_k = a.top_k;
    g.n_local = a.n_local; g.scale = a.scale; g.poll = g_wait_limit.load();
    return hils::run_select_gtc(g, st);
  }
  return hils::run_select_simt(a, st);
}

hils_status hils_select(const hils_shape* s, const void* q, const float* kbar, const float* hbias,
                        int32_t* topk_idx, float* topk_score, void* ws, size_t ws_bytes, void* stream) {
  hils_status st = check_shape(s, true);
  if (st != HILS_OK) return st;
  if ((size_t)s->batch * s->seq_len * s->top_k == 0) return HILS_OK;
  const int C = s->seq_len / s->chunk;
  if (!q || !topk_idx || (C > 0 && (!kbar || !hbias))) return HILS_ERR_INVALID_ARG;
  if (!aligned16(q) || (C > 0 && !aligned16(kbar))) return HILS_ERR_INVALID_ARG;
  const size_t gb = gtc_bytes(s);
  if (!ws || ws_bytes < kHeader + gb || !aligned16(ws)) return HILS_ERR_WORKSPACE;
  hils::SelectArgs a{};
  a.q = q; a.kbar = kbar; a.hbias = hbias; a.idx = topk_idx; a.score = topk_score;
  a.err = static_cast<unsigned*>(ws);
  a.b = s->batch; a.h = s->heads_q; a.g = s->heads_kv; a.n = s->seq_len; a.d = s->head_dim;
  a.n_chunks = C; a.top_k = s->top_k; a.scale = eff_scale(s); a.bf16 = s->dtype == HILS_BF16;
  a.n_local = n_local(s);
  return cuda_status(run_select(a, gb ? static_cast<char*>(ws) + kHeader : nullptr, (cudaStream_t)stream));
}

hils_status hils_attend(const hils_shape* s, const void* q, const void* k, const void* v,
                        const void* landmark_q, void* out, float* lse_out, int32_t* topk_idx_out, void* ws,
                        size_t ws_bytes, void* stream) {
  hils_status st = check_shape(s, true);
  if (st != HILS_OK) return st;
  if ((size_t)s->batch * s->seq_len == 0) return HILS_OK;
  const int C = s->seq_len / s->chunk;
  if (!q || !k || !v || !out || (C > 0 && !landmark_q)) return HILS_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) ||
      (C > 0 && !aligned16(landmark_q)))
    return HILS_ERR_INVALID_ARG;
  const AttendLayout L = attend_layout(s);
  if (!ws || ws_bytes < L.total || !aligned16(ws)) return HILS_ERR_WORKSPACE;
  cudaStream_t cs = (cudaStream_t)stream;
  char* w = static_cast<char*>(ws);
  float* kbar = reinterpret_cast<float*>(w + L.kbar);
  float* hbias = reinterpret_cast<float*>(w + L.hbias);
  int32_t* idx = topk_idx_out ? topk_idx_out : reinterpret_cast<int32_t*>(w + L.idx);
  float* ssel = reinterpret_cast<float*>(w + L.ssel);
  const bool bf16 = s->dtype == HILS_BF16;
  const float scale = eff_scale(s);

  if (C > 0) {
    hils::SummarizeArgs sa{};
    sa.k = k; sa.lm = landmark_q; sa.kbar = kbar; sa.hbias = hbias;
    sa.b = s->batch; sa.h = s->heads_q; sa.g = s->heads_kv; sa.n = s->seq_len; sa.d = s->head_dim;
    sa.n_chunks = C; sa.scale = scale; sa.bf16 = bf16; sa.page_ids = nullptr;
    if (hils::run_summarize(sa, cs) != cudaSuccess) return HILS_ERR_CUDA;
  }
  if (s->top_k > 0) {
    hils::SelectArgs se{};
    se.q = q; se.kbar = kbar; se.hbias = hbias; se.idx = idx; se.score = ssel;
    se.b = s->batch; se.h = s->heads_q; se.g = s->heads_kv; se.n = s->seq_len; se.d = s->head_dim;
    se.n_chunks = C; se.top_k = s->top_k; se.scale = scale; se.bf16 = bf16; se.n_local = n_local(s);
    se.err = reinterpret_cast<unsigned*>(w);
    if (run_select(se, L.gtc != L.cm ? w + L.gtc : nullptr, cs) != cudaSuccess) return HILS_ERR_CUDA;
  }
  return cuda_status(run_prefill_attention(s, q, k, v, idx, ssel, out, lse_out, reinterpret_cast<unsigned*>(w),
                                           L.cm != L.total ? w + L.cm : nullptr, cs));
}

hils_status hils_attend_selected(const hils_shape* s, const void* q, const void* k, const void* v,
                                 const int32_t* topk_idx, const float* topk_score, void* out, float* lse_out,
                                 void* ws, size_t ws_bytes, void* stream) {
  hils_status st = check_shape(s, true);
  if (st != HILS_OK) return st;
  if ((size_t)s->batch * s->seq_len == 0) return HILS_OK;
  if (!q || !k || !v || !out || (s->top_k > 0 && (!topk_idx || !topk_score))) return HILS_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return HILS_ERR_INVALID_ARG;
  const size_t cmb = cm_bytes(s);
  if (!ws || ws_bytes < kHeader + cmb || !aligned16(ws)) return HILS_ERR_WORKSPACE;
  char* w = static_cast<char*>(ws);
  return cuda_status(run_prefill_attention(s, q, k, v, topk_idx, topk_score, out, lse_out,
                                           reinterpret_cast<unsigned*>(ws), cmb ? w + kHeader : nullptr,
                                           (cudaStream_t)stream));
}

hils_status hils_backward(const hils_shape* s, const void* q, const void* k, const void* v,
                          const void* landmark_q, const void* out, const float* lse, const int32_t* topk_idx,
                          const float* topk_score, const void* dout, float* dq, float* dk, float* dv,
                          float* dlandmark, void* ws, size_t ws_bytes, void* stream) {
  hils_status st = check_shape(s, true);
  if (st != HILS_OK) return st;
  if (s->dtype != HILS_BF16) return HILS_ERR_UNSUPPORTED;
  if ((size_t)s->batch * s->seq_len == 0) return HILS_OK;
  if ((long long)s->seq_len * s->top_k >= (1ll << 31) || s->seq_len >= (1 << 25)) return HILS_ERR_UNSUPPORTED;
  const int C = s->seq_len / s->chunk;
  if (!q || !k || !v || !out || !lse || !dout || !dq || !dk || !dv) return HILS_ERR_INVALID_ARG;
  if (C > 0 && (!landmark_q || !dlandmark)) return HILS_ERR_INVALID_ARG;
  if (s->top_k > 0 && (!topk_idx || !topk_score)) return HILS_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(dout) || !aligned16(dq) ||
      !aligned16(dk) || !aligned16(dv) || (C > 0 && !aligned16(landmark_q)))
    return HILS_ERR_INVALID_ARG;
  const BackwardLayout L = backward_layout(s);
  if (!ws || ws_bytes < L.total || !aligned16(ws)) return HILS_ERR_WORKSPACE;
  char* w = static_cast<char*>(ws);
  hils::BwdArgs a{};
  a.q = q; a.k = k; a.v = v; a.landmark = landmark_q; a.out = out; a.dout = dout; a.lse = lse;
  a.idx = topk_idx; a.ssel = topk_score; a.dq = dq; a.dk = dk; a.dv = dv; a.dlandmark = dlandmark;
  a.drow = reinterpret_cast<float*>(w + L.drow);
  a.list_off = reinterpret_cast<int*>(w + L.list_off);
  a.list = reinterpret_cast<int*>(w + L.list);
  a.err = reinterpret_cast<unsigned*>(w);
  a.b = s->batch; a.h = s->heads_q; a.g = s->heads_kv; a.n = s->seq_len; a.d = s->head_dim;
  a.top_k = s->top_k; a.n_local = n_local(s); a.scale = eff_scale(s);
  return cuda_status(hils::run_backward(a, (cudaStream_t)stream));
}

hils_status hils_decode(const hils_shape* s, const void* q, const void* k_pages, const void* v_pages,
                        const float* kbar_pages, const float* hbias_pages, const int32_t* block_table,
                        int32_t max_chunks, const int32_t* seq_lens, int32_t n_pages, void* out,
                        int32_t* topk_idx_out, void* ws, size_t ws_bytes, void* stream) {
  return hils_decode_ex(s, q, k_pages, v_pages, kbar_pages, HILS_F32, hbias_pages, block_table, max_chunks,
                        seq_lens, n_pages, out, topk_idx_out, ws, ws_bytes, stream);
}

hils_status hils_decode_ex(const hils_shape* s, const void* q, const void* k_pages, const void* v_pages,
                           const void* kbar_pages, int32_t summary_dtype, const float* hbias_pages,
                           const int32_t* block_table, int32_t max_chunks, const int32_t* seq_lens,
                           int32_t n_pages, void* out, int32_t* topk_idx_out, void* ws, size_t ws_bytes,
                           void* stream) {
  hils_status st = check_shape(s, true);
  if (st != HILS_OK) return st;
  if (summary_dtype != HILS_F32 && summary_dtype != HILS_BF16) return HILS_ERR_INVALID_ARG;
  if (summary_dtype == HILS_BF16 && s->dtype != HILS_BF16) return HILS_ERR_UNSUPPORTED;
  if (s->batch == 0) return HILS_OK;
  if (!hils::decode_supported(s->heads_q, s->head_dim) || n_local(s) > kMaxDecodeLocal) return HILS_ERR_UNSUPPORTED;
  if (max_chunks <= 0 || n_pages <= 0) return HILS_ERR_INVALID_ARG;
  if ((long long)max_chunks > ((long long)s->seq_len + s->chunk - 1) / s->chunk) return HILS_ERR_INVALID_ARG;
  if (!hils::decode_merge_supported(s->batch, max_chunks, s->top_k)) return HILS_ERR_UNSUPPORTED;
  if (!q || !k_pages || !v_pages || !kbar_pages || !hbias_pages || !block_table || !seq_lens || !out)
    return HILS_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(kbar_pages) ||
      !aligned16(out))
    return HILS_ERR_INVALID_ARG;
  const DecodeLayout L = decode_layout(s);
  if (!ws || ws_bytes < L.total || !aligned16(ws)) return HILS_ERR_WORKSPACE;
  cudaStream_t cs = (cudaStream_t)stream;
  char* w = static_cast<char*>(ws);
  unsigned* err = reinterpret_cast<unsigned*>(w);
  int32_t* idx = topk_idx_out ? topk_idx_out : reinterpret_cast<int32_t*>(w + L.idx);
  hils::DecodeArgs da{};
  da.q = q; da.k_pages = k_pages; da.v_pages = v_pages; da.kbar_pages = kbar_pages;
  da.hbias_pages = hbias_pages; da.block_table = block_table; da.seq_lens = seq_lens; da.out = out;
  da.idx = idx;
  da.ssel = reinterpret_cast<float*>(w + L.ssel);
  da.sel_page = reinterpret_cast<int32_t*>(w + L.sel_page);
  da.part_keys = reinterpret_cast<unsigned long long*>(w + L.part_keys);
  da.part_att = reinterpret_cast<float*>(w + L.part_att);
  da.scan_ticket = reinterpret_cast<unsigned*>(w + L.scan_ticket);
  da.att_ticket = reinterpret_cast<unsigned*>(w + L.att_ticket);
  da.err = err;
  da.b = s->batch; da.h = s->heads_q; da.g = s->heads_kv; da.d = s->head_dim; da.top_k = s->top_k;
  da.max_chunks = max_chunks; da.n_pages = n_pages; da.scale = eff_scale(s);
  da.bf16 = s->dtype == HILS_BF16;
  da.kbar_bf16 = summary_dtype == HILS_BF16;
  da.n_local = n_local(s);
  return cuda_status(hils::run_decode(da, cs));
}

hils_status hils_rotate(const hils_shape* s, const hils_rows* q, const hils_rows* k, const hils_rope* rope,
                        const int32_t* positions, int64_t position_stride, int32_t inverse, const hils_rows* q_out,
                        const hils_rows* k_out, int32_t out_dtype, void* stream) {
  hils_status st = check_shape(s, true);
  if (st != HILS_OK) return st;
  if (out_dtype != HILS_F32 && out_dtype != HILS_BF16) return HILS_ERR_INVALID_ARG;
  if ((k == nullptr) != (k_out == nullptr)) return HILS_ERR_INVALID_ARG;
  if (position_stride < 0 || !aligned4(positions)) return HILS_ERR_INVALID_ARG;
  if ((st = check_rope(rope, s->head_dim)) != HILS_OK) return st;
  if ((size_t)s->batch * s->seq_len == 0) return HILS_OK;
  if ((long long)s->batch * s->seq_len > 0x7fffffffll) return HILS_ERR_UNSUPPORTED;
  {
    const long long nb = s->batch, nt = s->seq_len;
    const size_t ei = elem_size(s->dtype), eo = elem_size(out_dtype);
    if ((st = check_rows(q, nb, s->heads_q, nt, ei)) != HILS_OK ||
        (st = check_rows(q_out, nb, s->heads_q, nt, eo)) != HILS_OK)
      return st;
    if (k && ((st = check_rows(k, nb, s->heads_kv, nt, ei)) != HILS_OK ||
              (st = check_rows(k_out, nb, s->heads_kv, nt, eo)) != HILS_OK))
      return st;
    if (!rows_apart(q_out, nb, s->heads_q, nt, s->head_dim) ||
        (k && !rows_apart(k_out, nb, s->heads_kv, nt, s->head_dim)))
      return HILS_ERR_INVALID_ARG;
    // each output apart from every other tensor, its own input in place excepted
    const RowSet qi = row_set(q, nb, s->heads_q, nt, s->head_dim, ei), qo = row_set(q_out, nb, s->heads_q, nt, s->head_dim, eo);
    if (!(ei == eo && in_place(q_out, q, nb, s->heads_q, nt)) && sharing(qo, qi)) return HILS_ERR_INVALID_ARG;
    if (k) {
      const RowSet ki = row_set(k, nb, s->heads_kv, nt, s->head_dim, ei), ko = row_set(k_out, nb, s->heads_kv, nt, s->head_dim, eo);
      if (!(ei == eo && in_place(k_out, k, nb, s->heads_kv, nt)) && sharing(ko, ki)) return HILS_ERR_INVALID_ARG;
      if (sharing(qo, ki) || sharing(ko, qi) || sharing(qo, ko)) return HILS_ERR_INVALID_ARG;
    }
  }
  hils::RotateArgs a{};
  a.in[0] = rows_of(q); a.out[0] = rows_of(q_out); a.heads[0] = s->heads_q;
  if (k) { a.in[1] = rows_of(k); a.out[1] = rows_of(k_out); a.heads[1] = s->heads_kv; }
  a.inv_freq = rope->inv_freq; a.rot = rope->rotary_dim; a.interleaved = rope->interleaved != 0;
  a.positions = positions; a.position_stride = position_stride; a.inverse = inverse != 0;
  a.b = s->batch; a.n = s->seq_len; a.d = s->head_dim;
  a.in_bf16 = s->dtype == HILS_BF16; a.out_bf16 = out_dtype == HILS_BF16;
  return cuda_status(hils::run_rotate(a, (cudaStream_t)stream));
}

hils_status hils_append_paged(const hils_shape* s, const hils_rows* k, const hils_rows* v, const hils_rows* q,
                              const hils_rows* q_out, int32_t n_new, const int32_t* cu_new,
                              const int32_t* new_lens, const int32_t* seq_lens, const int32_t* block_table,
                              int32_t max_chunks, int32_t n_pages, const hils_rope* rope, void* k_pages,
                              void* v_pages, int32_t* full_pages, void* ws, size_t ws_bytes, void* stream) {
  hils_status st = check_shape(s, false);
  if (st != HILS_OK) return st;
  if (n_new < 0 || (q == nullptr) != (q_out == nullptr) || (cu_new && new_lens)) return HILS_ERR_INVALID_ARG;
  if (rope && (st = check_rope(rope, s->head_dim)) != HILS_OK) return st;
  const long long tokens = cu_new ? n_new : (long long)s->batch * n_new;
  if (s->batch == 0) {  // every row is padding: no page is filled
    if (!full_pages || tokens < s->chunk) return HILS_OK;
    return cuda_status(cudaMemsetAsync(full_pages, 0xff, (size_t)(tokens / s->chunk) * 4, (cudaStream_t)stream));
  }
  if (tokens > 0x7fffffffll) return HILS_ERR_UNSUPPORTED;
  if (max_chunks <= 0 || n_pages <= 0) return HILS_ERR_INVALID_ARG;
  if (max_chunks > (0x7fffffff / s->chunk)) return HILS_ERR_UNSUPPORTED;  // positions are 32-bit
  if (!seq_lens || !block_table) return HILS_ERR_INVALID_ARG;
  if (!aligned4(seq_lens) || !aligned4(block_table) || !aligned4(cu_new) || !aligned4(new_lens) || !aligned4(full_pages))
    return HILS_ERR_INVALID_ARG;
  const size_t es = elem_size(s->dtype);
  if (tokens > 0) {
    if (!k_pages || !v_pages || !aligned16(k_pages) || !aligned16(v_pages)) return HILS_ERR_INVALID_ARG;
    const long long nb = cu_new ? 1 : s->batch;
    if ((st = check_rows(k, nb, s->heads_kv, n_new, es)) != HILS_OK ||
        (st = check_rows(v, nb, s->heads_kv, n_new, es)) != HILS_OK)
      return st;
    if (q && ((st = check_rows(q, nb, s->heads_q, n_new, es)) != HILS_OK ||
              (st = check_rows(q_out, nb, s->heads_q, n_new, es)) != HILS_OK))
      return st;
    const size_t pool = (size_t)n_pages * s->heads_kv * s->chunk * s->head_dim * es;
    const Span kp{reinterpret_cast<uintptr_t>(k_pages), reinterpret_cast<uintptr_t>(k_pages) + pool};
    const Span vp{reinterpret_cast<uintptr_t>(v_pages), reinterpret_cast<uintptr_t>(v_pages) + pool};
    const Span ki = span_of(k, nb, s->heads_kv, n_new, s->head_dim, es);
    const Span vi = span_of(v, nb, s->heads_kv, n_new, s->head_dim, es);
    if (overlap(kp, vp) || overlap(kp, ki) || overlap(kp, vi) || overlap(vp, ki) || overlap(vp, vi))
      return HILS_ERR_INVALID_ARG;
    if (q) {
      const Span qi = span_of(q, nb, s->heads_q, n_new, s->head_dim, es);
      const Span qo = span_of(q_out, nb, s->heads_q, n_new, s->head_dim, es);
      if (!rows_apart(q_out, nb, s->heads_q, n_new, s->head_dim)) return HILS_ERR_INVALID_ARG;
      if (overlap(qo, kp) || overlap(qo, vp) || overlap(qi, kp) || overlap(qi, vp)) return HILS_ERR_INVALID_ARG;
      const RowSet rows = row_set(q_out, nb, s->heads_q, n_new, s->head_dim, es);
      if ((!in_place(q_out, q, nb, s->heads_q, n_new) && sharing(rows, row_set(q, nb, s->heads_q, n_new, s->head_dim, es))) ||
          sharing(rows, row_set(k, nb, s->heads_kv, n_new, s->head_dim, es)) ||
          sharing(rows, row_set(v, nb, s->heads_kv, n_new, s->head_dim, es)))
        return HILS_ERR_INVALID_ARG;
    }
  } else if (!full_pages) {
    return HILS_OK;
  }
  if (!ws || ws_bytes < kHeader || !aligned16(ws)) return HILS_ERR_WORKSPACE;
  hils::AppendArgs a{};
  if (tokens > 0) {
    a.k = rows_of(k); a.v = rows_of(v);
    if (q) { a.q = rows_of(q); a.q_out = rows_of(q_out); a.h = s->heads_q; }
  }
  a.g = s->heads_kv; a.b = s->batch; a.d = s->head_dim; a.n_new = n_new;
  a.cu_new = cu_new; a.new_lens = new_lens; a.seq_lens = seq_lens; a.block_table = block_table;
  a.max_chunks = max_chunks; a.n_pages = n_pages;
  if (rope) { a.inv_freq = rope->inv_freq; a.rot = rope->rotary_dim; a.interleaved = rope->interleaved != 0; }
  a.bf16 = s->dtype == HILS_BF16; a.k_pages = k_pages; a.v_pages = v_pages;
  a.full_pages = full_pages;
  const long long slots = s->batch + tokens / s->chunk;
  if (slots > 0x7fffffffll) return HILS_ERR_UNSUPPORTED;
  a.n_slots = full_pages ? (int)slots : 0;
  a.err = static_cast<unsigned*>(ws);
  return cuda_status(hils::run_append(a, (cudaStream_t)stream));
}

hils_status hils_decode_dense(const hils_shape* s, const void* q, const void* k_pages, const void* v_pages,
                              const int32_t* block_table, int32_t max_chunks, const int32_t* seq_lens,
                              int32_t n_pages, void* out, float* lse_out, void* ws, size_t ws_bytes, void* stream) {
  hils_status st = check_shape(s, true, kAnyWindow);
  if (st != HILS_OK) return st;
  if (s->batch == 0) return HILS_OK;
  if (max_chunks <= 0 || n_pages <= 0) return HILS_ERR_INVALID_ARG;
  if ((long long)max_chunks > ((long long)s->seq_len + s->chunk - 1) / s->chunk) return HILS_ERR_INVALID_ARG;
  if (!q || !k_pages || !v_pages || !block_table || !seq_lens || !out) return HILS_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out)) return HILS_ERR_INVALID_ARG;
  if (!aligned4(block_table) || !aligned4(seq_lens) || !aligned4(lse_out)) return HILS_ERR_INVALID_ARG;
  if (!hils::decode_dense_supported(s->heads_kv, max_chunks, n_pages)) return HILS_ERR_UNSUPPORTED;
  {
    auto span = [](const void* p, size_t bytes) {
      const uintptr_t x = reinterpret_cast<uintptr_t>(p);
      return Span{x, x + bytes};
    };
    const size_t es = elem_size(s->dtype), row = (size_t)s->head_dim * es, nr = (size_t)s->batch * s->heads_q;
    const size_t pool = (size_t)n_pages * s->heads_kv * s->chunk * row;
    const Span o = span(out, nr * row), l = span(lse_out, lse_out ? nr * 4 : 0);
    for (const Span& in : {span(k_pages, pool), span(v_pages, pool), span(q, nr * row)})
      if (overlap(l, in) || (overlap(o, in) && o.lo != reinterpret_cast<uintptr_t>(q))) return HILS_ERR_INVALID_ARG;
    if (overlap(o, l)) return HILS_ERR_INVALID_ARG;
  }
  if (!ws || ws_bytes < dense_bytes(s) || !aligned16(ws)) return HILS_ERR_WORKSPACE;
  hils::DenseArgs a{};
  a.q = q; a.k_pages = k_pages; a.v_pages = v_pages; a.block_table = block_table; a.seq_lens = seq_lens;
  a.out = out; a.lse = lse_out; a.err = static_cast<unsigned*>(ws);
  a.b = s->batch; a.h = s->heads_q; a.g = s->heads_kv; a.d = s->head_dim;
  a.max_chunks = max_chunks; a.n_pages = n_pages; a.n_win = s->window / s->chunk;
  a.scale = eff_scale(s); a.bf16 = s->dtype == HILS_BF16; a.poll = g_wait_limit.load();
  return cuda_status(hils::run_decode_dense(a, static_cast<char*>(ws) + kHeader, (cudaStream_t)stream));
}

hils_status hils_device_status(void* ws, void* stream) {
  if (!ws) return HILS_ERR_INVALID_ARG;
  cudaStream_t cs = (cudaStream_t)stream;
  unsigned word = 0;
  if (cudaMemcpyAsync(&word, ws, sizeof(word), cudaMemcpyDeviceToHost, cs) != cudaSuccess)
    return HILS_ERR_CUDA;
  if (cudaStreamSynchronize(cs) != cudaSuccess) return HILS_ERR_CUDA;
  if (word != 0) {
    if (cudaMemsetAsync(ws, 0, sizeof(word), cs) != cudaSuccess) return HILS_ERR_CUDA;
    if (cudaStreamSynchronize(cs) != cudaSuccess) return HILS_ERR_CUDA;
  }
  if (word & hils::kErrTimeout) return HILS_ERR_DEVICE_TIMEOUT;
  if (word & hils::kErrBadPage) return HILS_ERR_DEVICE_CHECK;
  return HILS_OK;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// hils_decode_static: decode whose scratch is a device array owned by this
// file, for callers that cannot hand the library a workspace (no counterpart
// in the HiLS notes).  Nothing here allocates or frees device memory.
namespace {

constexpr size_t kStaticScratchBytes = HILS_DECODE_STATIC_SCRATCH_BYTES;
constexpr size_t kStaticTicketSlots = 4096;  // batch * heads_kv limit
constexpr int kStaticMaxDevices = 64;

// Scratch of hils_decode_static.  Byte layout (fixed parts first, so the ticket
// counters never share bytes with the data of a call of another shape):
//   [0, 256)                 error word, when the caller passes no status word
//   [256, 256 + 16 KiB)      scan tickets, one per (sequence, KV head)
//   [.., + 16 KiB)           attention tickets
//   then, per call's shape: part_keys, part_att, idx, sel_page, ssel
// The ticket counters must be zero when a call starts: device memory of a
// __device__ array is zero when the module is loaded, and every call that
// completes leaves them at zero (the CTA that consumes a ticket resets it).
static __device__ __align__(256) unsigned char g_decode_scratch[kStaticScratchBytes];

struct StaticLayout {
  size_t scan_ticket, att_ticket, part_keys, part_att, idx, sel_page, ssel, total;
};
StaticLayout static_decode_layout(const hils_shape* s) {
  const size_t b = s->batch, h = s->heads_q, g = s->heads_kv, K = s->top_k, d = s->head_dim;
  const size_t G = h / g;
  const int cmax = (s->seq_len + s->chunk - 1) / s->chunk;
  const size_t nsplit = hils::decode_splits(s->batch, cmax);
  StaticLayout L;
  size_t off = kHeader;
  L.scan_ticket = off; off += kStaticTicketSlots * 4;
  L.att_ticket = off; off += kStaticTicketSlots * 4;
  L.part_keys = off; off = align_up(off + b * g * nsplit * K * 8);
  L.part_att = off; off = align_up(off + b * g * 2 * (K + n_local(s)) * G * (d + 2) * 4);  // half-chunk partials
  L.idx = off; off = align_up(off + b * g * K * 4);
  L.sel_page = off; off = align_up(off + b * g * K * 4);
  L.ssel = off; off = align_up(off + b * h * K * 4);
  L.total = off;
  return L;
}

std::mutex g_static_mu;
unsigned char* g_static_ptr[kStaticMaxDevices];

// Device address of the scratch array on the current device, looked up once
// per device (the lookup may load this library's device code onto it).
cudaError_t static_scratch(unsigned char** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kStaticMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_static_mu);
  if (!g_static_ptr[dev]) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_decode_scratch);
    if (e != cudaSuccess) return e;
    g_static_ptr[dev] = static_cast<unsigned char*>(p);
  }
  *out = g_static_ptr[dev];
  return cudaSuccess;
}

}  // namespace

extern "C" {

hils_status hils_decode_static(const hils_shape* s, const void* q, const void* k_pages, const void* v_pages,
                               const float* kbar_pages, const float* hbias_pages, const int32_t* block_table,
                               int32_t max_chunks, const int32_t* seq_lens, int32_t n_pages, void* out,
                               int32_t* topk_idx_out, unsigned* status_word, void* stream) {
  hils_status st = check_shape(s, true);
  if (st != HILS_OK) return st;
  if (s->batch == 0) return HILS_OK;
  if (!hils::decode_supported(s->heads_q, s->head_dim) || n_local(s) > kMaxDecodeLocal) return HILS_ERR_UNSUPPORTED;
  if (max_chunks <= 0 || n_pages <= 0) return HILS_ERR_INVALID_ARG;
  if ((long long)max_chunks > ((long long)s->seq_len + s->chunk - 1) / s->chunk) return HILS_ERR_INVALID_ARG;
  if (!hils::decode_merge_supported(s->batch, max_chunks, s->top_k)) return HILS_ERR_UNSUPPORTED;
  if (!q || !k_pages || !v_pages || !kbar_pages || !hbias_pages || !block_table || !seq_lens || !out)
    return HILS_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(kbar_pages) ||
      !aligned16(out) || (reinterpret_cast<uintptr_t>(status_word) & 3u) != 0)
    return HILS_ERR_INVALID_ARG;
  if ((size_t)s->batch * s->heads_kv > kStaticTicketSlots) return HILS_ERR_WORKSPACE;
  const StaticLayout L = static_decode_layout(s);
  if (L.total > kStaticScratchBytes) return HILS_ERR_WORKSPACE;
  unsigned char* w = nullptr;
  if (static_scratch(&w) != cudaSuccess) return HILS_ERR_CUDA;
  hils::DecodeArgs da{};
  da.q = q; da.k_pages = k_pages; da.v_pages = v_pages; da.kbar_pages = kbar_pages;
  da.hbias_pages = hbias_pages; da.block_table = block_table; da.seq_lens = seq_lens; da.out = out;
  da.idx = topk_idx_out ? topk_idx_out : reinterpret_cast<int32_t*>(w + L.idx);
  da.ssel = reinterpret_cast<float*>(w + L.ssel);
  da.sel_page = reinterpret_cast<int32_t*>(w + L.sel_page);
  da.part_keys = reinterpret_cast<unsigned long long*>(w + L.part_keys);
  da.part_att = reinterpret_cast<float*>(w + L.part_att);
  da.scan_ticket = reinterpret_cast<unsigned*>(w + L.scan_ticket);
  da.att_ticket = reinterpret_cast<unsigned*>(w + L.att_ticket);
  da.err = status_word ? status_word : reinterpret_cast<unsigned*>(w);
  da.b = s->batch; da.h = s->heads_q; da.g = s->heads_kv; da.d = s->head_dim; da.top_k = s->top_k;
  da.max_chunks = max_chunks; da.n_pages = n_pages; da.scale = eff_scale(s);
  da.bf16 = s->dtype == HILS_BF16;
  da.n_local = n_local(s);
  return cuda_status(hils::run_decode(da, (cudaStream_t)stream));
}

}  // extern "C"
