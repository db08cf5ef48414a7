// Host side of the serving cache (include/kvc.h): argument checks and launches
// of the cache write, the cache read and the attention. Nothing here allocates
// or synchronises.
#include <cmath>

#include "serving.h"

using namespace kvc;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
uint32_t value_bytes(uint32_t dtype) {
  return dtype == KVC_DTYPE_F32 ? 4u : dtype == KVC_DTYPE_BF16 || dtype == KVC_DTYPE_FP16 ? 2u : 0u;
}
bool stride_ok(int64_t s, uint32_t vb) { return (uint64_t(s) * vb) % 16u == 0; }

// Shape fields only.
bool cache_shape_ok(const kvc_cache* c) {
  if (!c || c->reserved) return false;
  if (c->format < KVC_CACHE_E4M3 || c->format > KVC_CACHE_E2M1) return false;
  if (!c->n_heads || c->n_heads > 65535u || !c->n_pages || c->n_pages > 0x7fffffffu) return false;
  if (c->head_dim < 32 || c->head_dim > 256 || c->head_dim % 32u) return false;
  if (c->page_tokens < 16 || c->page_tokens > 1024 || (c->page_tokens & (c->page_tokens - 1))) return false;
  // rows stay far below 2^55, so byte offsets (at most 256 bytes a row) fit 64 bits
  return uint64_t(c->n_pages) * 2u * c->n_heads < (uint64_t(1) << 45);
}
uint64_t cache_rows(const kvc_cache* c) { return uint64_t(c->n_pages) * 2u * c->n_heads * c->page_tokens; }

// KVC_OK and the kernels' view of the cache.
int cache_view(const kvc_cache* c, CacheView& v) {
  if (!cache_shape_ok(c)) return KVC_ERR_INVALID;
  const bool micro = c->format == KVC_CACHE_E2M1;
  if (!c->d_codes || !c->d_scales || !aligned16(c->d_codes) || !aligned16(c->d_scales)) return KVC_ERR_INVALID;
  if (micro != (c->d_micro != nullptr) || !aligned16(c->d_micro)) return KVC_ERR_INVALID;
  v.codes = static_cast<uint8_t*>(c->d_codes);
  v.scales = c->d_scales;
  v.micro = static_cast<uint8_t*>(c->d_micro);
  v.fmt = c->format;
  v.H = c->n_heads;
  v.D = c->head_dim;
  v.n_pages = c->n_pages;
  v.page_shift = 0;
  while ((1u << v.page_shift) < c->page_tokens) ++v.page_shift;
  v.page_mask = c->page_tokens - 1;
  v.row_bytes = micro ? c->head_dim / 2 : c->head_dim;
  return KVC_OK;
}

// Checks a description and turns it into the kernels' arguments.
int attend_args(const kvc_attend_desc* d, AttendArgs& a, CacheView& cv, bool pointers) {
  if (!d || d->reserved) return KVC_ERR_INVALID;
  if (d->dtype != KVC_DTYPE_BF16 && d->dtype != KVC_DTYPE_FP16) return KVC_ERR_INVALID;
  if (!d->n_heads || !d->n_q_heads || d->n_q_heads % d->n_heads) return KVC_ERR_INVALID;
  if (d->n_q_heads > 65535u || d->n_rows > 0x7fffffffu || d->n_seqs > 65535u) return KVC_ERR_INVALID;
  if (uint64_t(d->n_rows) * d->n_q_heads > 0x7fffffffu) return KVC_ERR_INVALID;
  if (d->prefix_tokens > 0x7fffffffu || d->max_kv > 0x7fffffffu) return KVC_ERR_INVALID;
  if (!d->prefix_tokens && !d->cache) return KVC_ERR_INVALID;
  if (!std::isfinite(d->scale)) return KVC_ERR_INVALID;
  if (d->head_dim != 64 && d->head_dim != 128) return KVC_ERR_UNSUPPORTED;
  cv = CacheView{};
  if (d->cache) {
    if (pointers) {
      const int st = cache_view(d->cache, cv);
      if (st != KVC_OK) return st;
    } else if (!cache_shape_ok(d->cache)) {
      return KVC_ERR_INVALID;
    }
    if (d->cache->n_heads != d->n_heads || d->cache->head_dim != d->head_dim) return KVC_ERR_INVALID;
  }
  if (pointers) {
    const uint32_t vb = 2;
    if (!d->d_q || !d->d_out || !aligned16(d->d_q) || !aligned16(d->d_out)) return KVC_ERR_INVALID;
    if (!stride_ok(d->q_token_stride, vb) || !stride_ok(d->q_head_stride, vb) ||
        !stride_ok(d->out_token_stride, vb) || !stride_ok(d->out_head_stride, vb))
      return KVC_ERR_INVALID;
    if (d->cache && (!d->d_pages || !d->d_kv_len || !d->pages_stride)) return KVC_ERR_INVALID;
    if (d->prefix_tokens) {
      if (!d->d_prefix_k || !d->d_prefix_v || !aligned16(d->d_prefix_k) || !aligned16(d->d_prefix_v))
        return KVC_ERR_INVALID;
      if (d->prefix_head_stride < 0 || !stride_ok(d->prefix_head_stride, vb)) return KVC_ERR_INVALID;
      if (d->n_heads > 1 && uint64_t(d->prefix_head_stride) < uint64_t(d->prefix_tokens) * d->head_dim)
        return KVC_ERR_INVALID;
    }
  }
  a = AttendArgs{};
  a.q = d->d_q;
  a.out = d->d_out;
  a.lse = d->d_lse;
  a.q_start = d->d_q_start;
  a.pages = d->d_pages;
  a.kv_len = d->d_kv_len;
  a.prefix_len = d->d_prefix_len;
  a.pk = d->d_prefix_k;
  a.pv = d->d_prefix_v;
  a.q_tok = d->q_token_stride;
  a.q_head = d->q_head_stride;
  a.o_tok = d->out_token_stride;
  a.o_head = d->out_head_stride;
  a.p_head = d->prefix_head_stride;
  // a scale of (almost) zero weighs all tokens alike; kept off zero, where a
  // hidden token's -infinity would lose its meaning
  const double sl = double(d->scale) * 1.4426950408889634;
  a.scale_log2 = std::fabs(sl) < 1e-30 ? 1e-30f : float(sl);
  if (!std::isfinite(a.scale_log2)) return KVC_ERR_INVALID;
  a.dtype = d->dtype;
  a.n_rows = d->n_rows;
  a.Hq = d->n_q_heads;
  a.H = d->n_heads;
  a.G = d->n_q_heads / d->n_heads;
  a.D = d->head_dim;
  a.n_seqs = d->n_seqs;
  a.pages_stride = d->pages_stride;
  a.prefix_tokens = d->prefix_tokens;
  a.has_cache = d->cache != nullptr;
  return KVC_OK;
}

}  // namespace

extern "C" int kvc_cache_bytes(const kvc_cache* cache, size_t* codes, size_t* scales, size_t* micro) {
  if (!cache_shape_ok(cache)) return KVC_ERR_INVALID;
  const uint64_t rows = cache_rows(cache);
  const bool m = cache->format == KVC_CACHE_E2M1;
  if (codes) *codes = size_t(rows * (m ? cache->head_dim / 2 : cache->head_dim));
  if (scales) *scales = size_t(rows * sizeof(float));
  if (micro) *micro = m ? size_t(rows * (cache->head_dim / 16)) : 0;
  return KVC_OK;
}

extern "C" int kvc_cache_write(const kvc_cache* cache, uint32_t dtype, uint32_t n_tokens, const void* d_k,
                               int64_t k_token_stride, int64_t k_head_stride, const void* d_v,
                               int64_t v_token_stride, int64_t v_head_stride, const int64_t* d_slots,
                               kvc_result* d_res, cudaStream_t stream) {
  CacheView c;
  const int st = cache_view(cache, c);
  if (st != KVC_OK) return st;
  const uint32_t vb = value_bytes(dtype);
  if (!vb || n_tokens > 0x7fffffffu) return KVC_ERR_INVALID;
  if (!n_tokens) return KVC_OK;
  if (!d_k || !d_v || !d_slots || !aligned16(d_k) || !aligned16(d_v)) return KVC_ERR_INVALID;
  if ((reinterpret_cast<uintptr_t>(d_slots) & 7u) || (reinterpret_cast<uintptr_t>(d_res) & 7u)) return KVC_ERR_INVALID;
  if (!stride_ok(k_token_stride, vb) || !stride_ok(k_head_stride, vb) || !stride_ok(v_token_stride, vb) ||
      !stride_ok(v_head_stride, vb))
    return KVC_ERR_INVALID;
  const WriteArgs a{d_k,    d_v,     k_token_stride, k_head_stride, v_token_stride, v_head_stride,
                    d_slots, d_res, dtype,          n_tokens};
  return launch_cache_write(c, a, stream) == cudaSuccess ? KVC_OK : KVC_ERR_CUDA;
}

extern "C" int kvc_cache_read(const kvc_cache* cache, uint32_t dtype, uint32_t n_seqs, const int32_t* d_pages,
                              uint32_t pages_stride, const int32_t* d_start, const int32_t* d_out_start,
                              void* d_out, uint32_t out_tokens, kvc_result* d_res, cudaStream_t stream) {
  CacheView c;
  const int st = cache_view(cache, c);
  if (st != KVC_OK) return st;
  if (!value_bytes(dtype) || out_tokens > 0x7fffffffu || n_seqs > 0x7ffffffeu) return KVC_ERR_INVALID;
  if (!n_seqs || !out_tokens) return KVC_OK;
  if (!d_pages || !pages_stride || !d_start || !d_out_start || !d_out || !aligned16(d_out)) return KVC_ERR_INVALID;
  if ((reinterpret_cast<uintptr_t>(d_pages) & 3u) || (reinterpret_cast<uintptr_t>(d_start) & 3u) ||
      (reinterpret_cast<uintptr_t>(d_out_start) & 3u) || (reinterpret_cast<uintptr_t>(d_res) & 7u))
    return KVC_ERR_INVALID;
  const ReadArgs a{d_pages, d_start, d_out_start, d_out, d_res, dtype, n_seqs, pages_stride, out_tokens};
  return launch_cache_read(c, a, stream) == cudaSuccess ? KVC_OK : KVC_ERR_CUDA;
}

extern "C" size_t kvc_attend_workspace_bytes(const kvc_attend_desc* desc) {
  AttendArgs a;
  CacheView c;
  if (attend_args(desc, a, c, false) != KVC_OK) return 0;
  return size_t(attend_ws_bytes(a, desc->max_queries, desc->max_kv, false));
}

extern "C" size_t kvc_attend_workspace_min(const kvc_attend_desc* desc) {
  AttendArgs a;
  CacheView c;
  if (attend_args(desc, a, c, false) != KVC_OK) return 0;
  return size_t(attend_ws_bytes(a, desc->max_queries, desc->max_kv, true));
}

extern "C" int kvc_attend(const kvc_attend_desc* desc, void* d_ws, size_t ws_bytes, kvc_result* d_res,
                          cudaStream_t stream) {
  AttendArgs a;
  CacheView c;
  // a step without rows or sequences has empty arrays, whose addresses may be NULL
  const bool work = desc && desc->n_rows && desc->n_seqs;
  const int st = attend_args(desc, a, c, work);
  if (st != KVC_OK) return st;
  if (!desc->d_q_start && desc->n_rows < desc->n_seqs) return KVC_ERR_INVALID;  // sequence b is row b
  if (!aligned16(d_ws) || (reinterpret_cast<uintptr_t>(d_res) & 7u)) return KVC_ERR_INVALID;
  const uintptr_t words = reinterpret_cast<uintptr_t>(a.lse) | reinterpret_cast<uintptr_t>(a.q_start) |
                          reinterpret_cast<uintptr_t>(a.pages) | reinterpret_cast<uintptr_t>(a.kv_len) |
                          reinterpret_cast<uintptr_t>(a.prefix_len);
  if (words & 3u) return KVC_ERR_INVALID;
  if (!work) return KVC_OK;
  if (!d_ws) ws_bytes = 0;
  if (ws_bytes < attend_ws_bytes(a, desc->max_queries, desc->max_kv, true)) return KVC_ERR_CAPACITY;
  a.res = d_res;
  return launch_attend(a, c, desc->max_queries, desc->max_kv, d_ws, ws_bytes, stream) == cudaSuccess ? KVC_OK
                                                                                                      : KVC_ERR_CUDA;
}
