// Host/device interface of the serving cache: cache writes and reads, and the
// attention that reads the cache. GPU-library only.
#pragma once
#include "kvc.h"
#include "kvc_internal.h"

namespace kvc {

// A validated cache description, passed to kernels by value.
struct CacheView {
  uint8_t* codes;
  float* scales;
  uint8_t* micro;
  uint32_t fmt, H, D, n_pages;
  uint32_t page_shift, page_mask;  // page_tokens is a power of two
  uint32_t row_bytes;              // code bytes of a row: D, or D / 2
};
// Row (page, kv, head, 0); rows of consecutive tokens follow.
__host__ __device__ inline uint64_t cache_row(const CacheView& c, uint32_t page, uint32_t kv, uint32_t h) {
  return ((uint64_t(page) * 2u + kv) * c.H + h) << c.page_shift;
}

struct WriteArgs {
  const void *k, *v;
  int64_t k_tok, k_head, v_tok, v_head;  // in values
  const int64_t* slots;
  kvc_result* res;
  uint32_t dtype, n_tokens;
};
cudaError_t launch_cache_write(const CacheView& c, const WriteArgs& a, cudaStream_t st);

struct ReadArgs {
  const int32_t *pages, *start, *out_start;
  void* out;
  kvc_result* res;
  uint32_t dtype, n_seqs, pages_stride, out_tokens;
};
cudaError_t launch_cache_read(const CacheView& c, const ReadArgs& a, cudaStream_t st);

// Attention arguments as kernels take them.
struct AttendArgs {
  const void* q;
  void* out;
  float* lse;
  const int32_t *q_start, *pages, *kv_len, *prefix_len;
  const void *pk, *pv;
  kvc_result* res;
  int64_t q_tok, q_head, o_tok, o_head, p_head;  // in values
  float scale_log2;                              // scale * log2(e)
  uint32_t dtype, n_rows, Hq, H, G, D, n_seqs, pages_stride, prefix_tokens;
  uint32_t has_cache;
};
cudaError_t launch_attend(const AttendArgs& a, const CacheView& c, uint32_t max_queries, uint32_t max_kv, void* ws,
                          size_t ws_bytes, cudaStream_t st);
uint64_t attend_ws_bytes(const AttendArgs& a, uint32_t max_queries, uint32_t max_kv, bool least);

#ifdef __CUDACC__
// Sticky status in the caller's result; of two the larger code stays, whichever
// comes first: KVC_ERR_TIMEOUT before KVC_ERR_INVALID.
__device__ inline void flag_status(kvc_result* res, int32_t status) {
  if (res) atomicMax(&res->status, status);
}
// An index the device refuses to follow.
__device__ inline void flag_invalid(kvc_result* res) { flag_status(res, KVC_ERR_INVALID); }
#endif

}  // namespace kvc
