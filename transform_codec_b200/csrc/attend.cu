// Attention over the serving cache and a shared prefix (include/kvc.h,
// kvc_attend). One block per query row and head: its warps take every fourth
// token of the prefix and of the sequence's cache, each with a running maximum
// and sum, and are joined at the end.
#include "cache_codes.cuh"
#include "serving.h"

namespace kvc {
namespace {

constexpr uint32_t kWarps = 4;

struct RowPlace {
  int32_t seq, first, last;  // sequence (-1: none) and its rows
};
__device__ inline RowPlace place_of(const AttendArgs& a, int32_t i) {
  if (!a.q_start) return {i < int32_t(a.n_seqs) ? i : -1, i, i + 1};
  uint32_t lo = 0, hi = a.n_seqs - 1;
  while (lo < hi) {
    const uint32_t mid = (lo + hi + 1) >> 1;
    if (__ldg(a.q_start + mid) <= i) lo = mid; else hi = mid - 1;
  }
  const int32_t first = __ldg(a.q_start + lo), last = __ldg(a.q_start + lo + 1);
  if (i < first || i >= last) return {-1, 0, 0};
  if (first < 0 || last > int32_t(a.n_rows)) {
    flag_invalid(a.res);
    return {-1, 0, 0};
  }
  return {int32_t(lo), first, last};
}

__device__ inline float code_value(const CacheView& c, uint64_t row, uint32_t ch) {
  const uint8_t* p = c.codes + row * c.row_bytes;
  if (c.fmt == KVC_CACHE_E4M3) return e4m3_f32(p[ch]);
  if (c.fmt == KVC_CACHE_INT8) return float(int8_t(p[ch]));
  const float2 f = half2_f32(e2m1x2_half2(p[ch >> 1]));
  return (ch & 1 ? f.y : f.x) * e4m3_f32(c.micro[row * (c.D / 16u) + ch / 16u]);
}
__device__ inline float value16(uint32_t dtype, const void* p, int64_t at) {
  const uint32_t w = static_cast<const uint16_t*>(p)[at];
  return dtype == KVC_DTYPE_BF16 ? bf16_lo(w) : half2_f32(w).x;
}

template <uint32_t NC>  // channels a lane
__global__ void __launch_bounds__(kWarps * 32) k_attend_rows(const AttendArgs a, const CacheView c) {
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int32_t i = int32_t(blockIdx.x);
  const uint32_t hq = blockIdx.y, h = hq / a.G;
  const RowPlace at = place_of(a, i);
  if (at.seq < 0) return;
  float q[NC], acc[NC], m = -INFINITY, l = 0.f;
#pragma unroll
  for (uint32_t j = 0; j < NC; ++j) {
    q[j] = value16(a.dtype, a.q, i * a.q_tok + hq * a.q_head + lane * NC + j) * a.scale_log2;
    acc[j] = 0.f;
  }
  auto step = [&](const float* k, const float* v) {
    float s = 0.f;
#pragma unroll
    for (uint32_t j = 0; j < NC; ++j) s = fmaf(q[j], k[j], s);
    for (uint32_t o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float m2 = s > m ? s : m;
    const float f = m2 == m ? 1.f : exp2f(m - m2), p = m2 == -INFINITY ? (s == s ? 0.f : s) : exp2f(s - m2);
    l = fmaf(l, f, p);
#pragma unroll
    for (uint32_t j = 0; j < NC; ++j) acc[j] = fmaf(acc[j], f, p * v[j]);
    m = m2;
  };
  float k[NC], v[NC];
  if (a.prefix_tokens) {
    int32_t n = int32_t(a.prefix_tokens);
    if (a.prefix_len) {
      const int32_t w = __ldg(a.prefix_len + at.seq);
      if (w < 0 || w > n) flag_invalid(a.res);
      n = max(0, min(w, n));
    }
    for (int32_t t = int32_t(warp); t < n; t += kWarps) {
      const int64_t o = h * a.p_head + int64_t(t) * a.D + lane * NC;
#pragma unroll
      for (uint32_t j = 0; j < NC; ++j) {
        k[j] = value16(a.dtype, a.pk, o + j);
        v[j] = value16(a.dtype, a.pv, o + j);
      }
      step(k, v);
    }
  }
  if (a.has_cache) {
    int64_t len = __ldg(a.kv_len + at.seq);
    const int64_t room = int64_t(a.pages_stride) << c.page_shift;
    if (len < 0 || len > room) flag_invalid(a.res);
    len = max(int64_t(0), min(len, room));
    const int64_t sees = len - (at.last - at.first) + (i - at.first) + 1;
    for (int64_t t = warp; t < sees; t += kWarps) {
      const int32_t page = __ldg(a.pages + uint64_t(at.seq) * a.pages_stride + (t >> c.page_shift));
      if (page < 0 || uint32_t(page) >= c.n_pages) {
        flag_invalid(a.res);
        continue;
      }
      const uint64_t rk = cache_row(c, page, 0, h) + (t & c.page_mask), rv = cache_row(c, page, 1, h) + (t & c.page_mask);
      const float sk = c.scales[rk], sv = c.scales[rv];
#pragma unroll
      for (uint32_t j = 0; j < NC; ++j) {
        k[j] = code_value(c, rk, lane * NC + j) * sk;
        v[j] = code_value(c, rv, lane * NC + j) * sv;
      }
      step(k, v);
    }
  }
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][NC * 32];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (uint32_t j = 0; j < NC; ++j) so[warp][lane * NC + j] = acc[j];
  __syncthreads();
  if (warp) return;
  float top = -INFINITY, sum = 0.f;
  for (uint32_t w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
#pragma unroll
  for (uint32_t j = 0; j < NC; ++j) acc[j] = 0.f;
  for (uint32_t w = 0; w < kWarps; ++w) {
    const float f = sm[w] == -INFINITY ? (sl[w] == 0.f ? 0.f : NAN) : exp2f(sm[w] - top);
    sum = fmaf(sl[w], f, sum);
    for (uint32_t j = 0; j < NC; ++j) acc[j] = fmaf(so[w][lane * NC + j], f, acc[j]);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  for (uint32_t j = 0; j < NC; ++j) {
    const float y = acc[j] * inv;
    const int64_t o = i * a.o_tok + hq * a.o_head + lane * NC + j;
    static_cast<uint16_t*>(a.out)[o] =
        uint16_t(a.dtype == KVC_DTYPE_BF16 ? pack_bf16(y, y) : pack_half(y, y));
  }
  if (a.lse && lane == 0)
    a.lse[uint64_t(i) * a.Hq + hq] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace

uint64_t attend_ws_bytes(const AttendArgs&, uint32_t, uint32_t, bool) { return 0; }

cudaError_t launch_attend(const AttendArgs& a, const CacheView& c, uint32_t, uint32_t, void*, size_t,
                          cudaStream_t st) {
  ProfRange p("attend_rows", st);
  const dim3 grid(a.n_rows, a.Hq);
  if (a.D == 64)
    k_attend_rows<2><<<grid, kWarps * 32, 0, st>>>(a, c);
  else
    k_attend_rows<4><<<grid, kWarps * 32, 0, st>>>(a, c);
  return cudaGetLastError();
}

}  // namespace kvc
