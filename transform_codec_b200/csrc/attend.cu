// Attention over the serving cache and a shared prefix (include/kvc.h,
// kvc_attend): launches, the division of work into parts, and their join.
#include "attend_cache.cuh"
#include "attend_parts.cuh"

namespace kvc {
namespace {

// Prefix: one block per query row and head, for now.
constexpr uint32_t kRowWarps = 4;
__device__ inline float value16(uint32_t dtype, const void* p, int64_t at) {
  const uint32_t w = static_cast<const uint16_t*>(p)[at];
  return dtype == KVC_DTYPE_BF16 ? bf16_lo(w) : half2_f32(w).x;
}
template <uint32_t NC>
__global__ void __launch_bounds__(kRowWarps * 32) k_attend_prefix_rows(const AttendArgs a, const PartsView parts) {
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int32_t i = int32_t(blockIdx.x);
  const uint32_t hq = blockIdx.y, h = hq / a.G;
  const RowPlace at = place_of_row(a, i);
  if (at.seq < 0) return;
  float q[NC], acc[NC], m = -INFINITY, l = 0.f;
#pragma unroll
  for (uint32_t j = 0; j < NC; ++j) {
    q[j] = value16(a.dtype, a.q, i * a.q_tok + hq * a.q_head + lane * NC + j) * a.scale_log2;
    acc[j] = 0.f;
  }
  const int32_t n = int32_t(prefix_seen(a, at.seq));
  for (int32_t t = int32_t(warp); t < n; t += kRowWarps) {
    const int64_t off = h * a.p_head + int64_t(t) * a.D + lane * NC;
    float s = 0.f;
#pragma unroll
    for (uint32_t j = 0; j < NC; ++j) s = fmaf(q[j], value16(a.dtype, a.pk, off + j), s);
    for (uint32_t o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float m2 = s > m ? s : m;
    const float f = m2 == m ? 1.f : exp2f(m - m2), p = exp2f(s - m2);
    l = fmaf(l, f, p);
#pragma unroll
    for (uint32_t j = 0; j < NC; ++j) acc[j] = fmaf(acc[j], f, p * value16(a.dtype, a.pv, off + j));
    m = m2;
  }
  __shared__ float sm[kRowWarps], sl[kRowWarps], so[kRowWarps][NC * 32];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (uint32_t j = 0; j < NC; ++j) so[warp][lane * NC + j] = acc[j];
  __syncthreads();
  if (warp) return;
  float top = -INFINITY, sum = 0.f;
  for (uint32_t w = 0; w < kRowWarps; ++w) top = fmaxf(top, sm[w]);
#pragma unroll
  for (uint32_t j = 0; j < NC; ++j) acc[j] = 0.f;
  for (uint32_t w = 0; w < kRowWarps; ++w) {
    const float f = sl[w] == 0.f ? 0.f : exp2f(sm[w] - top);
    sum = fmaf(sl[w], f, sum);
    for (uint32_t j = 0; j < NC; ++j) acc[j] = fmaf(so[w][lane * NC + j], f, acc[j]);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const uint64_t id = uint64_t(i) * a.Hq + hq;
  for (uint32_t j = 0; j < NC; ++j) parts.o[id * a.D + lane * NC + j] = acc[j] * inv;
  if (lane == 0) parts.lse[id] = sum == 0.f ? -INFINITY : top + log2f(sum);
}

// Join the parts of each row: a warp a row, D / 32 channels a lane. Reads parts *
// (D + 1) * 4 bytes a row.
constexpr uint32_t kJoinWarps = 4;
template <uint32_t D>
__global__ void __launch_bounds__(kJoinWarps * 32)
k_attend_join(const AttendArgs a, const CacheView c, const PartsView parts, const uint32_t prefix_parts,
              const uint32_t splits) {
  constexpr uint32_t kPer = D / 32;
  const uint32_t lane = threadIdx.x & 31u;
  const uint64_t id = uint64_t(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5);
  if (id >= parts.rows) return;
  const int32_t i = int32_t(id / a.Hq);
  const uint32_t hq = uint32_t(id % a.Hq);
  const RowPlace at = place_of_row(a, i);
  if (at.seq < 0) return;
  uint32_t n = prefix_parts;
  if (a.has_cache) {
    const uint32_t own = chunks_of(cache_len(a, c, at.seq), splits).parts;
    if (own == 1 && !prefix_parts) return;  // written by the part itself
    n += own;
  }
  float top = -INFINITY;
  for (uint32_t p = lane; p < n; p += 32) top = fmaxf(top, parts.lse[p * parts.rows + id]);
#pragma unroll
  for (uint32_t o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float sum = 0.f, y[kPer];
#pragma unroll
  for (uint32_t j = 0; j < kPer; ++j) y[j] = 0.f;
  for (uint32_t p0 = 0; p0 < n; p0 += 32) {
    float f = 0.f;
    if (p0 + lane < n) {
      const float L = parts.lse[(p0 + lane) * parts.rows + id];
      f = L == -INFINITY ? 0.f : ex2(L - top);
    }
    const uint32_t here = min(32u, n - p0);
#pragma unroll 4
    for (uint32_t p = 0; p < here; ++p) {
      const float w = __shfl_sync(0xffffffffu, f, p);
      const float* src = parts.o + ((p0 + p) * parts.rows + id) * D + lane * kPer;
      float v[4];
      if (kPer == 4) {
        const float4 x = *reinterpret_cast<const float4*>(src);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(src);
        v[0] = x.x, v[1] = x.y;
      }
      sum += w;
#pragma unroll
      for (uint32_t j = 0; j < kPer; ++j) y[j] = fmaf(w, v[j], y[j]);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (uint32_t j = 0; j < kPer; ++j) y[j] *= inv;
  store_out<kPer>(a, i, hq, lane * kPer, y);
  if (a.lse && lane == 0) a.lse[id] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// ---- how a call is divided

constexpr uint32_t kSMs = 148;
struct Division {
  uint32_t row_tiles;      // 8-row tiles a block takes: 1 or 2
  uint32_t row_groups;     // blocks along a sequence's query rows
  uint32_t splits;         // parts of a sequence's cache tokens at most
  uint32_t prefix_parts;
  uint32_t parts;          // of a row at most
};

uint64_t parts_bytes(const AttendArgs& a, uint64_t parts) {
  const uint64_t rows = uint64_t(a.n_rows) * a.Hq;
  return (parts * rows * sizeof(float) + 15) / 16 * 16 + parts * rows * a.D * sizeof(float);
}

// most: parts that the workspace has room for
Division divide(const AttendArgs& a, uint32_t max_queries, uint32_t max_kv, uint64_t most) {
  Division d{1, 1, 1, a.prefix_tokens ? 1u : 0u, 1};
  if (a.has_cache) {
    const uint64_t rows = uint64_t(std::max(max_queries, 1u)) * a.G;
    d.row_tiles = rows > 8 ? 2 : 1;
    d.row_groups = uint32_t(std::min<uint64_t>((rows + 8 * d.row_tiles - 1) / (8 * d.row_tiles), 4096u));
    // One wave of blocks (3 an SM) is filled with parts of at least 64 tokens;
    // with more blocks than that, parts of about 1024 tokens until there are
    // some six waves, so that sequences of different lengths even out.
    const uint64_t wave = kSMs * 3, blocks = uint64_t(a.n_seqs) * a.H * d.row_groups;
    const uint64_t fine = std::max<uint64_t>(1, (uint64_t(max_kv) + kLeastTiles * kTile - 1) / (kLeastTiles * kTile));
    const uint64_t coarse = std::max<uint64_t>(1, uint64_t(max_kv) / 1024);
    uint64_t s = std::min(fine, std::max<uint64_t>(1, wave / std::max<uint64_t>(blocks, 1)));
    s = std::max(s, std::min(coarse, std::max<uint64_t>(1, 6 * wave / std::max<uint64_t>(blocks, 1))));
    s = std::min<uint64_t>(s, 512);
    if (s + d.prefix_parts > 1 && s + d.prefix_parts > most) s = most > d.prefix_parts + 1 ? most - d.prefix_parts : 1;
    d.splits = uint32_t(s);
  }
  d.parts = d.prefix_parts + (a.has_cache ? d.splits : 0);
  return d;
}

template <uint32_t FMT, uint32_t D, uint32_t R>
cudaError_t run_cache(const AttendArgs& a, const CacheView& c, const PartsView& parts, const Division& d,
                      cudaStream_t st) {
  using T = CacheTile<FMT, D, R>;
  static SmemAttr track;
  cudaError_t e = smem_attr(track, reinterpret_cast<const void*>(k_attend_cache<FMT, D, R>), T::kSmem);
  if (e != cudaSuccess) return e;
  ProfRange p("attend_cache", st);
  k_attend_cache<FMT, D, R><<<dim3(d.row_groups * d.splits, a.H, a.n_seqs), T::kThreads, T::kSmem, st>>>(
      a, c, parts, d.prefix_parts, d.splits, d.row_groups);
  return cudaGetLastError();
}
template <uint32_t FMT, uint32_t D>
cudaError_t pick_cache(const AttendArgs& a, const CacheView& c, const PartsView& parts, const Division& d,
                       cudaStream_t st) {
  return d.row_tiles == 1 ? run_cache<FMT, D, 1>(a, c, parts, d, st) : run_cache<FMT, D, 2>(a, c, parts, d, st);
}
template <uint32_t D>
cudaError_t run_all(const AttendArgs& a, const CacheView& c, const PartsView& parts, const Division& d,
                    cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (a.prefix_tokens) {
    ProfRange p("attend_prefix", st);
    k_attend_prefix_rows<D / 32><<<dim3(a.n_rows, a.Hq), kRowWarps * 32, 0, st>>>(a, parts);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (a.has_cache) {
    e = c.fmt == KVC_CACHE_E4M3   ? pick_cache<KVC_CACHE_E4M3, D>(a, c, parts, d, st)
        : c.fmt == KVC_CACHE_INT8 ? pick_cache<KVC_CACHE_INT8, D>(a, c, parts, d, st)
                                  : pick_cache<KVC_CACHE_E2M1, D>(a, c, parts, d, st);
    if (e != cudaSuccess) return e;
  }
  if (d.parts == 1 && !a.prefix_tokens) return e;
  ProfRange p("attend_join", st);
  const uint64_t blocks = (parts.rows + kJoinWarps - 1) / kJoinWarps;
  k_attend_join<D><<<uint32_t(blocks), kJoinWarps * 32, 0, st>>>(a, c, parts, d.prefix_parts, d.splits);
  return cudaGetLastError();
}

}  // namespace

uint64_t attend_ws_bytes(const AttendArgs& a, uint32_t max_queries, uint32_t max_kv, bool least) {
  const Division d = divide(a, max_queries, max_kv, least ? 0 : UINT64_MAX);
  return d.parts == 1 && !a.prefix_tokens ? 0 : parts_bytes(a, d.parts);
}

cudaError_t launch_attend(const AttendArgs& a, const CacheView& c, uint32_t max_queries, uint32_t max_kv, void* ws,
                          size_t ws_bytes, cudaStream_t st) {
  const uint64_t rows = uint64_t(a.n_rows) * a.Hq;
  const uint64_t most = ws_bytes < 16 ? 0 : (ws_bytes - 16) / (rows * sizeof(float) * (a.D + 1));
  const Division d = divide(a, max_queries, max_kv, most);
  const uint64_t lse_bytes = (uint64_t(d.parts) * rows * sizeof(float) + 15) / 16 * 16;
  const PartsView parts{static_cast<float*>(ws), reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + lse_bytes), rows};
  return a.D == 64 ? run_all<64>(a, c, parts, d, st) : run_all<128>(a, c, parts, d, st);
}

}  // namespace kvc
