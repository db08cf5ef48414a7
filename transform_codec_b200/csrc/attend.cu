// Attention over the serving cache and a shared prefix (include/kvc.h,
// kvc_attend): launches, the division of work into parts, and their join.
#include "attend_cache.cuh"
#include "attend_parts.cuh"
#include "attend_prefix.cuh"

namespace kvc {
namespace {

// ---- how a call is divided

constexpr uint32_t kSMs = 148;
struct Division {
  uint32_t row_tiles;      // 8-row tiles a block takes: 1 or 2
  uint32_t row_groups;     // blocks along a sequence's query rows
  uint32_t splits;         // parts of a sequence's cache tokens at most
  uint32_t prefix_parts, prefix_blocks;  // parts of the prefix, 128-token blocks in each
  uint32_t parts;          // of a row at most
};

// A launch that may begin before this call's kernel ahead of it has ended (`behind`).
template <class... P, class... A>
cudaError_t launch_behind(void (*kern)(P...), dim3 grid, uint32_t threads, size_t smem, cudaStream_t st, bool behind,
                          A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = behind ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

// Join the parts of each row, D / 32 channels a lane; reads parts * (D + 1) * 4
// bytes a row. A warp takes a row, or kWarps warps its parts in turn where there
// are many: with 64 rows of 128 parts (one query, 131,072 tokens) one warp a row
// spent 59 us on loads one after another, eight spent 8 (and 4 on 74 parts).
constexpr uint32_t kJoinThreads = 256;
template <uint32_t D, uint32_t kWarps>
__global__ void __launch_bounds__(kJoinThreads)
k_attend_join(const AttendArgs a, const CacheView c, const PartsView parts, const uint32_t prefix_parts,
              const uint32_t splits) {
  constexpr uint32_t kPer = D / 32, kRows = kJoinThreads / 32 / kWarps;
  __shared__ float ssum[kRows][kWarps], sy[kWarps > 1 ? kRows * kWarps : 1][D];
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, part0 = warp % kWarps;
  const uint64_t id = uint64_t(blockIdx.x) * kRows + warp / kWarps;
  await_previous();
  int32_t i = 0;
  uint32_t hq = 0, n = 0;
  if (id < parts.rows) {
    i = int32_t(id / a.Hq);
    hq = uint32_t(id % a.Hq);
    const RowPlace at = place_of_row(a, i);
    if (at.seq >= 0) {
      n = prefix_parts;
      if (a.has_cache) {
        const uint32_t own = chunks_of(cache_len(a, c, at.seq), splits).parts;
        n = own == 1 && !prefix_parts ? 0u : n + own;  // one part alone has written the row itself
      }
    }
  }
  const float* lse = parts.lse + id;
  float top = -INFINITY;
  for (uint32_t p = lane; p < n; p += 32) top = fmaxf(top, lse[p * parts.rows]);
#pragma unroll
  for (uint32_t o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float sum = 0.f, y[kPer];
#pragma unroll
  for (uint32_t j = 0; j < kPer; ++j) y[j] = 0.f;
  // this warp's parts: part0, part0 + kWarps, ..; 32 half factors at a time, one a lane
  for (uint32_t p0 = part0; p0 < n; p0 += 32 * kWarps) {
    float f = 0.f;
    const uint32_t mine = p0 + lane * kWarps;
    if (mine < n) {
      const float L = lse[mine * parts.rows];
      f = L == -INFINITY ? 0.f : ex2(0.5f * (L - top));
    }
    const uint32_t here = min(32u, (n - p0 + kWarps - 1) / kWarps);
    for (uint32_t q = 0; q < here; q += 4) {
      float w[4], v[4][kPer];
#pragma unroll
      for (uint32_t u = 0; u < 4; ++u) {
        w[u] = __shfl_sync(0xffffffffu, f, (q + u) & 31u);
        if (q + u >= here) w[u] = 0.f;
        // a part that saw nothing need not have written an output
        const float* src = parts.o + ((p0 + (q + u) * kWarps) * parts.rows + id) * D + lane * kPer;
#pragma unroll
        for (uint32_t j = 0; j < kPer; ++j) v[u][j] = 0.f;
        if (w[u] != 0.f) {
          if constexpr (kPer == 4) {
            const float4 x = *reinterpret_cast<const float4*>(src);
            v[u][0] = x.x, v[u][1] = x.y, v[u][2] = x.z, v[u][3] = x.w;
          } else {
            const float2 x = *reinterpret_cast<const float2*>(src);
            v[u][0] = x.x, v[u][1] = x.y;
          }
        }
      }
#pragma unroll
      for (uint32_t u = 0; u < 4; ++u) {
        sum = fmaf(w[u], w[u], sum);
#pragma unroll
        for (uint32_t j = 0; j < kPer; ++j) y[j] = fmaf(w[u], w[u] * v[u][j], y[j]);
      }
    }
  }
  if (kWarps > 1) {
    if (lane == 0) ssum[warp / kWarps][part0] = sum;
#pragma unroll
    for (uint32_t j = 0; j < kPer; ++j) sy[warp][lane * kPer + j] = y[j];
    __syncthreads();
    if (part0) return;
    for (uint32_t w = 1; w < kWarps; ++w) {
      sum += ssum[warp / kWarps][w];
#pragma unroll
      for (uint32_t j = 0; j < kPer; ++j) y[j] += sy[warp + w][lane * kPer + j];
    }
  }
  if (!n) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (uint32_t j = 0; j < kPer; ++j) y[j] *= inv;
  store_out<kPer>(a, i, hq, lane * kPer, y);
  if (a.lse && lane == 0) a.lse[id] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

template <uint32_t D, uint32_t kWarps>
cudaError_t run_join(const AttendArgs& a, const CacheView& c, const PartsView& parts, const Division& d,
                     cudaStream_t st) {
  ProfRange p("attend_join", st);
  constexpr uint32_t kRows = kJoinThreads / 32 / kWarps;
  return launch_behind(k_attend_join<D, kWarps>, dim3(uint32_t((parts.rows + kRows - 1) / kRows)), kJoinThreads, 0, st,
                       true, a, c, parts, d.prefix_parts, d.splits);
}

uint64_t parts_bytes(const AttendArgs& a, uint64_t parts) {
  const uint64_t rows = uint64_t(a.n_rows) * a.Hq;
  return (parts * rows * sizeof(float) + 15) / 16 * 16 + parts * rows * a.D * sizeof(float);
}

// Parts of the cache's tokens where the longest sequence is not known: as many as a
// long one takes, within this many bytes of results (one query over 64 heads of 128
// takes 74 parts, 2.4 MB; rows that pass it fill the SMs by themselves).
constexpr uint64_t kUnknownBytes = 32u << 20;

// most: parts that the workspace has room for
Division divide(const AttendArgs& a, uint32_t max_queries, uint32_t max_kv, uint64_t most) {
  Division d{1, 1, 1, 0, 0, 1};
  if (a.prefix_tokens) {
    const uint64_t rows = uint64_t(a.n_rows) * a.G, room = most > uint64_t(a.has_cache) ? most - a.has_cache : 1;
    const uint32_t nb = a.prefix_tokens / 128 + (a.prefix_tokens % 128 != 0);
    const uint64_t units = (rows + 255) / 256 * a.H;
    // Time of n parts as measured: waves of blocks (one an SM), each 12 us and 0.71
    // a 128-token block for up to 128 rows, 19 us and 1.4 for two tiles of rows, and
    // n results a row written and joined at 1.9 KB a ns. (8192 tokens for 128 rows of
    // 8 heads: 1 part 66 us, 4 33, 8 29, 16 33, 32 45 with the call's other kernels;
    // 32,768 for 1024 rows: 1 part 406, 4 144, 9 168, 13 180.) The figures are those of
    // D = 128; at D = 64 what they choose is within 3% of the best as well (prefix alone,
    // 128 rows over 8192: 13 parts 19.1, the best of all 16 parts 18.6; 1024 over 32,768:
    // 4 parts 106 to 108, 8 114; 16 over 32,768: 18 parts 26.9, 12 31.0, 24 37.1).
    const double step = rows <= 128 ? 0.71 : 1.4, begin = rows <= 128 ? 12.0 : 19.0,
                 result = double(rows) * a.H * a.D * 8.0 / 1.9e6;
    double best = 0.0;
    for (uint32_t n = 1; n <= std::min<uint64_t>({nb, room, 256}); ++n) {
      const uint32_t per = (nb + n - 1) / n;
      if (n > 1 && (nb + per - 1) / per != n) continue;
      const double cost = double((units * n + kSMs - 1) / kSMs) * (begin + per * step) + n * result;
      if (n == 1 || cost < best) {
        best = cost;
        d.prefix_parts = n;
        d.prefix_blocks = per;
      }
    }
  }
  if (a.has_cache) {
    const uint64_t rows = uint64_t(std::max(max_queries, 1u)) * a.G;
    d.row_tiles = rows > 8 ? 2 : 1;
    d.row_groups = uint32_t(std::min<uint64_t>((rows + 8 * d.row_tiles - 1) / (8 * d.row_tiles), 4096u));
    // One sequence: as many parts as fill the SMs once (4 or 3 blocks each), of at
    // least 64 tokens. A batch: the same, or parts of about 512 tokens until there
    // are some four waves of blocks, so that different lengths even out.
    const bool known = max_kv != 0;
    if (!known) max_kv = 0x7fffffffu;
    const uint64_t wave = kSMs * (d.row_tiles == 1 ? 4 : 3), blocks = uint64_t(a.n_seqs) * a.H * d.row_groups;
    const uint64_t fine = std::max<uint64_t>(1, (uint64_t(max_kv) + kLeastTiles * kTile - 1) / (kLeastTiles * kTile));
    uint64_t s = std::min(fine, std::max<uint64_t>(1, wave / std::max<uint64_t>(blocks, 1)));
    if (a.n_seqs > 1) {
      const uint64_t coarse = std::max<uint64_t>(1, uint64_t(max_kv) / 512);
      s = std::max(s, std::min(coarse, std::max<uint64_t>(1, 4 * wave / std::max<uint64_t>(blocks, 1))));
    }
    if (!known) s = std::min(s, kUnknownBytes / (std::max<uint64_t>(a.n_rows, 1) * a.Hq * (a.D + 1) * sizeof(float)));
    s = std::max<uint64_t>(1, std::min<uint64_t>(s, 512));
    if (s + d.prefix_parts > 1 && s + d.prefix_parts > most) s = most > d.prefix_parts + 1 ? most - d.prefix_parts : 1;
    d.splits = uint32_t(s);
  }
  d.parts = d.prefix_parts + (a.has_cache ? d.splits : 0);
  return d;
}

// Blocks of 128 tokens x 64 channels of a [H][T][D] 16-bit slice array.
using EncodeMap = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                               const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeMap encode_map() {
  static const EncodeMap fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeMap>(p);
  }();
  return fn;
}
bool slice_map(CUtensorMap& m, const AttendArgs& a, const void* base) {
  const EncodeMap fn = encode_map();
  if (!fn) return false;
  const cuuint64_t dims[3] = {a.D, a.prefix_tokens, a.H};
  // one head needs no stride; the map wants a valid one all the same
  const cuuint64_t head = a.H > 1 ? cuuint64_t(a.p_head) * 2 : cuuint64_t(a.prefix_tokens) * a.D * 2;
  const cuuint64_t strides[2] = {cuuint64_t(a.D) * 2, head};
  const cuuint32_t box[3] = {64, 128, 1}, step[3] = {1, 1, 1};
  return fn(&m, a.dtype == KVC_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
            const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <uint32_t DT, uint32_t D>
cudaError_t run_prefix(const AttendArgs& a, const PartsView& parts, const Division& d, cudaStream_t st) {
  using T = PrefixTile<D>;
  static SmemAttr track;
  cudaError_t e = smem_attr(track, reinterpret_cast<const void*>(k_attend_prefix<DT, D>), T::kSmem);
  if (e != cudaSuccess) return e;
  CUtensorMap k, v;
  if (!slice_map(k, a, a.pk) || !slice_map(v, a, a.pv)) return cudaErrorInvalidValue;
  const uint64_t tiles = (uint64_t(a.n_rows) * a.G + 255) / 256;
  ProfRange p("attend_prefix", st);
  k_attend_prefix<DT, D><<<dim3(uint32_t(tiles * d.prefix_parts), a.H), T::kThreads, T::kSmem, st>>>(
      a, parts, k, v, d.prefix_parts, d.prefix_blocks, d.parts == 1);
  return cudaGetLastError();
}

template <uint32_t FMT, uint32_t D, uint32_t R>
cudaError_t run_cache(const AttendArgs& a, const CacheView& c, const PartsView& parts, const Division& d,
                      cudaStream_t st) {
  using T = CacheTile<FMT, D, R>;
  static SmemAttr track;
  cudaError_t e = smem_attr(track, reinterpret_cast<const void*>(k_attend_cache<FMT, D, R>), T::kSmem);
  if (e != cudaSuccess) return e;
  ProfRange p("attend_cache", st);
  return launch_behind(k_attend_cache<FMT, D, R>, dim3(d.row_groups * d.splits, a.H, a.n_seqs), T::kThreads, T::kSmem,
                       st, a.prefix_tokens != 0, a, c, parts, d.prefix_parts, d.splits, d.row_groups);
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
    e = a.dtype == KVC_DTYPE_BF16 ? run_prefix<KVC_DTYPE_BF16, D>(a, parts, d, st)
                                  : run_prefix<KVC_DTYPE_FP16, D>(a, parts, d, st);
    if (e != cudaSuccess) return e;
  }
  if (a.has_cache) {
    e = c.fmt == KVC_CACHE_E4M3   ? pick_cache<KVC_CACHE_E4M3, D>(a, c, parts, d, st)
        : c.fmt == KVC_CACHE_INT8 ? pick_cache<KVC_CACHE_INT8, D>(a, c, parts, d, st)
                                  : pick_cache<KVC_CACHE_E2M1, D>(a, c, parts, d, st);
    if (e != cudaSuccess) return e;
  }
  if (d.parts == 1) return e;
  return d.parts > 8 ? run_join<D, 8>(a, c, parts, d, st) : run_join<D, 1>(a, c, parts, d, st);
}

}  // namespace

uint64_t attend_ws_bytes(const AttendArgs& a, uint32_t max_queries, uint32_t max_kv, bool least) {
  const Division d = divide(a, max_queries, max_kv, least ? 0 : UINT64_MAX);
  return d.parts == 1 ? 0 : parts_bytes(a, d.parts);
}

cudaError_t launch_attend(const AttendArgs& a, const CacheView& c, uint32_t max_queries, uint32_t max_kv, void* ws,
                          size_t ws_bytes, cudaStream_t st) {
  const uint64_t rows = uint64_t(a.n_rows) * a.Hq;
  uint64_t most = ws_bytes / (rows * sizeof(float) * (a.D + 1));
  if (most && parts_bytes(a, most) > ws_bytes) --most;  // the results begin at a multiple of 16 bytes
  const Division d = divide(a, max_queries, max_kv, most);
  const uint64_t lse_bytes = (uint64_t(d.parts) * rows * sizeof(float) + 15) / 16 * 16;
  const PartsView parts{static_cast<float*>(ws), reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + lse_bytes), rows};
  return a.D == 64 ? run_all<64>(a, c, parts, d, st) : run_all<128>(a, c, parts, d, st);
}

}  // namespace kvc
