// Serving cache: quantising writes and reads (include/kvc.h, "Serving cache").
//
// Both move each value once: a bf16 row of 128 channels is 256 bytes on one side
// and 132 (8-bit) or 76 (4-bit, micro-scales included) on the other. Reading is
// bound by memory (eight sequences of e4m3 to bf16, 281 MB, 45 us: 6.2 TB/s of 6.56
// measured). Writing is bound by instructions: 30,247 tokens of 2 x 8 x 128 take 43
// to 46 us in 4 bits (165 MB, 25 us at 6.56; 140 warp instructions for each two rows,
// two reciprocals and the conversions above all; 78% of issue slots at 1.88 GHz), 40
// in e4m3 and 45 in int8 (188 MB, 29 us; e4m3 106 instructions, 73%). A row (token,
// key/value, head) belongs to a group of lanes, 8 values a lane, so a row is read and
// written in whole 32-byte sectors, its magnitude is a few shuffles, and every
// thread has several rows' loads in flight. Consecutive blocks take the 2 * H heads of the same tokens:
// they touch neighbouring memory on the token-major side at the same time.
#include "cache_codes.cuh"
#include "serving.h"

namespace kvc {
namespace {

constexpr uint32_t kThreads = 256;

// 8 values at p as fp32 (VT: value type)
template <uint32_t DT>
struct Vals {
  uint4 w[DT == KVC_DTYPE_F32 ? 2 : 1];
  __device__ void load(const void* base, int64_t at) {
    if (DT == KVC_DTYPE_F32) {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + at);
      w[0] = __ldg(p);
      w[DT == KVC_DTYPE_F32 ? 1 : 0] = __ldg(p + 1);
    } else {
      w[0] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at));
    }
  }
  __device__ void zero() {
    for (auto& x : w) x = make_uint4(0, 0, 0, 0);
  }
  __device__ void get(float* x) const {
    if (DT == KVC_DTYPE_F32) {
      const uint4 a = w[0], b = w[DT == KVC_DTYPE_F32 ? 1 : 0];
      const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u[i]);
    } else {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack16<DT == KVC_DTYPE_F32 ? KVC_DTYPE_BF16 : DT>(u[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
};

// Largest magnitudes as bits (an infinity or NaN sorts above every number): of a
// lane's 8 values, as a pattern of the value type. Two rows of 16-bit values go
// through the exchange between lanes in one word.
template <uint32_t DT>
__device__ inline uint32_t lane_max(const Vals<DT>& v) {
  uint32_t m = 0;
#pragma unroll
  for (const uint4& q : v.w) {
    constexpr uint32_t kMask = DT == KVC_DTYPE_F32 ? 0x7fffffffu : 0x7fff7fffu;
    const uint32_t u[4] = {q.x & kMask, q.y & kMask, q.z & kMask, q.w & kMask};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = DT == KVC_DTYPE_F32 ? max(m, u[i]) : __vmaxu2(m, u[i]);
  }
  return DT == KVC_DTYPE_F32 ? m : max(m & 0xffffu, m >> 16);
}
template <uint32_t DT>
__device__ inline uint32_t max_bits(uint32_t a, uint32_t b) {
  return DT == KVC_DTYPE_F32 ? max(a, b) : __vmaxu2(a, b);
}
template <uint32_t DT>
__device__ inline float bits_f32(uint32_t m) {
  if (DT == KVC_DTYPE_F32) return __uint_as_float(m);
  if (DT == KVC_DTYPE_BF16) return __uint_as_float(m << 16);
  return half2_f32(m & 0xffffu).x;
}

// Quantise one lane's 8 values x of a row and store them at row `row`; m and mb:
// the row's and the block's largest magnitude (bits of the value type).
template <uint32_t DT, uint32_t FMT>
__device__ inline void quantise_store(const CacheView& c, uint64_t row, uint32_t lane, const float* x, uint32_t m,
                                      uint32_t mb) {
  constexpr float kPeak = FMT == KVC_CACHE_E4M3 ? kE4m3Peak : FMT == KVC_CACHE_INT8 ? kInt8Peak : kE2m1Peak;
  const float top = bits_f32<DT>(m);
  const bool bad = !(top < INFINITY);
  float s = 0.f, inv = 0.f;
  if (!bad && top >= kRowFloor) {
    s = top * (1.0f / kPeak);
    inv = 1.0f / s;
  }
  if (lane == 0) c.scales[row] = bad ? __uint_as_float(0x7fc00000u) : s;
  if (lane * 8u >= c.D) return;
  uint8_t* dst = c.codes + row * c.row_bytes;
  if (FMT == KVC_CACHE_E2M1) {
    const uint32_t u = e4m3x2((bits_f32<DT>(mb) * inv) * (1.0f / 6.0f), 0.f) & 0xffu;
    const float uf = e4m3_f32(u);
    const float inv_b = uf > 0.f ? 1.0f / (s * uf) : 0.f;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] * inv_b;
    const uint32_t w = e2m1x8(y);
    *reinterpret_cast<uint32_t*>(dst + lane * 4u) = bad ? 0u : w;
    if (!(lane & 1u)) c.micro[row * (c.D / 16u) + (lane >> 1)] = bad ? uint8_t(0) : uint8_t(u);
  } else {
    uint32_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = x[4 * j + i] * inv;
      if (FMT == KVC_CACHE_E4M3)
        w[j] = e4m3x2(y[0], y[1]) | (e4m3x2(y[2], y[3]) << 16);
      else
        w[j] = __byte_perm(__byte_perm(int8_bits(y[0]), int8_bits(y[1]), 0x0040),
                           __byte_perm(int8_bits(y[2]), int8_bits(y[3]), 0x0040), 0x5410);
      if (bad) w[j] = 0;
    }
    *reinterpret_cast<uint2*>(dst + lane * 8u) = make_uint2(w[0], w[1]);
  }
}

// grid (2 H, token tiles); a block takes U * 256 / L tokens of one head
template <uint32_t DT, uint32_t FMT, uint32_t L, uint32_t U>
__global__ void __launch_bounds__(kThreads) k_cache_write(const CacheView c, const WriteArgs a, const uint32_t t0) {
  constexpr uint32_t kGroups = kThreads / L;
  __shared__ int64_t rows[U * kGroups];  // the tokens' cache rows, -1: none
  const uint32_t lane = threadIdx.x % L, group = threadIdx.x / L;
  const uint32_t kv = blockIdx.x >= c.H, h = blockIdx.x - kv * c.H;
  const uint32_t tile = t0 + blockIdx.y * U * kGroups;
  const void* src = kv ? a.v : a.k;
  const int64_t ts = kv ? a.v_tok : a.k_tok, hs = kv ? a.v_head : a.k_head;
  Vals<DT> v[U];
#pragma unroll
  for (uint32_t u = 0; u < U; ++u) {
    const uint32_t t = tile + u * kGroups + group;
    v[u].zero();
    if (t < a.n_tokens && lane * 8u < c.D) v[u].load(src, int64_t(t) * ts + int64_t(h) * hs + lane * 8u);
  }
  for (uint32_t i = threadIdx.x; i < U * kGroups; i += kThreads) {
    const int64_t slot = a.n_tokens - tile > i ? __ldg(a.slots + tile + i) : -1;
    const uint64_t page = uint64_t(slot) >> c.page_shift;
    int64_t row = -1;
    if (slot >= 0) {
      if (page >= c.n_pages)
        flag_invalid(a.res);
      else
        row = int64_t(cache_row(c, uint32_t(page), kv, h) + (uint64_t(slot) & c.page_mask));
    }
    rows[i] = row;
  }
  __syncthreads();
  // magnitudes: kPair rows to a word
  constexpr uint32_t kPair = DT == KVC_DTYPE_F32 || U == 1 ? 1 : 2;
  uint32_t m[U], mb[U];
#pragma unroll
  for (uint32_t u = 0; u < U; u += kPair) {
    uint32_t w = lane_max<DT>(v[u]);
    if (kPair == 2) w |= lane_max<DT>(v[u + kPair - 1]) << 16;
    if (FMT == KVC_CACHE_E2M1) w = max_bits<DT>(w, __shfl_xor_sync(0xffffffffu, w, 1));  // a block of 16 channels
    const uint32_t wb = w;
#pragma unroll
    for (uint32_t o = FMT == KVC_CACHE_E2M1 ? 2 : 1; o < L; o <<= 1)
      w = max_bits<DT>(w, __shfl_xor_sync(0xffffffffu, w, o));
    m[u] = kPair == 2 ? w & 0xffffu : w;
    mb[u] = kPair == 2 ? wb & 0xffffu : wb;
    if (kPair == 2) {
      m[u + kPair - 1] = w >> 16;
      mb[u + kPair - 1] = wb >> 16;
    }
  }
#pragma unroll
  for (uint32_t u = 0; u < U; ++u) {
    const int64_t row = rows[u * kGroups + group];
    if (row < 0) continue;
    float x[8];
    v[u].get(x);
    quantise_store<DT, FMT>(c, uint64_t(row), lane, x, m[u], mb[u]);
  }
}

// Where output token t comes from: its cache row for head 0 of the keys, or -1.
__device__ inline int64_t read_row(const CacheView& c, const ReadArgs& a, uint32_t t) {
  uint32_t lo = 0, hi = a.n_seqs - 1;  // the last sequence that starts at or before t
  while (lo < hi) {
    const uint32_t mid = (lo + hi + 1) >> 1;
    if (__ldg(a.out_start + mid) <= int32_t(t)) lo = mid; else hi = mid - 1;
  }
  const int32_t first = __ldg(a.out_start + lo);
  if (int32_t(t) < first || int32_t(t) >= __ldg(a.out_start + lo + 1) || first < 0) return -1;
  const int64_t p = int64_t(__ldg(a.start + lo)) + (int32_t(t) - first);
  const int64_t page_at = p >> c.page_shift;
  if (p < 0 || page_at >= int64_t(a.pages_stride)) {
    flag_invalid(a.res);
    return -1;
  }
  const int32_t page = __ldg(a.pages + uint64_t(lo) * a.pages_stride + page_at);
  if (page < 0 || uint32_t(page) >= c.n_pages) {
    flag_invalid(a.res);
    return -1;
  }
  return int64_t(cache_row(c, uint32_t(page), 0, 0) + (uint64_t(p) & c.page_mask));
}

// Codes of 8 channels as they lie in memory.
template <uint32_t FMT>
struct Codes {
  uint32_t w[2], micro;
  float s;
  __device__ void load(const CacheView& c, uint64_t row, uint32_t lane) {
    const uint8_t* p = c.codes + row * c.row_bytes;
    s = __ldg(c.scales + row);
    if (FMT == KVC_CACHE_E2M1) {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(p + lane * 4u));
      micro = __ldg(c.micro + row * (c.D / 16u) + (lane >> 1));
    } else {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(p + lane * 8u));
      w[0] = q.x;
      w[1] = q.y;
    }
  }
  __device__ void get(float* x) const {
    if (FMT == KVC_CACHE_E2M1) {
      const float u = e4m3_f32(micro);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = half2_f32(e2m1x2_half2((w[0] >> (8 * i)) & 0xffu));
        x[2 * i] = s * (f.x * u);  // f * u is exact
        x[2 * i + 1] = s * (f.y * u);
      }
    } else if (FMT == KVC_CACHE_E4M3) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = half2_f32(e4m3x2_half2((w[i >> 1] >> (16 * (i & 1))) & 0xffffu));
        x[2 * i] = s * f.x;
        x[2 * i + 1] = s * f.y;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        x[4 * j] = s * int8_f32<0>(w[j]);
        x[4 * j + 1] = s * int8_f32<1>(w[j]);
        x[4 * j + 2] = s * int8_f32<2>(w[j]);
        x[4 * j + 3] = s * int8_f32<3>(w[j]);
      }
    }
  }
};

template <uint32_t DT>
__device__ inline void store8(void* base, uint64_t at, const float* x) {
  if (DT == KVC_DTYPE_F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    constexpr uint32_t T = DT == KVC_DTYPE_F32 ? KVC_DTYPE_BF16 : DT;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) =
        make_uint4(pack16<T>(x[0], x[1]), pack16<T>(x[2], x[3]), pack16<T>(x[4], x[5]), pack16<T>(x[6], x[7]));
  }
}

// grid (2 H, token tiles); the block looks its tokens' rows up once
template <uint32_t DT, uint32_t FMT, uint32_t L, uint32_t U>
__global__ void __launch_bounds__(kThreads) k_cache_read(const CacheView c, const ReadArgs a, const uint32_t t0) {
  constexpr uint32_t kGroups = kThreads / L;
  __shared__ int64_t rows[U * kGroups];
  const uint32_t lane = threadIdx.x % L, group = threadIdx.x / L;
  const uint32_t tile = t0 + blockIdx.y * U * kGroups;
  // each range is looked at once, whether or not a token of out lies in it
  const uint64_t id = (uint64_t(blockIdx.y) * gridDim.x + blockIdx.x) * kThreads + threadIdx.x;
  for (uint64_t b = id; b < a.n_seqs; b += uint64_t(gridDim.x) * gridDim.y * kThreads) {
    const int32_t first = __ldg(a.out_start + b), last = __ldg(a.out_start + b + 1);
    if (first < 0 || last < first || last > int32_t(a.out_tokens)) flag_invalid(a.res);
  }
  for (uint32_t i = threadIdx.x; i < U * kGroups; i += kThreads)
    rows[i] = a.out_tokens - tile > i ? read_row(c, a, tile + i) : -1;
  __syncthreads();
  const uint64_t head = uint64_t(blockIdx.x) << c.page_shift;  // rows of earlier (kv, head) in a page
  Codes<FMT> q[U];
  int64_t row[U];
#pragma unroll
  for (uint32_t u = 0; u < U; ++u) {
    row[u] = rows[u * kGroups + group];
    if (row[u] >= 0 && lane * 8u < c.D) q[u].load(c, uint64_t(row[u]) + head, lane);
  }
#pragma unroll
  for (uint32_t u = 0; u < U; ++u) {
    if (row[u] < 0 || lane * 8u >= c.D) continue;
    float x[8];
    q[u].get(x);
    const uint64_t t = tile + u * kGroups + group;
    store8<DT>(a.out, (uint64_t(blockIdx.x) * a.out_tokens + t) * c.D + lane * 8u, x);
  }
}

// Rows in flight a thread: 4, or 1 while 4 would leave SMs without a block.
constexpr uint64_t kFewBlocks = 148 * 4;

template <uint32_t DT, uint32_t FMT, uint32_t L, uint32_t U>
cudaError_t run_write(const CacheView& c, const WriteArgs& a, cudaStream_t st) {
  constexpr uint32_t kTile = U * (kThreads / L);
  for (uint64_t t0 = 0; t0 < a.n_tokens; t0 += 65535ull * kTile) {
    const uint32_t tiles = uint32_t(std::min<uint64_t>((a.n_tokens - t0 + kTile - 1) / kTile, 65535u));
    ProfRange p("cache_write", st);
    k_cache_write<DT, FMT, L, U><<<dim3(2 * c.H, tiles), kThreads, 0, st>>>(c, a, uint32_t(t0));
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}
template <uint32_t DT, uint32_t FMT, uint32_t L, uint32_t U>
cudaError_t run_read(const CacheView& c, const ReadArgs& a, cudaStream_t st) {
  constexpr uint32_t kTile = U * (kThreads / L);
  for (uint64_t t0 = 0; t0 < a.out_tokens; t0 += 65535ull * kTile) {
    const uint32_t tiles = uint32_t(std::min<uint64_t>((a.out_tokens - t0 + kTile - 1) / kTile, 65535u));
    ProfRange p("cache_read", st);
    k_cache_read<DT, FMT, L, U><<<dim3(2 * c.H, tiles), kThreads, 0, st>>>(c, a, uint32_t(t0));
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <bool kWrite, uint32_t DT, uint32_t FMT, uint32_t L, class A>
cudaError_t pick_u(const CacheView& c, const A& a, uint64_t tokens, cudaStream_t st) {
  const bool few = tokens * 2 * c.H < kFewBlocks * 4 * (kThreads / L);
  if constexpr (kWrite)
    return few ? run_write<DT, FMT, L, 1>(c, a, st) : run_write<DT, FMT, L, 4>(c, a, st);
  else
    return few ? run_read<DT, FMT, L, 1>(c, a, st) : run_read<DT, FMT, L, 4>(c, a, st);
}
// lanes of a row: the power of two from D / 8 up
template <bool kWrite, uint32_t DT, uint32_t FMT, class A>
cudaError_t pick_l(const CacheView& c, const A& a, uint64_t tokens, cudaStream_t st) {
  if (c.D <= 32) return pick_u<kWrite, DT, FMT, 4>(c, a, tokens, st);
  if (c.D <= 64) return pick_u<kWrite, DT, FMT, 8>(c, a, tokens, st);
  if (c.D <= 128) return pick_u<kWrite, DT, FMT, 16>(c, a, tokens, st);
  return pick_u<kWrite, DT, FMT, 32>(c, a, tokens, st);
}
template <bool kWrite, uint32_t DT, class A>
cudaError_t pick_fmt(const CacheView& c, const A& a, uint64_t tokens, cudaStream_t st) {
  if (c.fmt == KVC_CACHE_E4M3) return pick_l<kWrite, DT, KVC_CACHE_E4M3>(c, a, tokens, st);
  if (c.fmt == KVC_CACHE_INT8) return pick_l<kWrite, DT, KVC_CACHE_INT8>(c, a, tokens, st);
  return pick_l<kWrite, DT, KVC_CACHE_E2M1>(c, a, tokens, st);
}
template <bool kWrite, class A>
cudaError_t pick(const CacheView& c, const A& a, uint64_t tokens, cudaStream_t st) {
  if (a.dtype == KVC_DTYPE_BF16) return pick_fmt<kWrite, KVC_DTYPE_BF16>(c, a, tokens, st);
  if (a.dtype == KVC_DTYPE_FP16) return pick_fmt<kWrite, KVC_DTYPE_FP16>(c, a, tokens, st);
  return pick_fmt<kWrite, KVC_DTYPE_F32>(c, a, tokens, st);
}

}  // namespace

cudaError_t launch_cache_write(const CacheView& c, const WriteArgs& a, cudaStream_t st) {
  return pick<true>(c, a, a.n_tokens, st);
}
cudaError_t launch_cache_read(const CacheView& c, const ReadArgs& a, cudaStream_t st) {
  return pick<false>(c, a, a.out_tokens, st);
}

}  // namespace kvc
