// Attention of a sequence's newest queries over its quantised cache, as one
// kernel over (sequence, head, part of the tokens). GPU-library only.
//
// What bounds it is reading the codes: 2 * (D + 4) bytes a token and head
// against 4 D multiply-adds a query row, so products run on mma.sync tiles of
// 16 tokens x 8 rows (m16n8k16, fp16 in, fp32 sums): tokens are the wide side
// of both products, and a group of 8 query heads fills the narrow one without
// padding. Codes are exact in fp16 whatever their format, so
//     S[token][row] = s_k (c_k . q'),  q' = q 2^e (e: the row's largest element to [2^7, 2^8)),
// is exact up to fp32 sums. For the second product the value scale goes into the weight,
//     w = 2^(S + log2 s_v - m),   o = sum w c_v,
// with m a running reference, 7 below the largest S + log2 s_v when it was set:
// the largest weight is 2^7 or more, so that fp16 leaves weights 2^-32 of it
// their place, and attention on rows of tiny values keeps its bits. The sum of
// exponentials has a reference of its own,
//     l = sum 2^(S - n),   answer = o 2^(m - n) / l,
// so that a token's share of it does not depend on how large its values are: a
// row of zeros beside rows of 2^100 counts like any other. (Summing w / s_v saves
// that exponential, 3 to 5% of the time, and loses tokens whose scale is 2^-126 of
// the largest.) m and n move only when passed by 15 (weights up to 2^15 are as
// exact), so the usual tile needs no exchange between lanes but one vote.
//
// Layout: the order of channels within the first product and of tokens within
// the second is free, and is chosen such that a thread's own fragments are
// contiguous bytes of rows: thread (g, t) = (lane / 4, lane % 4) holds token g
// and g + 8's bytes of channel group t for S = K q', and channel group g of
// tokens 2t, 2t + 1, 2t + 8, 2t + 9 for o = V^T w. A warp copies its tiles in
// whole lines, asynchronously and several tiles ahead, into a ring in shared
// memory where each thread's bytes are together; it needs no block-wide barrier.
// Each warp takes tiles of the block's part with a softmax of its own; the four are
// joined at the end.
//
// Measured: 131,072 tokens of 8 heads x 128 in int8 for one query, 277 MB, 72 us for
// the call (42 us at the measured 6.56 TB/s); the kernel issues 452 instructions a
// tile and warp, half of its slots. 64 sequences of up to 8192 tokens on 4-bit pages,
// 321 MB, 106 us (49): 464 a tile, 68% of the slots of SMs that run, and SMs stand
// still for 17% of the launch, since sequences of different lengths are cut into the
// same number of parts. With more than 16 query rows a sequence each 16 take the
// codes again: 32 sequences of 32,768 tokens, up to 4 queries of 8 heads, 731 us (332).
#pragma once
#include <type_traits>

#include "attend_parts.cuh"

namespace kvc {
namespace {

template <int BYTES>
__device__ inline void copy_async(uint32_t dst, const void* src, bool in) {
  const int n = in ? BYTES : 0;  // the rest is filled with zeros
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}
__device__ inline void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ inline void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ inline void mma16816(float* d, const uint32_t* a, const uint32_t* b) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ inline uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ inline float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ inline float lg2(float x) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ inline uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ inline uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// four 8-bit codes to two half pairs
template <uint32_t FMT>
__device__ inline void codes4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (FMT == KVC_CACHE_E4M3) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {  // 1024 + (c + 128) as fp16 bits, less 1152
    const uint32_t x = w ^ 0x80808080u;
    lo = hsub2(__byte_perm(x, 0x64646464u, 0x4140u), 0x64806480u);
    hi = hsub2(__byte_perm(x, 0x64646464u, 0x4342u), 0x64806480u);
  }
}
// eight 4-bit codes, a byte at a time, to four half pairs
__device__ inline void codes8(uint32_t w, uint32_t* h) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

template <uint32_t FMT, uint32_t D, uint32_t R>
struct CacheTile {
  static constexpr uint32_t kWarps = 4, kThreads = 128, kRows = 8 * R;
  static constexpr bool k4 = FMT == KVC_CACHE_E2M1;
  static constexpr uint32_t kRow = k4 ? D / 2 : D;         // code bytes of a row
  static constexpr uint32_t kSteps = D / 16;               // k16 steps of S, m16 tiles of o
  static constexpr uint32_t kKBytes = kRow / 4;            // a thread's bytes of one key row
  static constexpr uint32_t kKCopy = kKBytes > 16 ? 16 : kKBytes;
  static constexpr uint32_t kKChunks = kKBytes / kKCopy;
  static constexpr uint32_t kVBytes = kRow / 8;            // a thread's bytes of one value row
  static constexpr uint32_t kKArea = 2 * kKBytes * 32, kVArea = 4 * kVBytes * 32;
  static constexpr uint32_t kScales = kKArea + kVArea;     // fp32 [k 16][v 16]
  static constexpr uint32_t kMicro = kScales + 128;        // e4m3 [k 16][D / 16], [v 16][D / 16]
  static constexpr uint32_t kStage = kMicro + (k4 ? 32 * (D / 16) : 0);
  // A tile's keys, and its values, lie together in memory: 512 bytes of them a copy
  // of the warp, whole lines. Lane l's 16 bytes of copy j belong to this token, and
  // to the slots of the thread that will use them.
  static constexpr uint32_t kRowChunks = kRow / 16, kCopies = kRow / 32;
  __device__ static constexpr uint32_t token(uint32_t j, uint32_t l) { return j * (32 / kRowChunks) + l / kRowChunks; }
  __device__ static constexpr uint32_t key_slot(uint32_t j, uint32_t l) {
    const uint32_t r = token(j, l), b = l % kRowChunks * 16;  // byte of the row
    const uint32_t x = b / (4 * kKCopy), t = b / kKCopy % 4;
    return (((r >> 3) * kKChunks + x) * 32 + (r & 7u) * 4 + t) * kKCopy + b % kKCopy;
  }
  // slots of 16 bytes by (g, t), smaller ones by (t, g): groups side by side
  __device__ static constexpr uint32_t value_place(uint32_t g, uint32_t t) {
    return kVBytes == 16 ? g * 4 + t : t * 8 + g;
  }
  __device__ static constexpr uint32_t value_slot(uint32_t j, uint32_t l) {
    const uint32_t r = token(j, l), b = l % kRowChunks * 16;
    const uint32_t i = (r & 1u) + 2 * (r >> 3), t = (r & 7u) >> 1;
    return (i * 32 + value_place(b / kVBytes, t)) * kVBytes;
  }
  // blocks an SM that registers allow; together they keep up to 200 KB on the way
  static constexpr uint32_t kBlocks = R == 1 ? 4 : 3;
  static constexpr uint32_t kFit = 204800 / kBlocks / kWarps / kStage;
  static constexpr uint32_t kStages = kFit > 8 ? 8 : kFit;
  static constexpr uint32_t kRing = kWarps * kStages * kStage;
  static constexpr uint32_t kJoin = kWarps * kRows * (D + 1) * 4;  // the end's o and L of each warp
  static constexpr uint32_t kSmem = kRing > kJoin ? kRing : kJoin;
};

// grid (row groups * splits, H, sequences)
template <uint32_t FMT, uint32_t D, uint32_t R>
__global__ void __launch_bounds__(128, (CacheTile<FMT, D, R>::kBlocks))
k_attend_cache(const AttendArgs a, const CacheView c, const PartsView parts, const uint32_t part0,
               const uint32_t splits, const uint32_t row_groups) {
  using T = CacheTile<FMT, D, R>;
  extern __shared__ __align__(16) uint8_t smem[];
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3u;
  const uint32_t part = blockIdx.x / row_groups, h = blockIdx.y, b = blockIdx.z;
  let_next_begin();
  const SeqRows rows = rows_of_seq(a, b);
  const uint32_t len = cache_len(a, c, b);
  const Chunks ch = chunks_of(len, splits);
  if (part >= ch.parts) return;
  const bool direct = ch.parts == 1 && !a.prefix_tokens;
  // This warp's tiles are `first`, first + stride, ..: the blocks of a sequence walk
  // through it side by side, so that what is read at a time lies together.
  const uint32_t n_tiles = (len + kTile - 1) / kTile, first = part * T::kWarps + warp, stride = ch.parts * T::kWarps;
  const uint32_t mine = first < n_tiles ? (n_tiles - 1 - first) / stride + 1 : 0u;
  const int32_t* pages = a.pages + uint64_t(b) * a.pages_stride;
  const uint64_t v_rows = uint64_t(c.H) << c.page_shift;  // from a key row to its value row
  const uint32_t ring = uint32_t(__cvta_generic_to_shared(smem)) + warp * (T::kStages * T::kStage);
  // what this lane copies of a tile at row 0: 16 bytes of each 512, and a scale and
  // micro-scales (lanes 0 - 15 keys, 16 - 31 values)
  const uint8_t* codes = c.codes + lane * 16;
  const float* scales = c.scales + (lane & 15u) + (lane >= 16 ? v_rows : 0u);
  const uint8_t* micro = T::k4 ? c.micro + ((lane & 15u) + (lane >= 16 ? v_rows : 0u)) * (D / 16) : nullptr;
  const uint32_t total_rows = uint32_t(rows.n) * a.G;

  for (uint32_t group = blockIdx.x % row_groups; group * T::kRows < total_rows; group += row_groups) {
    // ---- copies: this warp's k-th tile into the ring's next stage
    int64_t row_of = -1;  // lane j: key row of tile (k & ~31) + j, -1: nothing to read there
    uint32_t to_stage = 0;
    auto copy = [&](int64_t row, uint32_t n, auto whole) {
      constexpr bool kWhole = decltype(whole)::value;
      const uint32_t dst = ring + to_stage * T::kStage;
      const uint8_t* kp = codes + row * T::kRow;
      const uint8_t* vp = kp + v_rows * T::kRow;
#pragma unroll
      for (uint32_t j = 0; j < T::kCopies; ++j)
        copy_async<16>(dst + T::key_slot(j, lane), kp + j * 512, kWhole || T::token(j, lane) < n);
#pragma unroll
      for (uint32_t j = 0; j < T::kCopies; ++j)
        copy_async<16>(dst + T::kKArea + T::value_slot(j, lane), vp + j * 512, kWhole || T::token(j, lane) < n);
      copy_async<4>(dst + T::kScales + lane * 4, scales + row, kWhole || (lane & 15u) < n);
      if constexpr (T::k4)
        copy_async<D / 16>(dst + T::kMicro + lane * (D / 16), micro + row * (D / 16), kWhole || (lane & 15u) < n);
    };
    auto issue = [&](uint32_t k) {
      if (k < mine) {
        if ((k & 31u) == 0) {
          const uint32_t kk = k + lane, at = (first + kk * stride) * kTile;
          row_of = -1;
          if (kk < mine) {
            const int32_t page = __ldg(pages + (at >> c.page_shift));
            if (page < 0 || uint32_t(page) >= c.n_pages)
              flag_invalid(a.res);
            else
              row_of = int64_t(cache_row(c, uint32_t(page), 0, h) + (at & c.page_mask));
          }
        }
        const int64_t row = __shfl_sync(0xffffffffu, row_of, k & 31u);
        const uint32_t at = (first + k * stride) * kTile;
        if (row >= 0 && at + kTile <= len)
          copy(row, kTile, std::true_type{});
        else  // tokens that are there, and zeros
          copy(max(row, int64_t(0)), row < 0 ? 0u : len - at, std::false_type{});
        if (++to_stage == T::kStages) to_stage = 0;
      }
      copy_commit();
    };
#pragma unroll
    for (uint32_t k = 0; k < T::kStages - 1; ++k) issue(k);

    // ---- queries: row g of each 8 as the second operand of S, scaled to fp16
    uint32_t q[R][T::kSteps][2];
    float rs[R][2];    // scale of rows 2t, 2t + 1 (this thread's columns of S), base 2
    int32_t lim[R][2]; // tokens that they see
#pragma unroll
    for (uint32_t r = 0; r < R; ++r) {
      const uint32_t row = group * T::kRows + r * 8 + g;
      const bool in = row < total_rows;
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + (rows.first + int64_t(row / a.G)) * a.q_tok +
                            int64_t(h * a.G + row % a.G) * a.q_head;
      float x[T::kSteps][4], top = 0.f;
      bool odd = false;
#pragma unroll
      for (uint32_t s = 0; s < T::kSteps; ++s) {
        // the channels of a thread's bytes 4 s .. 4 s + 3 (two bytes of 4-bit codes) of a key row
        const uint32_t chn = T::k4 ? t * (D / 4) + 4 * s : (s / 4) * 64 + t * 16 + (s % 4) * 4;
        uint2 w = make_uint2(0, 0);
        if (in) w = *reinterpret_cast<const uint2*>(src + chn);
        const float2 p0 = a.dtype == KVC_DTYPE_BF16 ? unpack16<KVC_DTYPE_BF16>(w.x) : unpack16<KVC_DTYPE_FP16>(w.x);
        const float2 p1 = a.dtype == KVC_DTYPE_BF16 ? unpack16<KVC_DTYPE_BF16>(w.y) : unpack16<KVC_DTYPE_FP16>(w.y);
        x[s][0] = p0.x, x[s][1] = p0.y, x[s][2] = p1.x, x[s][3] = p1.y;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          top = fmaxf(top, fabsf(x[s][j]));
          odd |= !(fabsf(x[s][j]) < INFINITY);
        }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^e takes the largest element to [2^7, 2^8); e is kept where 2^-e is normal
      int e = 7 - (int(__float_as_uint(top) >> 23) - 127);
      e = top > 0.f ? max(-120, min(120, e)) : 0;
      float up = __uint_as_float(uint32_t(127 + e) << 23);
      if (odd) up = __uint_as_float(0x7fc00000u);  // a NaN or an infinity: the row's answer is NaN
#pragma unroll
      for (uint32_t s = 0; s < T::kSteps; ++s) {
        q[r][s][0] = pack_half(x[s][0] * up, x[s][1] * up);
        q[r][s][1] = pack_half(x[s][2] * up, x[s][3] * up);
      }
      const float down = __uint_as_float(uint32_t(127 - e) << 23) * a.scale_log2;
#pragma unroll
      for (uint32_t j = 0; j < 2; ++j) {
        // lane 4 (2t + j) holds row 2t + j
        rs[r][j] = __shfl_sync(0xffffffffu, down, (2 * t + j) * 4);
        const uint32_t rj = group * T::kRows + r * 8 + 2 * t + j;
        lim[r][j] = rj < total_rows ? int32_t(len) - rows.n + int32_t(rj / a.G) + 1 : 0x7fffffff;
      }
    }
    // the first token that some row of the group does not see
    int32_t all_see = lim[0][0];
#pragma unroll
    for (uint32_t r = 0; r < R; ++r)
#pragma unroll
      for (uint32_t j = 0; j < 2; ++j) all_see = min(all_see, lim[r][j]);
    all_see = min(all_see, __shfl_xor_sync(0xffffffffu, all_see, 1));
    all_see = min(all_see, __shfl_xor_sync(0xffffffffu, all_see, 2));
    all_see = min(all_see, int32_t(len));

    float m[R][2], n[R][2], l[R][2], o[R][T::kSteps][4];
#pragma unroll
    for (uint32_t r = 0; r < R; ++r) {
      m[r][0] = m[r][1] = n[r][0] = n[r][1] = -INFINITY;
      l[r][0] = l[r][1] = 0.f;
#pragma unroll
      for (uint32_t j = 0; j < T::kSteps; ++j) o[r][j][0] = o[r][j][1] = o[r][j][2] = o[r][j][3] = 0.f;
    }

    uint32_t at_stage = 0;
    for (uint32_t k = 0; k < mine; ++k) {
      copy_wait<T::kStages - 2>();
      __syncwarp();  // the tile's scales were copied by other lanes
      issue(k + T::kStages - 1);
      const uint8_t* st = smem + warp * (T::kStages * T::kStage) + at_stage * T::kStage;
      if (++at_stage == T::kStages) at_stage = 0;
      const float* sc = reinterpret_cast<const float*>(st + T::kScales);
      // ---- S
      float s2[2][R][4];  // two chains of sums
#pragma unroll
      for (uint32_t r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) s2[0][r][j] = s2[1][r][j] = 0.f;
      uint32_t kw[2][T::kKBytes / 4];
#pragma unroll
      for (uint32_t u = 0; u < 2; ++u)
#pragma unroll
        for (uint32_t x = 0; x < T::kKChunks; ++x) {
          const uint8_t* p = st + ((u * T::kKChunks + x) * 32 + lane) * T::kKCopy;
          if constexpr (T::kKCopy == 16) {
            const uint4 w = *reinterpret_cast<const uint4*>(p);
            kw[u][4 * x] = w.x, kw[u][4 * x + 1] = w.y, kw[u][4 * x + 2] = w.z, kw[u][4 * x + 3] = w.w;
          } else {
            const uint2 w = *reinterpret_cast<const uint2*>(p);
            kw[u][0] = w.x, kw[u][1] = w.y;
          }
        }
      if constexpr (!T::k4) {
#pragma unroll
        for (uint32_t s = 0; s < T::kSteps; ++s) {
          uint32_t f[4];
          codes4<FMT>(kw[0][s], f[0], f[2]);
          codes4<FMT>(kw[1][s], f[1], f[3]);
#pragma unroll
          for (uint32_t r = 0; r < R; ++r) mma16816(s2[s & 1][r], f, q[r][s]);
        }
      } else {
        // thread t's D / 4 channels are D / 64 blocks of 16; a word is half a block
        uint32_t mu[2][D / 64];
#pragma unroll
        for (uint32_t u = 0; u < 2; ++u)
#pragma unroll
          for (uint32_t x = 0; x < D / 64; ++x) {
            const uint32_t e = st[T::kMicro + (g + 8 * u) * (D / 16) + t * (D / 64) + x];
            mu[u][x] = e4m3x2_half2(e | (e << 8));
          }
#pragma unroll
        for (uint32_t w = 0; w < T::kSteps / 2; ++w) {
          uint32_t h0[4], h1[4];
          codes8(kw[0][w], h0);
          codes8(kw[1][w], h1);
#pragma unroll
          for (uint32_t y = 0; y < 2; ++y) {
            const uint32_t f[4] = {hmul2(h0[2 * y], mu[0][w / 2]), hmul2(h1[2 * y], mu[1][w / 2]),
                                   hmul2(h0[2 * y + 1], mu[0][w / 2]), hmul2(h1[2 * y + 1], mu[1][w / 2])};
#pragma unroll
            for (uint32_t r = 0; r < R; ++r) mma16816(s2[y][r], f, q[r][2 * w + y]);
          }
        }
      }
      // ---- softmax: this thread's tokens g, g + 8 and rows 2t, 2t + 1
      const float sk[2] = {sc[g], sc[g + 8]}, sv[2] = {sc[16 + g], sc[24 + g]};
      const int32_t tok = int32_t((first + k * stride) * kTile + g);
      const bool border = tok - int32_t(g) + int32_t(kTile) > all_see;
      float x[R][4], lv[2];  // S, then the weights
      bool slow = false;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        lv[u] = lg2(fmaxf(sv[u], 0x1p-149f));  // a row of zeros has codes of zero: any finite logarithm does
        slow |= sv[u] != sv[u];
#pragma unroll
        for (uint32_t r = 0; r < R; ++r)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float& v = x[r][2 * u + j];
            v = (s2[0][r][2 * u + j] + s2[1][r][2 * u + j]) * (sk[u] * rs[r][j]);
            if (border && !(tok + 8 * u < min(lim[r][j], int32_t(len)))) v = -INFINITY;
            slow |= fmaxf(v - n[r][j], (v + lv[u]) - m[r][j]) > 15.f;
          }
      }
      bool nans = false;  // a value row is NaN
      if (__any_sync(0xffffffffu, slow)) {
        nans = __any_sync(0xffffffffu, sv[0] != sv[0] || sv[1] != sv[1]);
        // one row's m or n, up to 7 below the largest v of its tokens; the factor that its sums take
        auto move = [](float& ref, float v0, float v1) {
          float top = fmaxf(v0, v1);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          const float to = fmaxf(ref, top - 7.f), f = to == ref ? 1.f : ex2(ref - to);
          ref = to;
          return f;
        };
#pragma unroll
        for (uint32_t r = 0; r < R; ++r)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            l[r][j] *= move(n[r][j], x[r][j], x[r][j + 2]);
            const float f = move(m[r][j], x[r][j] + lv[0], x[r][j + 2] + lv[1]);
#pragma unroll
            for (uint32_t i = 0; i < T::kSteps; ++i) {
              o[r][i][j] *= f;
              o[r][i][j + 2] *= f;
            }
          }
      }
      uint32_t pw[R][2];
#pragma unroll
      for (uint32_t r = 0; r < R; ++r) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool hidden = border && x[r][j] == -INFINITY;
          l[r][j & 1] += hidden ? 0.f : ex2(x[r][j] - n[r][j & 1]);
          const float w = hidden ? 0.f : ex2((x[r][j] + lv[j >> 1]) - m[r][j & 1]);
          x[r][j] = nans && !hidden && sv[j >> 1] != sv[j >> 1] ? sv[j >> 1] : w;
        }
        pw[r][0] = transpose8x8(pack_half(x[r][0], x[r][1]));
        pw[r][1] = transpose8x8(pack_half(x[r][2], x[r][3]));
      }
      // ---- o: channel group g of tokens 2t, 2t + 1 | 2t + 8, 2t + 9
      const uint8_t* vs = st + T::kKArea + T::value_place(g, t) * T::kVBytes;
      uint32_t vw[4][T::kVBytes / 4];
#pragma unroll
      for (uint32_t u = 0; u < 4; ++u) {
        const uint8_t* p = vs + u * 32 * T::kVBytes;
        if constexpr (T::kVBytes == 16) {
          const uint4 w = *reinterpret_cast<const uint4*>(p);
          vw[u][0] = w.x, vw[u][1] = w.y, vw[u][2] = w.z, vw[u][3] = w.w;
        } else if constexpr (T::kVBytes == 8) {
          const uint2 w = *reinterpret_cast<const uint2*>(p);
          vw[u][0] = w.x, vw[u][1] = w.y;
        } else {
          vw[u][0] = *reinterpret_cast<const uint32_t*>(p);
        }
      }
      if constexpr (!T::k4) {
        // channels 4 i .. 4 i + 3 of the group: pairs of tokens of one channel
#pragma unroll
        for (uint32_t i = 0; i < T::kVBytes / 4; ++i) {
          uint32_t f[2][4];
          codes4<FMT>(__byte_perm(vw[0][i], vw[1][i], 0x5140), f[0][0], f[0][1]);
          codes4<FMT>(__byte_perm(vw[2][i], vw[3][i], 0x5140), f[0][2], f[0][3]);
          codes4<FMT>(__byte_perm(vw[0][i], vw[1][i], 0x7362), f[1][0], f[1][1]);
          codes4<FMT>(__byte_perm(vw[2][i], vw[3][i], 0x7362), f[1][2], f[1][3]);
#pragma unroll
          for (uint32_t r = 0; r < R; ++r) {
            mma16816(o[r][2 * i], f[0], pw[r]);
            mma16816(o[r][2 * i + 1], f[1], pw[r]);
          }
        }
      } else {
        uint32_t mu[2];  // micro-scales of the pairs
#pragma unroll
        for (uint32_t u = 0; u < 2; ++u) {
          const uint8_t* e = st + T::kMicro + (16 + 2 * t + 8 * u) * (D / 16) + g * D / 128;
          mu[u] = e4m3x2_half2(uint32_t(e[0]) | (uint32_t(e[D / 16]) << 8));
        }
#pragma unroll
        for (uint32_t i = 0; i < T::kVBytes / 4; ++i) {  // channels 8 i .. 8 i + 7 of the group
          uint32_t even[2][4], uneven[2][4];
#pragma unroll
          for (uint32_t u = 0; u < 2; ++u) {
            const uint32_t p = vw[2 * u][i], n = vw[2 * u + 1][i];
            codes8((p & 0x0f0f0f0fu) | ((n & 0x0f0f0f0fu) << 4), even[u]);
            codes8(((p >> 4) & 0x0f0f0f0fu) | (n & 0xf0f0f0f0u), uneven[u]);
          }
#pragma unroll
          for (uint32_t y = 0; y < 4; ++y) {
            const uint32_t f[4] = {hmul2(even[0][y], mu[0]), hmul2(uneven[0][y], mu[0]), hmul2(even[1][y], mu[1]),
                                   hmul2(uneven[1][y], mu[1])};
#pragma unroll
            for (uint32_t r = 0; r < R; ++r) mma16816(o[r][4 * i + y], f, pw[r]);
          }
        }
      }
    }
    copy_wait<0>();
    __syncthreads();  // the ring is free for the join

    // ---- join the warps: L and the normalised o of each
    float* jl = reinterpret_cast<float*>(smem);              // [warp][row]
    float* jo = jl + T::kWarps * T::kRows;                   // [warp][row][D]
#pragma unroll
    for (uint32_t r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float s = l[r][j];
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        // 2^(m - n) in two halves: it may leave fp32's range where the answer does not
        const float inv = s == 0.f ? 0.f : 1.f / s, half = s == 0.f ? 0.f : exp2f(0.5f * (m[r][j] - n[r][j]));
        const uint32_t row = r * 8 + 2 * t + j;
        if (g == 0) jl[warp * T::kRows + row] = s == 0.f ? -INFINITY : n[r][j] + log2f(s);
        float* dst = jo + (warp * T::kRows + row) * D + g * (D / 8);
#pragma unroll
        for (uint32_t i = 0; i < T::kSteps; ++i) {
          dst[2 * i] = o[r][i][j] * inv * half * half;
          dst[2 * i + 1] = o[r][i][j + 2] * inv * half * half;
        }
      }
    __syncthreads();
    constexpr uint32_t kPer = D / 32;  // channels a lane
    for (uint32_t row = warp; row < T::kRows && group * T::kRows + row < total_rows; row += T::kWarps) {
      float top = -INFINITY, sum = 0.f, w[T::kWarps], y[kPer];
#pragma unroll
      for (uint32_t i = 0; i < T::kWarps; ++i) {
        w[i] = jl[i * T::kRows + row];
        top = fmaxf(top, w[i]);
      }
#pragma unroll
      for (uint32_t j = 0; j < kPer; ++j) y[j] = 0.f;
#pragma unroll
      for (uint32_t i = 0; i < T::kWarps; ++i) {
        const float f = w[i] == -INFINITY ? 0.f : ex2(0.5f * (w[i] - top));  // half the factor
        sum = fmaf(f, f, sum);
#pragma unroll
        for (uint32_t j = 0; j < kPer; ++j)
          y[j] = fmaf(f, f * jo[(i * T::kRows + row) * D + lane * kPer + j], y[j]);
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (uint32_t j = 0; j < kPer; ++j) y[j] *= inv;
      const float L = sum == 0.f ? -INFINITY : top + log2f(sum);
      const uint32_t rr = group * T::kRows + row;
      const int32_t i = rows.first + int32_t(rr / a.G);
      const uint32_t hq = h * a.G + rr % a.G;
      const uint64_t id = uint64_t(i) * a.Hq + hq;
      if (direct) {
        store_out<kPer>(a, i, hq, lane * kPer, y);
        if (a.lse && lane == 0) a.lse[id] = L * kLn2;
      } else {
        const uint64_t at = uint64_t(part0 + part) * parts.rows + id;
        if (lane == 0) parts.lse[at] = L;
        float* dst = parts.o + at * D + lane * kPer;
        if (kPer == 4)
          *reinterpret_cast<float4*>(dst) = make_float4(y[0], y[1], y[kPer - 2], y[kPer - 1]);
        else
          *reinterpret_cast<float2*>(dst) = make_float2(y[0], y[1]);
      }
    }
    __syncthreads();
  }
  await_previous();
}

}  // namespace
}  // namespace kvc
