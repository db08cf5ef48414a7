// Attention of all the batch's query rows over the prefix they share, on the
// 5th-generation tensor cores. GPU-library only.
//
// Per head the rows of every sequence stand below one another, so that each
// 128-token block of keys and values is read once for 256 rows: 4 * 256 * 128 *
// D operations against 512 D bytes, beyond the card's operations per byte; with
// few rows it is the reading that bounds.
//
// A block of 10 warps: two groups of four do the softmax of one 128-row tile
// each, one row a thread; one warp brings K and V blocks by TMA (128-byte
// swizzle) through a ring; one issues the products. Two tiles take turns, so the
// products of one run while the other's softmax does:
//     S_r = Q_r K_j^T                        (Q, K in shared memory, S in tensor memory)
//     P_r = 2^(scale S_r - m_r), 16 bits     (threads; P over S in tensor memory)
//     O_r += P_r V_j                         (P in tensor memory, V token-major in shared memory)
// With more than 128 rows the tiles are 256 different rows on the same blocks;
// with fewer they are the same rows on alternate blocks, joined at the end.
// m_r is a reference 7 below the row's largest score when it was set; O moves to
// a new one only when a score passes it by 15 (P up to 2^15 keeps its bits in
// fp16 as in bf16), which is rare after the first blocks. P is rounded to the
// values' type, the sum l takes it before the rounding.
//
// Every wait is bounded: one that runs out sets KVC_ERR_TIMEOUT, stops all roles,
// and the block leaves after what it has in flight has landed.
#pragma once
#include <cuda.h>

#include "attend_parts.cuh"
#include "tcgen05.cuh"

#ifndef KVC_MMA_WAIT_POLLS
#define KVC_MMA_WAIT_POLLS (1u << 22)
#endif

namespace kvc {
namespace {

constexpr uint32_t kDrainPolls = 1u << 22;  // waits for what is in flight, in every build

__device__ inline void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc::smem_addr(bar)) : "memory");
}
__device__ inline void mbar_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(tc::smem_addr(bar)), "r"(bytes)
               : "memory");
}
__device__ inline void tma_load3(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
          "r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(tc::smem_addr(bar))
      : "memory");
}
// 16-bit operands, fp32 sums; b_mn: B's N index is the contiguous one in memory
__host__ __device__ constexpr uint32_t idesc_16(bool bf16, uint32_t M, uint32_t N, bool b_mn) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_mn ? 1u : 0u) << 16) |
         ((N >> 3) << 17) | ((M >> 4) << 24);
}
// A from tensor memory
__device__ inline void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Operand whose contiguous index is N: 128-byte-swizzled atoms of 64 N x 8 K, the
// next 64 N `lead` bytes on, the next 8 K 1024 bytes on.
__device__ inline uint64_t desc_mn_sw128(uint32_t saddr, uint32_t lead) {
  return uint64_t((saddr >> 4) & 0x3fffu) | (uint64_t(lead >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
__device__ inline void tmem_ld32(uint32_t addr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ inline void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}
__device__ inline void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <uint32_t D>
struct PrefixTile {
  static constexpr uint32_t kThreads = 320, kRows = 128, kTokens = 128;
  static constexpr uint32_t kBlock = kTokens * D * 2;  // bytes of a K or V block, or of a Q tile
  static constexpr uint32_t kHalf = kTokens * 128;     // 64 channels of it
  static constexpr uint32_t kStages = D == 128 ? 5 : 8;
  static constexpr uint32_t kRing = 2 * kBlock;        // offset: after two Q tiles
  static constexpr uint32_t kBars = kRing + kStages * kBlock;
  static constexpr uint32_t kSmem = 1024 + kBars + 256;
  static constexpr uint32_t kO = 256;                  // tensor-memory column of O_0; S_r at 128 r
};
struct PrefixBars {
  uint64_t full[8], empty[8], s_full[2], p_full[2], pv_done[2], drain;
  uint32_t tmem, stop, seen;
};
static_assert(sizeof(PrefixBars) <= 256, "barrier area");

// grid (prefix parts * row blocks, H)
template <uint32_t DT, uint32_t D>
__global__ void __launch_bounds__(320, 1)
k_attend_prefix(const AttendArgs a, const PartsView parts, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap, const uint32_t n_parts, const uint32_t blocks_per_part,
                const uint32_t direct) {
  using T = PrefixTile<D>;
  constexpr bool kBf16 = DT == KVC_DTYPE_BF16;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  PrefixBars& B = *reinterpret_cast<PrefixBars*>(smem + T::kBars);
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
  const uint32_t part = blockIdx.x % n_parts, h = blockIdx.y;
  const uint64_t total_rows = uint64_t(a.n_rows) * a.G;
  const bool same_rows = total_rows <= T::kRows;  // both tiles hold the same rows
  const uint64_t row0 = uint64_t(blockIdx.x / n_parts) * (2 * T::kRows);

  if (tid == 0) {
    for (uint32_t i = 0; i < T::kStages; ++i) {
      tc::mbar_init(&B.full[i], 1);
      tc::mbar_init(&B.empty[i], 1);
    }
    for (uint32_t r = 0; r < 2; ++r) {
      tc::mbar_init(&B.s_full[r], 1);
      tc::mbar_init(&B.p_full[r], T::kRows);
      tc::mbar_init(&B.pv_done[r], 1);
    }
    tc::mbar_init(&B.drain, 1);
    B.stop = 0;
    B.seen = 0;
  }
  if (warp == 9) {
    tc::tmem_alloc(&B.tmem, 512u);
    tc::tmem_relinquish();
  }
  __syncthreads();

  // ---- rows: Q tiles into shared memory, and how far each row sees
  const uint32_t r = warp >> 2, my = tid & 127u;  // softmax groups: tile and row of it
  const uint64_t row = row0 + (same_rows ? 0 : r * T::kRows) + my;
  const uint32_t token0 = part * blocks_per_part * T::kTokens;
  const uint32_t token1 = min(a.prefix_tokens, token0 + blocks_per_part * T::kTokens);
  uint32_t see = 0;  // tokens [token0, see) of this part are seen
  bool live = false;
  if (warp < 8) {
    if (row < total_rows) {
      const RowPlace at = place_of_row(a, int32_t(row / a.G));
      live = at.seq >= 0;
      if (live) see = min(prefix_seen(a, uint32_t(at.seq)), token1);
    }
    if (see <= token0) see = 0;
    if (see) atomicMax(&B.seen, see);
    const uint16_t* src =
        static_cast<const uint16_t*>(a.q) + int64_t(row / a.G) * a.q_tok + int64_t(h * a.G + row % a.G) * a.q_head;
    const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative scale goes into q's signs
#pragma unroll
    for (uint32_t i = 0; i < D / 8; ++i) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (see) {
        w = *reinterpret_cast<const uint4*>(src + i * 8);
        w.x ^= flip, w.y ^= flip, w.z ^= flip, w.w ^= flip;
      }
      *reinterpret_cast<uint4*>(smem + r * T::kBlock + tc::sw128_offset(my, i * 16, T::kRows)) = w;
    }
    tc::fence_async_smem();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t seen = B.seen;  // the longest share in this block's rows
  const uint32_t nb = seen > token0 ? (seen - token0 + T::kTokens - 1) / T::kTokens : 0u;
  const uint32_t tmem = B.tmem;
  // items: (tile, token block) pairs in the order of their products
  const uint32_t items = same_rows ? nb : 2 * nb;
  // K and V blocks enter the ring in the order they are used
  auto k_at = [&](uint32_t b) { return same_rows ? (b ? 2 * b - 1 : 0u) : 2 * b; };
  auto v_at = [&](uint32_t b) { return same_rows && b + 1 < nb ? 2 * b + 2 : 2 * b + 1; };
  volatile uint32_t* stop = &B.stop;
  // one answer for the whole warp
  auto await = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, !*stop && tc::mbar_wait(bar, parity, KVC_MMA_WAIT_POLLS)) != 0;
  };

  if (warp == 8) {
    // ---- loads
    if (lane == 0) {
      uint32_t issued = 0;
      for (; issued < 2 * nb && !*stop; ++issued) {
        const uint32_t s = issued % T::kStages, use = issued / T::kStages;
        if (use && !tc::mbar_wait(&B.empty[s], (use - 1) & 1u, KVC_MMA_WAIT_POLLS)) {
          *stop = 1;
          break;
        }
        // which block is this?
        bool is_v;
        uint32_t b;
        if (!same_rows) {
          is_v = issued & 1u;
          b = issued >> 1;
        } else if (issued == 0) {
          is_v = false;
          b = 0;
        } else if (issued == 2 * nb - 1) {
          is_v = true;
          b = nb - 1;
        } else {
          is_v = !(issued & 1u);
          b = is_v ? (issued - 2) / 2 : (issued + 1) / 2;
        }
        const CUtensorMap* map = is_v ? &vmap : &kmap;
        const uint32_t dst = tc::smem_addr(smem + T::kRing + s * T::kBlock);
        mbar_expect(&B.full[s], T::kBlock);
#pragma unroll
        for (uint32_t x = 0; x < D / 64; ++x)
          tma_load3(dst + x * T::kHalf, map, int32_t(x * 64), int32_t(token0 + b * T::kTokens), int32_t(h), &B.full[s]);
      }
      // what was issued lands before the block leaves, also after a stop
      for (uint32_t i = issued > T::kStages ? issued - T::kStages : 0; i < issued; ++i)
        tc::mbar_wait(&B.full[i % T::kStages], (i / T::kStages) & 1u, kDrainPolls);
    }
  } else if (warp == 9) {
    // ---- products
    const uint32_t s_desc = idesc_16(kBf16, 128, 128, false), o_desc = idesc_16(kBf16, 128, D, true);
    bool ok = true;
    auto await_full = [&](uint32_t at) {
      ok = await(&B.full[at % T::kStages], (at / T::kStages) & 1u);
    };
    auto issue_s = [&](uint32_t it) {
      const uint32_t t = it & 1u, b = same_rows ? it : it >> 1, at = k_at(b);
      if (same_rows || !t) await_full(at);
      if (!ok) return;
      tc::fence_after_sync();
      if (lane == 0) {
        const uint32_t q = tc::smem_addr(smem + t * T::kBlock), k = tc::smem_addr(smem + T::kRing + (at % T::kStages) * T::kBlock);
#pragma unroll
        for (uint32_t s = 0; s < D / 16; ++s) {
          const uint32_t off = (s / 4) * T::kHalf + (s % 4) * 32;
          const uint64_t qd = tc::desc_sw128(q + off), kd = tc::desc_sw128(k + off);
          tc::mma_bf16(tmem + t * 128, qd, kd, s_desc, s != 0);
        }
        tc::mma_commit(&B.s_full[t]);
        if (same_rows || t) tc::mma_commit(&B.empty[at % T::kStages]);
      }
      __syncwarp();
    };
    if (items > 0) issue_s(0);
    if (items > 1) issue_s(1);
    for (uint32_t it = 0; it < items && ok; ++it) {
      const uint32_t t = it & 1u, b = same_rows ? it : it >> 1, at = v_at(b), turn = it >> 1;
      if (same_rows || !t) {
        await_full(at);
        if (!ok) break;
        // tokens that no row of the block sees may hold anything: their weights are
        // zero, and so must be what they are multiplied with
        const uint32_t base = token0 + b * T::kTokens;
        if (base + T::kTokens > seen) {
          uint8_t* v = smem + T::kRing + (at % T::kStages) * T::kBlock;
          const uint32_t first = seen - base, n = (T::kTokens - first) * 8;
          for (uint32_t i = lane; i < n * (D / 64); i += 32)
            *reinterpret_cast<uint4*>(v + (i / n) * T::kHalf + first * 128 + (i % n) * 16) = make_uint4(0, 0, 0, 0);
          tc::fence_async_smem();
          __syncwarp();
        }
      }
      ok = await(&B.p_full[t], turn & 1u);
      if (!ok) break;
      tc::fence_after_sync();
      if (lane == 0) {
        const uint32_t v = tc::smem_addr(smem + T::kRing + (at % T::kStages) * T::kBlock);
#pragma unroll
        for (uint32_t s = 0; s < T::kTokens / 16; ++s)
          mma_ts(tmem + T::kO + t * D, tmem + t * 128 + s * 8, desc_mn_sw128(v + s * 2048, T::kHalf), o_desc,
                 turn != 0 || s != 0);
        tc::mma_commit(&B.pv_done[t]);
        if (same_rows || t) tc::mma_commit(&B.empty[at % T::kStages]);
      }
      __syncwarp();
      // S over P of the same tile: products run in the order of their issue
      if (it + 2 < items) issue_s(it + 2);
    }
    if (!ok) *stop = 1;
    if (lane == 0) {  // products in flight end before tensor memory is given back, also after a stop
      tc::mma_commit(&B.drain);
      tc::mbar_wait(&B.drain, 0, kDrainPolls);
    }
    __syncwarp();
  } else {
    // ---- softmax of row `my` of tile r
    const uint32_t turns = same_rows ? (nb + 1 - r) / 2 : nb;
    const uint32_t lanes = ((warp & 3u) * 32u) << 16;  // this warp's lanes of tensor memory
    const uint32_t s_at = tmem + lanes + r * 128, o_at = tmem + lanes + T::kO + r * D;
    const float scale = fabsf(a.scale_log2);
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (uint32_t n = 0; n < turns; ++n) {
      const uint32_t b = same_rows ? 2 * n + r : n;
      ok = await(&B.s_full[r], n & 1u);
      if (!ok) break;
      tc::fence_after_sync();
      float s[128];
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) tmem_ld32(s_at + 32 * i, s + 32 * i);
      tc::tmem_wait_ld();
      const uint32_t base = token0 + b * T::kTokens;
      const uint32_t left = see > base ? see - base : 0u;  // tokens of the block that the row sees
      if (__any_sync(0xffffffffu, left < T::kTokens)) {
#pragma unroll
        for (uint32_t i = 0; i < 128; ++i) s[i] = i < left ? s[i] : -INFINITY;
      }
      float top = s[0];
#pragma unroll
      for (uint32_t i = 1; i < 128; ++i) top = fmaxf(top, s[i]);
      top *= scale;
      const bool move = top > m + 15.f;
      if (__any_sync(0xffffffffu, move)) {
        const float to = move ? top - 7.f : m;
        const float f = move ? exp2f(m - to) : 1.f;
        m = to;
        l *= f;
        if (n) {
          ok = await(&B.pv_done[r], (n - 1) & 1u);
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll
          for (uint32_t i = 0; i < D / 32; ++i) {
            float o[32];
            tmem_ld32(o_at + 32 * i, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (uint32_t j = 0; j < 32; ++j) o[j] *= f;
            tmem_st32(o_at + 32 * i, reinterpret_cast<const uint32_t*>(o));
          }
          tmem_wait_st();
        }
      }
      // a row that has seen nothing yet: every weight is zero
      const float ref = m == -INFINITY ? 0.f : m;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i) {
        uint32_t p[32];
#pragma unroll
        for (uint32_t j = 0; j < 32; ++j) {
          const float x = ex2(fmaf(s[64 * i + 2 * j], scale, -ref)), y = ex2(fmaf(s[64 * i + 2 * j + 1], scale, -ref));
          sum[j & 1] += x;
          sum[2 + (j & 1)] += y;
          p[j] = pack16<DT>(x, y);
        }
        tmem_st32(s_at + 32 * i, p);
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tmem_wait_st();
      tc::fence_before_sync();
      mbar_arrive(&B.p_full[r]);
    }
    if (ok && turns) ok = await(&B.pv_done[r], (turns - 1) & 1u);  // the tile's last products
    if (!ok) {
      *stop = 1;
      if (a.res) *reinterpret_cast<volatile int32_t*>(&a.res->status) = KVC_ERR_TIMEOUT;
    }
    tc::fence_after_sync();
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const float L = l == 0.f ? -INFINITY : m + log2f(l);
    float* other = reinterpret_cast<float*>(smem + T::kRing);  // the second tile's results: [D][128], then L
    float f0 = inv, f1 = 0.f, LL = L;
    if (same_rows) {
      // every load and product of this block has ended once both groups are here
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (r == 1) {
#pragma unroll
        for (uint32_t i = 0; i < D / 32; ++i) {
          float o[32];
          if (turns) tmem_ld32(o_at + 32 * i, o);
          tc::tmem_wait_ld();
#pragma unroll
          for (uint32_t j = 0; j < 32; ++j) other[(32 * i + j) * 128 + my] = turns && l != 0.f ? o[j] * inv : 0.f;
        }
        other[D * 128 + my] = L;
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (r == 0) {
        const float L1 = other[D * 128 + my];
        const float t2 = fmaxf(L, L1);
        const float w0 = L == -INFINITY ? 0.f : exp2f(L - t2), w1 = L1 == -INFINITY ? 0.f : exp2f(L1 - t2);
        const float w = w0 + w1;
        LL = w == 0.f ? -INFINITY : t2 + log2f(w);
        f0 = w == 0.f ? 0.f : inv * (w0 / w);
        f1 = w == 0.f ? 0.f : w1 / w;
      }
    }
    if (r == 0 || !same_rows) {
      const int32_t i0 = int32_t(row / a.G);
      const uint32_t hq = h * a.G + uint32_t(row % a.G);
      const uint64_t id = uint64_t(i0) * a.Hq + hq;
      const uint64_t at = uint64_t(part) * parts.rows + id;
#pragma unroll
      for (uint32_t i = 0; i < D / 32; ++i) {
        float o[32];
        if (turns) tmem_ld32(o_at + 32 * i, o);
        tc::tmem_wait_ld();
#pragma unroll
        for (uint32_t j = 0; j < 32; ++j) {
          o[j] = turns && l != 0.f ? o[j] * f0 : 0.f;
          if (same_rows) o[j] = fmaf(other[(32 * i + j) * 128 + my], f1, o[j]);
        }
        if (live && direct) {
          store_out<32>(a, i0, hq, 32 * i, o);
        } else if (live && !direct && LL != -INFINITY) {
          float4* dst = reinterpret_cast<float4*>(parts.o + at * D + 32 * i);
#pragma unroll
          for (uint32_t j = 0; j < 8; ++j) dst[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        }
      }
      if (live) {
        if (!direct)
          parts.lse[at] = LL;
        else if (a.lse)
          a.lse[id] = LL * kLn2;
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 9) tc::tmem_dealloc(B.tmem, 512u);
}

}  // namespace
}  // namespace kvc
