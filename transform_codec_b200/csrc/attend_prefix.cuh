// Attention of all the batch's query rows over the prefix they share, on the
// 5th-generation tensor cores. GPU-library only.
//
// Per head the rows of every sequence stand below one another, so that each
// 128-token block of keys and values is read once for 256 rows: 4 * 256 * 128 *
// D operations against 512 D bytes, beyond the card's operations per byte; with
// few rows it is the reading that bounds.
//
// A block of 12 warps: two groups of four do the softmax of one 128-row tile
// each, one row a thread; the third group's warps bring K blocks, bring V blocks
// (TMA, 128-byte swizzle, a ring each), issue Q K^T and issue P V, and leave
// registers to the others: 200 * 256 + 104 * 128 is the 168 * 384 that the block
// starts with. Two tiles take turns, so the
// products of one run while the other's softmax does:
//     S_r = Q_r K_j^T                        (Q, K in shared memory, S in tensor memory)
//     P_r = 2^(scale S_r - m_r), 16 bits     (threads; back to tensor memory)
//     O_r += P_r V_j                         (P in tensor memory, V token-major in shared memory)
// With more than 128 rows the tiles are 256 different rows on the same blocks;
// with fewer they are the same rows on alternate blocks, joined at the end.
// m_r is a reference 7 below the row's largest score when it was set; O moves to
// a new one only when a score passes it by 15 (P up to 2^15 keeps its bits in
// fp16 as in bf16), which is rare after the first blocks. P is rounded to the
// values' type, the sum l takes it before the rounding.
//
// Measured: 32,768 tokens for 1024 rows of 8 heads of 128 (137 GFLOP), 4 parts, 128
// blocks: 114 us between events in a stream of calls (1.2 PFLOP/s), 123 alone and
// cold at 1.60 GHz, where the tensor pipe is 69% active and the special-function
// pipe 70%. A step of 2 x 128 rows x 128 tokens takes 2700 clocks of the tensor
// pipe's 2048; beginning and end of a block take 19 us. 128 rows over 8192 tokens: 26
// us cold, of which a block works for 6; the rest is its beginning and end.
//
// Every wait is bounded: one that runs out sets KVC_ERR_TIMEOUT, stops all roles,
// and the block leaves NaN behind after what it has in flight has landed.
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

// A bounded wait that another role's stop ends too.
__device__ inline bool wait_or_stop(uint32_t bar, uint32_t parity, const volatile uint32_t* stop) {
  for (uint32_t i = 0; i + 1 <= KVC_MMA_WAIT_POLLS; ++i) {
    uint32_t there;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(there)
        : "r"(bar), "r"(parity)
        : "memory");
    if (there) return true;
    if (*stop) return false;
  }
  return false;
}
__device__ inline bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// Whether a phase has ended, without waiting: asked early, the answer's own
// latency is hidden.
__device__ inline uint32_t is_there(uint32_t bar, uint32_t parity) {
  uint32_t there;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(there)
      : "r"(bar), "r"(parity)
      : "memory");
  return there;
}
__device__ inline void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
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
// The loads' end: values in v are used after it, not before.
__device__ inline void tmem_landed32(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]),
                 "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28])
               :
               : "memory");
  asm volatile("" : "+f"(v[29]), "+f"(v[30]), "+f"(v[31])::"memory");
}
// pairs of fp32 at once
__device__ inline float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return r;
}
__device__ inline float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ inline float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return r;
}
__device__ inline void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <uint32_t D>
struct PrefixTile {
  static constexpr uint32_t kThreads = 384, kRows = 128, kTokens = 128;
  static constexpr uint32_t kBlock = kTokens * D * 2;  // bytes of a K or V block, or of a Q tile
  static constexpr uint32_t kHalf = kTokens * 128;     // 64 channels of it
  static constexpr uint32_t kKStages = D == 128 ? 2 : 4, kVStages = D == 128 ? 3 : 4;
  static constexpr uint32_t kK = 2 * kBlock, kV = kK + kKStages * kBlock;  // rings, after two Q tiles
  static constexpr uint32_t kBars = kV + kVStages * kBlock;
  static constexpr uint32_t kSmem = 1024 + kBars + 256;
  static constexpr uint32_t kP = 128, kO = 256;        // tensor-memory columns of P_0 and O_0; S at 0
};
struct PrefixBars {
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4], s_full[2], s_free, p_full[2], o_done[2], drain[2], tail;
  uint32_t tmem, stop, seen;
};
static_assert(sizeof(PrefixBars) <= 256, "barrier area");

// grid (prefix parts * row blocks, H)
template <uint32_t DT, uint32_t D>
__global__ void __launch_bounds__(384, 1)
k_attend_prefix(const AttendArgs a, const PartsView parts, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap, const uint32_t n_parts, const uint32_t blocks_per_part,
                const uint32_t direct) {
  using T = PrefixTile<D>;
  constexpr bool kBf16 = DT == KVC_DTYPE_BF16;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  PrefixBars& B = *reinterpret_cast<PrefixBars*>(smem + T::kBars);
  const uint32_t tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31u;
  const uint32_t part = blockIdx.x % n_parts, h = blockIdx.y;
  const uint64_t total_rows = uint64_t(a.n_rows) * a.G;
  const bool same_rows = total_rows <= T::kRows;  // both tiles hold the same rows
  const uint64_t row0 = uint64_t(blockIdx.x / n_parts) * (2 * T::kRows);

  let_next_begin();
  if (tid == 0) {
    for (uint32_t i = 0; i < 4; ++i) {
      tc::mbar_init(&B.k_full[i], 1);
      tc::mbar_init(&B.k_empty[i], 1);
      tc::mbar_init(&B.v_full[i], 1);
      tc::mbar_init(&B.v_empty[i], 1);
    }
    for (uint32_t r = 0; r < 2; ++r) {
      tc::mbar_init(&B.s_full[r], 1);
      tc::mbar_init(&B.p_full[r], T::kRows);
      tc::mbar_init(&B.o_done[r], 1);
    }
    tc::mbar_init(&B.s_free, T::kRows);
    tc::mbar_init(&B.drain[0], 1);
    tc::mbar_init(&B.drain[1], 1);
    tc::mbar_init(&B.tail, 32);
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
    // rows with something to see; a warp brings its 32 rows, whole rows at a time
    const int64_t src = int64_t(row / a.G) * a.q_tok + int64_t(h * a.G + uint32_t(row % a.G)) * a.q_head;
    const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative scale goes into q's signs
    constexpr uint32_t kLanes = D / 8, kAtOnce = 32 / kLanes;
    uint4 w[32 / kAtOnce];
#pragma unroll
    for (uint32_t i = 0; i < 32 / kAtOnce; ++i) {
      const uint32_t from = i * kAtOnce + lane / kLanes;
      const int64_t at = __shfl_sync(0xffffffffu, src, from);
      const bool used = __shfl_sync(0xffffffffu, see, from) != 0;
      w[i] = make_uint4(0, 0, 0, 0);
      const uint16_t* p = static_cast<const uint16_t*>(a.q) + at + lane % kLanes * 8;
      if (used) w[i] = __ldg(reinterpret_cast<const uint4*>(p));
    }
#pragma unroll
    for (uint32_t i = 0; i < 32 / kAtOnce; ++i) {
      const uint32_t to = (warp & 3u) * 32 + i * kAtOnce + lane / kLanes;
      *reinterpret_cast<uint4*>(smem + r * T::kBlock + tc::sw128_offset(to, lane % kLanes * 16, T::kRows)) =
          make_uint4(w[i].x ^ flip, w[i].y ^ flip, w[i].z ^ flip, w[i].w ^ flip);
    }
    tc::fence_async_smem();
  } else if (a.q_start) {
    // each sequence's range and share are looked at once, also where no row lies in
    // it; with a cache its kernel looks at the ranges
    const uint64_t id = (uint64_t(blockIdx.y) * gridDim.x + blockIdx.x) * 128u + my;
    for (uint64_t b = id; b < a.n_seqs; b += uint64_t(gridDim.x) * gridDim.y * 128u) {
      if (!a.has_cache) rows_of_seq(a, uint32_t(b));
      prefix_seen(a, uint32_t(b));
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t seen = B.seen;  // the longest share in this block's rows
  const uint32_t nb = seen > token0 ? (seen - token0 + T::kTokens - 1) / T::kTokens : 0u;
  const uint32_t tmem = B.tmem;
  volatile uint32_t* stop = &B.stop;
  // one answer for the whole warp; another role's stop ends the wait too
  auto await = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_or_stop(tc::smem_addr(bar), parity, stop)) != 0;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 8 || warp == 11) {
      // ---- loads: K blocks, V blocks
      const bool is_v = warp == 11;
      const uint32_t stages = is_v ? T::kVStages : T::kKStages;
      uint64_t* full = is_v ? B.v_full : B.k_full;
      uint64_t* empty = is_v ? B.v_empty : B.k_empty;
      uint8_t* ring = smem + (is_v ? T::kV : T::kK);
      uint32_t b = 0;
      if (lane == 0) {
        const CUtensorMap* map = is_v ? &vmap : &kmap;
        for (; b < nb; ++b) {
          const uint32_t s = b % stages, use = b / stages;
          if (use && !wait_or_stop(tc::smem_addr(&empty[s]), (use - 1) & 1u, stop)) {
            *stop = 1;
            break;
          }
          const uint32_t dst = tc::smem_addr(ring + s * T::kBlock);
          mbar_expect(&full[s], T::kBlock);
#pragma unroll
          for (uint32_t x = 0; x < D / 64; ++x)
            tma_load3(dst + x * T::kHalf, map, int32_t(x * 64), int32_t(token0 + b * T::kTokens), int32_t(h), &full[s]);
        }
        // what was issued lands before the block leaves, also after a stop
        for (uint32_t i = b > stages ? b - stages : 0; i < b; ++i)
          tc::mbar_wait(&full[i % stages], (i / stages) & 1u, kDrainPolls);
      }
      __syncwarp();
      b = __shfl_sync(0xffffffffu, b, 0);
      const uint32_t first = (seen - token0) % T::kTokens;
      if (is_v && b == nb && nb && first) {
        // tokens of the last block that no row of this block sees may hold anything;
        // their weights are zero, and so must be what they multiply
        const uint32_t n = (T::kTokens - first) * 8;
        uint8_t* v = ring + (nb - 1) % stages * T::kBlock;
        for (uint32_t i = lane; i < n * (D / 64); i += 32)
          *reinterpret_cast<uint4*>(v + (i / n) * T::kHalf + first * 128 + (i % n) * 16) = make_uint4(0, 0, 0, 0);
        tc::fence_async_smem();
        mbar_arrive(&B.tail);
      }
    } else if (nb) {
      // ---- products: one warp issues Q K^T, the other P V. The issue of a product
      // waits for the tensor pipe, a few products deep, and a wait for a barrier that
      // is already there still takes some 200 clocks: with one warp for both the
      // pipe ran dry in between. One lane issues, the whole warp walks along, so that
      // operands are uniform.
      bool ok = true;
      uint32_t stage = 0, phase = 0;  // of the warp's next block
      auto await_u = [&](uint32_t bar, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, wait_or_stop(bar, parity, stop)) != 0;
        return ok;
      };
      if (warp == 9) {
        const uint32_t s_desc = idesc_16(kBf16, 128, 128, false);
        const uint64_t q0 = tc::desc_sw128(tc::smem_addr(smem)), k0 = tc::desc_sw128(tc::smem_addr(smem + T::kK));
        const uint32_t full0 = tc::smem_addr(&B.k_full[0]), empty0 = tc::smem_addr(&B.k_empty[0]),
                       s_full0 = tc::smem_addr(&B.s_full[0]), s_free = tc::smem_addr(&B.s_free);
        // One S at a time stands in tensor memory: the next may come once the last has
        // been taken to registers. So the S of a tile is there when its softmax
        // returns from the one before.
        const uint32_t items = same_rows ? nb : 2 * nb;
        for (uint32_t it = 0; it < items; ++it) {
          const uint32_t t = it & 1u;
          const bool takes = same_rows || !t, frees = same_rows || t;
          if (takes) await_u(full0 + stage * 8, phase);
          if (it) await_u(s_free, (it - 1) & 1u);
          if (!ok) break;
          tc::fence_after_sync();
          const uint64_t q = q0 + t * (T::kBlock >> 4), k = k0 + stage * (T::kBlock >> 4);
          if (elect_one()) {
#pragma unroll
            for (uint32_t s = 0; s < D / 16; ++s) {
              const uint32_t off = ((s / 4) * T::kHalf + (s % 4) * 32) >> 4;
              tc::mma_bf16(tmem, q + off, k + off, s_desc, s != 0);
            }
            commit(s_full0 + t * 8);
            if (frees) commit(empty0 + stage * 8);
          }
          if (frees && ++stage == T::kKStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      } else {
        const uint32_t o_desc = idesc_16(kBf16, 128, D, true);
        const uint64_t v0 = desc_mn_sw128(tc::smem_addr(smem + T::kV), T::kHalf);
        const uint32_t full0 = tc::smem_addr(&B.v_full[0]), empty0 = tc::smem_addr(&B.v_empty[0]),
                       p_full0 = tc::smem_addr(&B.p_full[0]), o_done0 = tc::smem_addr(&B.o_done[0]);
        const bool tail = (seen - token0) % T::kTokens != 0;
        const uint32_t items = same_rows ? nb : 2 * nb;
        for (uint32_t it = 0; it < items; ++it) {
          const uint32_t t = it & 1u, turn = it >> 1;
          const bool takes = same_rows || !t, frees = same_rows || t;
          if (takes) {
            await_u(full0 + stage * 8, phase);
            if (tail && (same_rows ? it : turn) + 1 == nb) await_u(tc::smem_addr(&B.tail), 0);
          }
          await_u(p_full0 + t * 8, turn & 1u);
          if (!ok) break;
          tc::fence_after_sync();
          const uint64_t v = v0 + stage * (T::kBlock >> 4);
          if (elect_one()) {
#pragma unroll
            for (uint32_t s = 0; s < T::kTokens / 16; ++s)
              mma_ts(tmem + T::kO + t * D, tmem + T::kP + t * 64 + s * 8, v + s * (2048 >> 4), o_desc,
                   turn != 0 || s != 0);
            commit(o_done0 + t * 8);
            if (frees) commit(empty0 + stage * 8);
          }
          if (frees && ++stage == T::kVStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) *stop = 1;
      // all products have ended before tensor memory is given back, also after a stop
      if (elect_one()) commit(tc::smem_addr(&B.drain[warp - 9]));
      tc::mbar_wait(&B.drain[warp - 9], 0, kDrainPolls);
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ---- softmax of row `my` of tile r
    const uint32_t turns = same_rows ? (nb + 1 - r) / 2 : nb;
    const uint32_t lanes = ((warp & 3u) * 32u) << 16;  // this warp's lanes of tensor memory
    const uint32_t s_at = tmem + lanes, p_at = s_at + T::kP + r * 64, o_at = s_at + T::kO + r * D;
    const float scale = fabsf(a.scale_log2);
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    uint32_t s_there = 0;
    for (uint32_t n = 0; n < turns; ++n) {
      const uint32_t b = same_rows ? 2 * n + r : n;
      if (!__all_sync(0xffffffffu, s_there)) {
        ok = await(&B.s_full[r], n & 1u);
        if (!ok) break;
      }
      tc::fence_after_sync();
      const uint32_t base = token0 + b * T::kTokens;
      const uint32_t left = see > base ? see - base : 0u;  // tokens of the block that the row sees
      const bool none = left == 0, part_seen = left < T::kTokens && !none;
      const bool border = __any_sync(0xffffffffu, part_seen), skips = __any_sync(0xffffffffu, none);
      float x[128];
#pragma unroll
      for (uint32_t c = 0; c < 4; ++c) tmem_ld32(s_at + 32 * c, x + 32 * c);
#pragma unroll
      for (uint32_t c = 0; c < 4; ++c) tmem_landed32(x + 32 * c);
      tc::fence_before_sync();
      mbar_arrive(&B.s_free);
      if (border) {
#pragma unroll
        for (uint32_t i = 0; i < 128; ++i) x[i] = i < left ? x[i] : -INFINITY;
      }
      float top[4];
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) top[i] = max3(x[i], x[4 + i], x[8 + i]);
#pragma unroll
      for (uint32_t i = 12; i < 124; i += 8)
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) top[j] = max3(top[j], x[i + j], x[i + 4 + j]);
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) top[j] = max3(top[j], x[124 + j], x[124 + j]);
      float high = max3(max3(top[0], top[1], top[2]), top[3], top[3]) * scale;
      const bool odd = !(high < INFINITY);  // a NaN or an infinity among the scores
      if (none) high = -INFINITY;
      const bool move = high > m + 15.f;
      const bool moves = __any_sync(0xffffffffu, move);
      float f = 1.f;
      if (moves && move) {
        f = exp2f(m - (high - 7.f));
        m = high - 7.f;
        l *= f;
      }
      // a row that has seen nothing yet: its weights are zero
      const float ref = m == -INFINITY ? 0.f : -m;
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      uint32_t p[64], o_there = 0;
#pragma unroll
      for (uint32_t i = 0; i < 64; ++i) {
        float2 e = fma2(make_float2(x[2 * i], x[2 * i + 1]), make_float2(scale, scale), make_float2(ref, ref));
        e.x = ex2(e.x);
        e.y = ex2(e.y);
        if (i == 40 && n) o_there = is_there(tc::smem_addr(&B.o_done[r]), (n - 1) & 1u);
        sum[i & 1] = add2(sum[i & 1], e);
        p[i] = pack16<DT>(e.x, e.y);
      }
      sum[0] = add2(sum[0], sum[1]);
      float add = sum[0].x + sum[0].y;
      if (odd) add = __uint_as_float(0x7fc00000u);
      if (skips) {
        const uint32_t keep = none ? 0u : 0xffffffffu;
#pragma unroll
        for (uint32_t i = 0; i < 64; ++i) p[i] &= keep;
        if (none) add = 0.f;
      }
      l += add;
      if (n) {  // the product of the last P has read it, and O is complete
        if (!__all_sync(0xffffffffu, o_there)) {
          ok = await(&B.o_done[r], (n - 1) & 1u);
          if (!ok) break;
        }
        tc::fence_after_sync();
        if (moves) {
#pragma unroll
          for (uint32_t i = 0; i < D / 32; ++i) {
            float o[32];
            tmem_ld32(o_at + 32 * i, o);
            tmem_landed32(o);
#pragma unroll
            for (uint32_t j = 0; j < 32; ++j) o[j] *= f;
            tmem_st32(o_at + 32 * i, reinterpret_cast<const uint32_t*>(o));
          }
        }
      }
      s_there = n + 1 < turns ? is_there(tc::smem_addr(&B.s_full[r]), (n + 1) & 1u) : 0u;
      tmem_st32(p_at, p);
      tmem_st32(p_at + 32, p + 32);
      tmem_wait_st();
      tc::fence_before_sync();
      mbar_arrive(&B.p_full[r]);
    }
    if (ok && turns) ok = await(&B.o_done[r], (turns - 1) & 1u);  // the last products
    if (!ok) {
      *stop = 1;
      flag_status(a.res, KVC_ERR_TIMEOUT);
      // what there is of O is no answer: NaN reaches the output and lse of every row
      // that needed it, also through the joins
      l = see ? __uint_as_float(0x7fc00000u) : 0.f;
    }
    tc::fence_after_sync();
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const float L = l == 0.f ? -INFINITY : m + log2f(l);
    float* other = reinterpret_cast<float*>(smem + T::kK);  // the second tile's results: [D][128], then L
    float f0 = inv, f1 = 0.f, LL = L;
    if (same_rows) {
      // every load and product of this block has ended once both groups are here
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (r == 1) {
#pragma unroll
        for (uint32_t i = 0; i < D / 32; ++i) {
          float o[32] = {};
          if (turns) tmem_ld32(o_at + 32 * i, o);
          tmem_landed32(o);
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
      // 32 channels of the warp's 32 rows at a time go through the tile's Q space,
      // so that rows leave 128 bytes at a time
      const int32_t i0 = int32_t(row / a.G);
      const uint32_t hq = h * a.G + uint32_t(row % a.G);
      const uint64_t id = uint64_t(i0) * a.Hq + hq;
      const uint64_t at = uint64_t(part) * parts.rows + id;
      float4* stage = reinterpret_cast<float4*>(smem + r * T::kBlock + (warp & 3u) * 4096);
      const bool writes = live && (direct || LL != -INFINITY);
      // the rows that this lane writes channels of: 4 k + lane / 8
      int64_t to[8];
      uint32_t w = 0;
      {
        const int64_t mine = direct ? i0 * a.o_tok + int64_t(hq) * a.o_head : int64_t(at * D);
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) {
          to[k] = __shfl_sync(0xffffffffu, mine, k * 4 + lane / 8);
          w |= uint32_t(__shfl_sync(0xffffffffu, uint32_t(writes), k * 4 + lane / 8)) << k;
        }
      }
#pragma unroll
      for (uint32_t i = 0; i < D / 32; ++i) {
        float o[32] = {};
        if (turns) tmem_ld32(o_at + 32 * i, o);
        tmem_landed32(o);
#pragma unroll
        for (uint32_t j = 0; j < 32; ++j) {
          o[j] = turns && l != 0.f ? o[j] * f0 : 0.f;
          if (same_rows) o[j] = fmaf(other[(32 * i + j) * 128 + my], f1, o[j]);
        }
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j)
          stage[lane * 8 + (j ^ (lane & 7u))] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        __syncwarp();
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) {
          const uint32_t rr = k * 4 + lane / 8, u = lane & 7u;
          const float4 v = stage[rr * 8 + (u ^ (rr & 7u))];
          if (!(w >> k & 1u)) continue;
          if (direct)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + to[k] + 32 * i + 4 * u) =
                make_uint2(pack16<DT>(v.x, v.y), pack16<DT>(v.z, v.w));
          else
            *reinterpret_cast<float4*>(parts.o + to[k] + 32 * i + 4 * u) = v;
        }
        __syncwarp();
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
