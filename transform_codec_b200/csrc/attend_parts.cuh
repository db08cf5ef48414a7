// What the attention kernels share: where rows and sequences lie, how the work
// on a row is divided into parts, and how parts are joined. GPU-library only.
//
// A part is attention over some of a row's tokens: the normalised output in
// fp32 and the base-2 logarithm of its sum of exponentials, L. Parts join as
// sum_p 2^(L_p - L) o_p with L = log2 sum_p 2^L_p; one that saw nothing has L =
// -infinity and o = 0. The factors are multiplied in as two halves, 2^((L_p - L) / 2):
// one below fp32's range may stand before values far above 1 (a part of zero rows
// with large scores beside one of rows of 2^100).
#pragma once
#include "cache_codes.cuh"
#include "serving.h"

namespace kvc {

constexpr float kLn2 = 0.6931471805599453f;

// Workspace: L of every (part, row, query head), then o.
struct PartsView {
  float* lse;     // [parts][n_rows * Hq]
  float* o;       // [parts][n_rows * Hq][D]
  uint64_t rows;  // n_rows * Hq
};

// The kernels of one call follow one another without a gap: each lets the next
// begin once all its blocks run, and waits for the one before only where it needs
// it done: the join before it reads, the cache kernel (which needs nothing of the
// prefix kernel's) before it ends, so that the join's wait for it covers both.
__device__ inline void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ inline void await_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Sequence b's query rows; a range that is not within the rows given is refused.
struct SeqRows {
  int32_t first, n;
};
__device__ inline SeqRows rows_of_seq(const AttendArgs& a, uint32_t b) {
  if (!a.q_start) return {int32_t(b), 1};
  const int32_t first = __ldg(a.q_start + b), last = __ldg(a.q_start + b + 1);
  if (first < 0 || last < first || last > int32_t(a.n_rows)) {
    flag_invalid(a.res);
    return {0, 0};
  }
  return {first, last - first};
}
// The sequence of query row i, -1: none.
struct RowPlace {
  int32_t seq, first, n;
};
__device__ inline RowPlace place_of_row(const AttendArgs& a, int32_t i) {
  if (!a.q_start) return {i < int32_t(a.n_seqs) ? i : -1, i, 1};
  uint32_t lo = 0, hi = a.n_seqs - 1;  // the last sequence that starts at or before i
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
  return {int32_t(lo), first, last - first};
}
// Cache tokens of sequence b, within what its page table can hold.
__device__ inline uint32_t cache_len(const AttendArgs& a, const CacheView& c, uint32_t b) {
  const int64_t len = __ldg(a.kv_len + b), room = int64_t(a.pages_stride) << c.page_shift;
  if (len < 0 || len > room) flag_invalid(a.res);
  return uint32_t(max(int64_t(0), min(len, room)));
}
// Prefix tokens that sequence b sees.
__device__ inline uint32_t prefix_seen(const AttendArgs& a, uint32_t b) {
  if (!a.prefix_len) return a.prefix_tokens;
  const int32_t n = __ldg(a.prefix_len + b);
  if (n < 0 || uint32_t(n) > a.prefix_tokens) flag_invalid(a.res);
  return n < 0 ? 0u : min(uint32_t(n), a.prefix_tokens);
}

// A sequence's cache in 16-token tiles, divided among at most `splits` blocks of
// at least kLeastTiles tiles each; `parts` is how many of them have work (1 for
// an empty sequence: its one block writes an empty part).
constexpr uint32_t kTile = 16, kLeastTiles = 4;
struct Chunks {
  uint32_t per, parts;  // tiles a block, blocks
};
__host__ __device__ inline Chunks chunks_of(uint32_t len, uint32_t splits) {
  const uint32_t tiles = len / kTile + (len % kTile != 0);
  uint32_t per = (tiles + splits - 1) / splits;
  if (per < kLeastTiles) per = kLeastTiles;
  const uint32_t parts = (tiles + per - 1) / per;
  return {per, parts ? parts : 1u};
}

// A finished row: 16-bit output of one channel group and the natural lse.
template <uint32_t N>
__device__ inline void store_out(const AttendArgs& a, int32_t i, uint32_t hq, uint32_t ch, const float* y) {
  uint16_t* p = static_cast<uint16_t*>(a.out) + i * a.o_tok + int64_t(hq) * a.o_head + ch;
#pragma unroll
  for (uint32_t j = 0; j < N; j += 2) {
    const uint32_t w = a.dtype == KVC_DTYPE_BF16 ? pack_bf16(y[j], y[j + 1]) : pack_half(y[j], y[j + 1]);
    *reinterpret_cast<uint32_t*>(p + j) = w;
  }
}

}  // namespace kvc
