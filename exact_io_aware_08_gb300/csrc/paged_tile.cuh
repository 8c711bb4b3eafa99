// What the kernels over the bf16 paged cache share: a sequence's place in a step, and 128-key tiles of
// one key head brought into shared memory by TMA, page by page.
#pragma once

#include "q4.cuh"
#include "q4_share.h"

namespace fa {

constexpr int kPagedTile = 128;                               // keys of a tile

// A sequence of a step: query tokens [first, first + nq), which are the last of its len cached tokens.
struct PagedSeq {
  int first, nq, len;
  __device__ __forceinline__ int base() const { return len - nq; }   // tokens in front of the step's
};

// Bad contents are reported where ``report`` is set and leave the sequence without query tokens.
__device__ __forceinline__ PagedSeq paged_seq(const int* __restrict__ cu, const int* __restrict__ seqlens, int b, int total, int max_q,
                                              int max_k, bool report, int where) {
  PagedSeq x;
  x.first = __ldg(cu + b);
  const int end = __ldg(cu + b + 1);
  x.len = __ldg(seqlens + b);
  x.nq = end - x.first;
  if (x.first < 0 || end < x.first || end > total || x.nq > max_q || x.len < x.nq || x.len > max_k) {
    if (report) report_device_error(FA_DEV_BAD_CONFIG, where);
    x.first = x.nq = x.len = 0;
  }
  return x;
}

// By a whole warp: equal shares of all sequences' units (``units(i, first)``, ``first``: asked for the first time), and the
// sequence that holds unit ``u_of(shares)`` (b = -1 where there is none), or sequence ``at`` where that is given, with the
// units before it.
template <typename U, typename F>
__device__ __forceinline__ Q4Share paged_share(int n_seqs, int ctas, U units, F u_of, int at, int* b, long long* before) {
  const int lane = threadIdx.x & 31;
  Q4Share sh;
  long long mine = 0, own = 0;
  for (int i = lane; i < n_seqs; i += 32) {
    const long long v = units(i, true);
    if (i == lane) own = v;
    mine += v;
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  sh.set(mine, ctas);
  const long long u = at >= 0 ? 1LL << 62 : u_of(sh);
  long long sum = 0;
  *b = -1;
  for (int base = 0; base < n_seqs && u >= 0; base += 32) {
    const long long v = base == 0 ? own : base + lane < n_seqs ? units(base + lane, false) : 0;
    long long inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    const uint32_t beyond = __ballot_sync(0xffffffffu, at >= 0 ? base + lane >= at : sum + inc > u);
    if (beyond) {
      const int l = __ffs(beyond) - 1;
      *b = base + l;
      *before = sum + __shfl_sync(0xffffffffu, inc - v, l);
      break;
    }
    sum += __shfl_sync(0xffffffffu, inc, 31);
  }
  return sh;
}

// The bf16 cache as the copying warp sees it.  ``piece``: the rows of a copy, which never cross a page.
struct PagedCache {
  const int* table;
  int H_kv, num_blocks, block_size, max_blocks, piece;
};

// The copying warp's window of 32 entries of a sequence's block table, one a lane.
struct PageWindow {
  int b = -1, at = 0, entry = 0;

  // Page of block ``blk`` of sequence ``seq``, for a warp whose lanes ask for blocks in [lo, hi], hi - lo < 32.
  __device__ __forceinline__ int page(const PagedCache& c, int seq, int lo, int hi, int blk, int where) {
    const int lane = threadIdx.x & 31;
    if (seq != b || lo < at || hi >= at + 32) {
      b = seq;
      at = lo;
      entry = lo + lane < c.max_blocks ? __ldg(c.table + static_cast<size_t>(seq) * c.max_blocks + lo + lane) : -1;
    }
    int p = __shfl_sync(0xffffffffu, entry, (blk - at) & 31);
    if (blk <= hi && (p < 0 || p >= c.num_blocks)) {
      report_device_error(FA_DEV_BAD_CONFIG, where);
      p = 0;                                                  // stays in bounds; the result is reported invalid
    }
    return p;
  }
};

// Brings keys [key, min(key + 128, end)) of key head ``hkv`` as a 128-byte-swizzled tile [D / 64][128][64]:
// by the whole warp, counted on ``bar``.  Rows behind ``end`` that share no copy with one before it keep what
// they held.
template <int D>
__device__ __forceinline__ void load_paged_tile(const PagedCache& c, PageWindow& w, const CUtensorMap* map, uint8_t* dst, uint64_t* bar,
                                                int seq, int hkv, int key, int end, int where) {
  constexpr int CH = D / 64;
  const int lane = threadIdx.x & 31;
  const int pieces = kPagedTile / c.piece, pi = lane % pieces;
  const int k = key + pi * c.piece;
  const bool mine = lane < pieces * CH && k < end;
  const int lo = key / c.block_size, hi = (min(key + kPagedTile, end) - 1) / c.block_size;
  const int blk = mine ? k / c.block_size : lo;
  const int page = w.page(c, seq, lo, hi, blk, where);
  const int live = __popc(__ballot_sync(0xffffffffu, mine));
  if (lane == 0) mbar_arrive_expect_tx(bar, live * c.piece * 128);
  __syncwarp();
  if (mine) {
    const int ch = lane / pieces;
    tma_load_3d(dst + ch * kPagedTile * 128 + pi * c.piece * 128, map, bar, ch * 64, hkv, page * c.block_size + (k - blk * c.block_size));
  }
  __syncwarp();
}

// Rows of a copy for a block size that is a multiple of 16.
inline int paged_piece(int block_size) {
  return block_size % 128 == 0 ? 128 : block_size % 64 == 0 ? 64 : block_size % 32 == 0 ? 32 : 16;
}

inline int paged_sm_count() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 152;
  if (dev < 64 && __atomic_load_n(&cached[dev], __ATOMIC_RELAXED)) return cached[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 152;
  if (dev < 64) __atomic_store_n(&cached[dev], n, __ATOMIC_RELAXED);
  return n;
}

}  // namespace fa
