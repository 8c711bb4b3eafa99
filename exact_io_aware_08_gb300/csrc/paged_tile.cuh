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

// The bf16 cache as the copying warp sees it.
struct PagedCache {
  const int* table;
  int H_kv, num_blocks, block_size, max_blocks;
  int shift;                                                  // a copy takes 2^shift rows, which never cross a page
  int step_blocks, step_rows;                                 // a tile on: whole blocks, and rows
};

// A sequence's tiles of 128 keys in a row, by the whole warp: a lane holds one piece of a tile (and one 64-column half).
// Tiles are counted on, without divisions, and the page of the next one is asked for ahead: a warp by itself takes 4 to 5
// clocks an instruction, and 200 of them a tile bound the long reads (16 x 32768 keys of 4 heads: 186 us).
template <int D>
struct PagedStream {
  static constexpr int HALVES = D / 64;
  const int* table;
  int key, end, blk, row, page;                               // of the lane's piece of the next tile
  int copies;                                                 // whether the lane has one
  int offset;                                                 // in the tile, bytes

  __device__ __forceinline__ explicit PagedStream(const PagedCache& c) {
    const int lane = threadIdx.x & 31, pieces_log2 = 7 - c.shift, half = lane >> pieces_log2, pi = lane & ((1 << pieces_log2) - 1);
    copies = half < HALVES;
    offset = half * kPagedTile * 128 + (pi << (c.shift + 7));
  }

  __device__ __forceinline__ int entry() const { return copies && key < end ? __ldg(table + blk) : 0; }

  // Keys [key0, end0) of sequence b, which lie within its table.
  __device__ __forceinline__ void begin(const PagedCache& c, int b, int key0, int end0) {
    table = c.table + static_cast<size_t>(b) * c.max_blocks;
    key = key0 + ((offset & (kPagedTile * 128 - 1)) >> 7);
    end = end0;
    blk = key / c.block_size;
    row = key - blk * c.block_size;
    page = entry();
  }

  // The cache row of the lane's piece of the next tile, or -1.
  __device__ __forceinline__ int next(const PagedCache& c, int where) {
    int at = -1;
    if (copies && key < end) {
      if (static_cast<unsigned>(page) >= static_cast<unsigned>(c.num_blocks)) {
        report_device_error(FA_DEV_BAD_CONFIG, where);
        page = 0;                                             // stays in bounds; the result is reported invalid
      }
      at = page * c.block_size + row;
    }
    key += kPagedTile;
    blk += c.step_blocks;
    row += c.step_rows;
    if (row >= c.block_size) {
      row -= c.block_size;
      ++blk;
    }
    page = entry();
    return at;
  }

  // Brings the tile whose pieces are at ``at`` as a 128-byte-swizzled one, [D / 64][128][64], counted on ``bar``.  Rows
  // behind the last key that share no copy with one before it keep what they held.
  __device__ __forceinline__ void load(const PagedCache& c, const CUtensorMap* map, uint8_t* dst, uint64_t* bar, int hkv, int at) const {
    const int live = __popc(__ballot_sync(0xffffffffu, at >= 0));
    if ((threadIdx.x & 31) == 0) mbar_arrive_expect_tx(bar, live << (c.shift + 7));
    __syncwarp();
    if (at >= 0) tma_load_3d(dst + offset, map, bar, offset >> 14 << 6, hkv, at);
    __syncwarp();
  }
};

// Rows of a copy for a block size that is a multiple of 16.
inline int paged_piece(int block_size) {
  return block_size % 128 == 0 ? 128 : block_size % 64 == 0 ? 64 : block_size % 32 == 0 ? 32 : 16;
}

inline PagedCache paged_cache(const int* table, int H_kv, int num_blocks, int block_size, int max_blocks) {
  const int piece = paged_piece(block_size);
  return {table, H_kv, num_blocks, block_size, max_blocks, piece == 128 ? 7 : piece == 64 ? 6 : piece == 32 ? 5 : 4,
          kPagedTile / block_size, kPagedTile % block_size};
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
