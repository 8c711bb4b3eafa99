// Keeping a paged cache short: the tokens that drew the most attention into new pages, and the accepted ones of a
// step's drafted tokens to the front of its places.
//
// Evict.  Of a sequence's tokens every key head keeps the first, the last, and between them those of the largest
// weights, the lower position where they are equal.  The weight at the border is found digit by digit: fp32 numbers
// become unsigned ones in the same order, eight bits of which are counted at a time, from the highest, among those
// that agree in all higher ones.  The kept positions then follow from two running counts along the sequence
// (above the border; at it), so that the order stays and nothing depends on the order of atomics.  Rows are copied
// by lanes of 16 bytes.
//
// What bounds it: the copy is bound by HBM (16 sequences of 10000 to 16384 tokens, 8 heads of 128, 1024 to 4096 of them
// kept: 61 us for about 330 MB read and written); the selection, 4 bytes a token, by latencies: four passes over the keys
// (from shared memory, up to kHeld of them), each with a scan of 256 counts (12 us for 4160 tokens, 22 for 16384).  Counts
// of each lane's own, or three passes of 11, 11 and 10 bits with equal digits of a warp counted together, were no faster,
// and choosing in every block that copies, without the list between them, was slower as a whole (123 us for that batch,
// 91 with the list at the time).  Candidates beyond kHeld are looked up again in every pass, through the table: 131072
// tokens of 8 heads 448 us, of which 8192 are kept (32768 tokens: 44).
//
// Accept.  Rows move down: token i of the path, at place a_i >= i of the step's, comes to place i.  A thread takes 16
// bytes of every row of a sequence, in ascending order, so that what it overwrites it has read.  It is bound by the chain
// of path, page and row: 4 trees of 26 tokens 3.7 us, with flushed caches 4.9; 128 of 64 5.7 and 7.1.
#include "fa_kernels.h"
#include "paged_tile.cuh"

namespace fa {

constexpr int kSelectThreads = 1024;
constexpr int kHeld = 48 * 1024;                              // keys held in shared memory

struct EvictParams {
  uint16_t *k, *v;
  float* weights;
  int *kept, *seqlens_out;
  const int *budgets, *seqlens, *table, *new_table;
  int H_kv, max_k, max_kept, keep_first, keep_last, max_blocks, new_max_blocks, block_size, num_blocks;
  int held;                                                   // keys that fit
};

// How many tokens a sequence keeps, or -1 (reported) where its length or budget cannot be.
__device__ __forceinline__ int evict_count(const EvictParams& p, int b, int* len, bool report) {
  *len = __ldg(p.seqlens + b);
  const int budget = __ldg(p.budgets + b), n = min(*len, budget);
  const bool bad = *len < 0 || *len > p.max_k || budget < 0 || n > p.max_kept ||
                   (*len > budget && static_cast<long long>(p.keep_first) + p.keep_last > budget);
  if (bad && report) report_device_error(FA_DEV_BAD_CONFIG, 700);
  return bad ? -1 : n;
}

// Order of weights as unsigned numbers, from 1 on; one that is no number counts as -inf.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint((w != w ? -INFINITY : w) + 0.f);   // (-0 + 0 = 0)
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Sum over the block of what the threads before this one hold, and of all (by two barriers).
__device__ __forceinline__ int block_before(int v, int* warp_sums, int* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  int s = warp_sums[lane], i = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, i, o);
    if (lane >= o) i += x;
  }
  *all = __shfl_sync(0xffffffffu, i, 31);
  return __shfl_sync(0xffffffffu, i - s, warp) + inc - v;
}

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictParams p) {
  extern __shared__ uint32_t held[];
  __shared__ int hist[256];
  __shared__ int warp_sums[32];
  __shared__ int digit[2];                                    // the border's, and how many lie above it
  const int b = blockIdx.x / p.H_kv, h = blockIdx.x - b * p.H_kv;
  int len;
  const int n = evict_count(p, b, &len, threadIdx.x == 0 && h == 0);
  pdl_launch_dependents();
  int* kept = p.kept + static_cast<size_t>(blockIdx.x) * p.max_kept;
  if (threadIdx.x == 0 && h == 0) p.seqlens_out[b] = n < 0 ? len : n;
  for (int i = max(0, n) + threadIdx.x; i < p.max_kept; i += kSelectThreads) kept[i] = -1;
  if (n < 0) return;
  if (n == len) {
    for (int i = threadIdx.x; i < n; i += kSelectThreads) kept[i] = i;
    return;
  }
  // candidates are tokens [keep_first, keep_first + c), of which k stay
  const int c = len - p.keep_first - p.keep_last, k = n - p.keep_first - p.keep_last;
  // Candidate i's key: the lowest where there is no page (reported where the row is copied).
  auto weight = [&](int i) {
    const int pos = p.keep_first + i, blk = pos / p.block_size;
    const int page = __ldg(p.table + static_cast<size_t>(b) * p.max_blocks + blk);
    if (page < 0 || page >= p.num_blocks) return 0u;
    return weight_key(p.weights[(page * p.H_kv + h) * p.block_size + (pos - blk * p.block_size)]);   // (below 2^31)
  };
  const bool hold = c <= p.held;
  if (hold)
    for (int i = threadIdx.x; i < c; i += kSelectThreads) held[i] = weight(i);
  auto key = [&](int i) { return hold ? held[i] : weight(i); };
  uint32_t border = 0;
  int want = k;                                               // of those that agree with the border so far
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += kSelectThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int i = threadIdx.x; i < c; i += kSelectThreads) {
      const uint32_t x = key(i);
      if ((x & mask) == border) atomicAdd(&hist[x >> shift & 255u], 1);
    }
    __syncthreads();
    // thread t holds digit 255 - t: the first one with ``want`` numbers at or above it
    const int mine = threadIdx.x < 256 ? hist[255 - threadIdx.x] : 0;
    int all;
    const int above = block_before(mine, warp_sums, &all);
    if (threadIdx.x < 256 && above < want && above + mine >= want) {
      digit[0] = 255 - threadIdx.x;
      digit[1] = above;
    }
    if (threadIdx.x == 0 && want == 0) digit[0] = digit[1] = -1;
    __syncthreads();
    if (want == 0) break;                                     // (k = 0: no candidate stays)
    border |= static_cast<uint32_t>(digit[0]) << shift;
    want -= digit[1];
  }
  // ``want`` of those at the border stay, the first ones.  A thread takes consecutive candidates, an odd number of them
  // (an even one met in few banks of shared memory: 32768 tokens 65 us, this way 38).
  for (int i = threadIdx.x; i < p.keep_first; i += kSelectThreads) kept[i] = i;
  for (int i = threadIdx.x; i < p.keep_last; i += kSelectThreads) kept[n - p.keep_last + i] = len - p.keep_last + i;
  if (k == 0) return;
  const int per = (c + kSelectThreads - 1) / kSelectThreads | 1;
  const int i0 = min(c, static_cast<int>(threadIdx.x) * per), i1 = min(c, i0 + per);
  int over = 0, at = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t x = key(i);
    over += x > border;
    at += x == border;
  }
  int all;
  const int over0 = block_before(over, warp_sums, &all);
  const int at0 = block_before(at, warp_sums, &all);
  int to = p.keep_first + over0 + min(at0, want), seen = at0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t x = key(i);
    if (x > border || (x == border && seen < want)) kept[to++] = p.keep_first + i;
    seen += x == border;
  }
}

constexpr int kCopyThreads = 256;
constexpr int kCopyRows = 32;                                 // kept tokens of a block (64: 240 us for 16 x 9000 of 8 heads, 32: 230)

// Copies kept rows of a key head: 16 bytes a lane, D / 8 lanes a row, K and V.
template <int D>
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const EvictParams p, int chunks) {
  constexpr int L = D / 8;
  constexpr int AT_ONCE = kCopyThreads / L;
  constexpr int U = kCopyRows / AT_ONCE;
  const int chunk = blockIdx.x % chunks, bh = blockIdx.x / chunks;
  const int b = bh / p.H_kv, h = bh - b * p.H_kv;
  int len;
  const int n = evict_count(p, b, &len, false);
  pdl_wait();
  if (chunk * kCopyRows >= n) return;
  const int u = threadIdx.x % L;
  const int* kept = p.kept + static_cast<size_t>(bh) * p.max_kept;
  size_t from[U], to[U];
  bool ok[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int i = chunk * kCopyRows + j * AT_ONCE + threadIdx.x / L;
    ok[j] = i < n;
    from[j] = to[j] = 0;
    if (ok[j]) {
      const int pos = kept[i], sb = pos / p.block_size, db = i / p.block_size;
      const int sp = sb < p.max_blocks ? __ldg(p.table + static_cast<size_t>(b) * p.max_blocks + sb) : -1;
      const int dp = db < p.new_max_blocks ? __ldg(p.new_table + static_cast<size_t>(b) * p.new_max_blocks + db) : -1;
      if (sp < 0 || sp >= p.num_blocks || dp < 0 || dp >= p.num_blocks) {
        report_device_error(FA_DEV_BAD_CONFIG, 701);
        ok[j] = false;
        continue;
      }
      from[j] = static_cast<size_t>(sp) * p.block_size + (pos - sb * p.block_size);
      to[j] = static_cast<size_t>(dp) * p.block_size + (i - db * p.block_size);
      if (u == 0) {
        const size_t sr = from[j] - static_cast<size_t>(sp) * p.block_size, dr = to[j] - static_cast<size_t>(dp) * p.block_size;
        p.weights[(static_cast<size_t>(dp) * p.H_kv + h) * p.block_size + dr] = p.weights[(static_cast<size_t>(sp) * p.H_kv + h) * p.block_size + sr];
      }
    }
  }
  uint4 x[U], y[U];
#pragma unroll
  for (int j = 0; j < U; ++j)
    if (ok[j]) {
      x[j] = reinterpret_cast<const uint4*>(p.k + (from[j] * p.H_kv + h) * D)[u];
      y[j] = reinterpret_cast<const uint4*>(p.v + (from[j] * p.H_kv + h) * D)[u];
    }
#pragma unroll
  for (int j = 0; j < U; ++j)
    if (ok[j]) {
      reinterpret_cast<uint4*>(p.k + (to[j] * p.H_kv + h) * D)[u] = x[j];
      reinterpret_cast<uint4*>(p.v + (to[j] * p.H_kv + h) * D)[u] = y[j];
    }
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
  EvictParams p{};
  p.k = static_cast<uint16_t*>(a.k_cache); p.v = static_cast<uint16_t*>(a.v_cache);
  p.weights = a.weights; p.kept = a.kept; p.seqlens_out = a.seqlens_out;
  p.budgets = a.budgets; p.seqlens = a.seqlens; p.table = a.block_table; p.new_table = a.new_table;
  p.H_kv = a.H_kv; p.max_k = a.max_k; p.max_kept = a.max_kept; p.keep_first = a.keep_first; p.keep_last = a.keep_last;
  p.max_blocks = a.max_blocks; p.new_max_blocks = a.new_max_blocks; p.block_size = a.block_size; p.num_blocks = a.num_blocks;
  p.held = min(a.max_k, kHeld);
  static int attr_done[64] = {0};
  cudaError_t e = ensure_smem_attr(evict_select_kernel, kHeld * 4, attr_done);
  if (e != cudaSuccess) return e;
  const unsigned heads = static_cast<unsigned>(a.n_seqs) * a.H_kv;
  log_launch("evict_select_kernel", heads, kSelectThreads, static_cast<unsigned long long>(p.held) * 4);
  evict_select_kernel<<<heads, kSelectThreads, p.held * 4, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.max_kept == 0) return e;
  const int chunks = (a.max_kept + kCopyRows - 1) / kCopyRows;
  log_launch("evict_copy_kernel<D>", static_cast<unsigned long long>(heads) * chunks, kCopyThreads, 0ull);
  return launch_join(a.d == 64 ? evict_copy_kernel<64> : evict_copy_kernel<128>, heads * chunks, kCopyThreads, stream, p, chunks);
}

struct AcceptParams {
  uint16_t *k, *v;
  int* seqlens_out;
  const int *accepted, *n_accepted, *cu, *seqlens, *table;
  int max_accepted, max_blocks, block_size, num_blocks, vectors;   // 16-byte vectors of a row
};

__global__ void __launch_bounds__(128) accept_kernel(const AcceptParams p) {
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int first = __ldg(p.cu + b), end = __ldg(p.cu + b + 1), len = __ldg(p.seqlens + b), n = __ldg(p.n_accepted + b);
  const int nq = end - first, base = len - nq;
  const int* path = p.accepted + static_cast<size_t>(b) * p.max_accepted;
  const int* pages = p.table + static_cast<size_t>(b) * p.max_blocks;
  bool ok = first >= 0 && end >= first && base >= 0 && n >= 0 && n <= nq && n <= p.max_accepted &&
            (nq == 0 || (len - 1) / p.block_size < p.max_blocks);
  // ascending places within the step, whose pages are there
  auto sound = [&](int place) {
    const int page = __ldg(pages + (base + place) / p.block_size);
    return page >= 0 && page < p.num_blocks;
  };
  for (int i = lane; ok && i < n; i += 32) {
    const int a = __ldg(path + i), before = i ? __ldg(path + i - 1) : -1;
    if (a <= before || a >= nq || !sound(a) || !sound(i)) ok = false;
  }
  ok = __all_sync(0xffffffffu, ok);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (!ok) report_device_error(FA_DEV_BAD_CONFIG, 710);
    p.seqlens_out[b] = ok ? base + n : len;
  }
  const int u = blockIdx.x * 128 + threadIdx.x;
  if (!ok || u >= 2 * p.vectors) return;
  uint4* cache = reinterpret_cast<uint4*>(u < p.vectors ? p.k : p.v) + (u < p.vectors ? u : u - p.vectors);
  auto row = [&](int place) {
    const int pos = base + place, blk = pos / p.block_size;
    return cache + (static_cast<size_t>(__ldg(pages + blk)) * p.block_size + (pos - blk * p.block_size)) * p.vectors;
  };
  constexpr int AT_ONCE = 8;
  for (int i0 = 0; i0 < n; i0 += AT_ONCE) {
    uint4 x[AT_ONCE];
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j)
      if (i0 + j < n) x[j] = *row(__ldg(path + i0 + j));
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j)
      if (i0 + j < n && __ldg(path + i0 + j) != i0 + j) *row(i0 + j) = x[j];
  }
}

cudaError_t launch_accept(const AcceptArgs& a, cudaStream_t stream) {
  AcceptParams p{static_cast<uint16_t*>(a.k_cache), static_cast<uint16_t*>(a.v_cache), a.seqlens_out, a.accepted, a.n_accepted,
                 a.cu, a.seqlens, a.block_table, a.max_accepted, a.max_blocks, a.block_size, a.num_blocks, a.H_kv * a.d / 8};
  const dim3 grid(static_cast<unsigned>((2 * p.vectors + 127) / 128), static_cast<unsigned>(a.n_seqs));
  log_launch("accept_kernel", static_cast<unsigned long long>(grid.x) * grid.y, 128, 0ull);
  accept_kernel<<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fa

FA_DEFINE_STATUS_FETCH(status_fetch_evict)
