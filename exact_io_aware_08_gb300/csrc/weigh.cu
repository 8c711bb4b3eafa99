// How much attention each cached token draws: w[k] = decay w[k] + sum over rows r of exp(scale q_r k - lse_r), where
// the rows of a key head are its query heads times the step's tokens, and a token's rows see the keys up to its own.
//
// Mathematics.  The attention's weights again, from its queries, keys and log-sum-exps, summed down the columns of
// S instead of along its rows: S^T = K Q^T puts a key on each lane of tensor memory, so that a thread adds up its own
// key's weights and nothing is exchanged.  A weight is 2^(c s - lse log2 e) with c = scale log2 e, one fused operation: c
// and lse log2 e are rounded, by 2^-24 of themselves each, which in a weight that counts is some 2^-23 |lse|.  Products
// are exact, sums fp32, and each tile of 128 rows is summed before it is added.
//
// What bounds it.  2 d flops and an exponential a (row, key): with few rows the reading of K, with many the
// exponentials (32 a clock and SM: 1024 clocks for 256 keys times 128 rows, as many as the products take).
//
// Layout of both kernels:
//   warp 0       copies K tiles, warp 2 tiles of Q (whole tokens, all heads of the group), warp 3 their lse: a tile of
//                Q is given back when its products are done, its lse when it has been added up.
//   warp 1       issues the products.
//   warps 4 on   the sums, thread = key.
// Few rows (up to three tiles of them): Q stays, each CTA gets an equal share of all keys (Q4Share), 256 at a time with two
// S buffers for each half.  (By the kernel for many rows, caches not flushed: two tiles, 32 x 64 tokens over 500 keys 31 us,
// this way 23; three, 4 x 90 over 1000 18 and 15, but 16 x 96 over 8000 both 110.)  Else a CTA keeps 512 keys and runs over
// the rows that see them, four tiles of keys by turns, so that a tile of Q is brought for 512 keys and the sums of one key tile run beside
// the products of the others.  The (512 keys, row tile) units are shared out equally too; the sums of 512 keys that lie in
// several shares are added up, in order, by a second kernel.  (2 x 4096 tokens in whole ranges of row tiles, dealt out in
// rounds: 152 us.)
//
// Measured, 32 heads over 8, d = 128, caches flushed before each call: 32 single tokens over 100 to 8191 62 us (5.4 TB/s of
// keys and weights), 16 x 64 tokens over 8000 88, 2 prompts of 4096 121 (1.13 PFLOP/s; without the sums 95).
#include "fa_kernels.h"
#include "paged_tile.cuh"

namespace fa {

template <int D>
struct WeighCfg {
  static constexpr int TILE = 128 * D * 2;
  static constexpr int CHUNK = 128 * 128;
  static constexpr int NK = D == 128 ? 4 : 8;                 // K tiles
  static constexpr int NQ = kWeighFewTiles;                   // tiles of Q
  static constexpr int OFF_K = 0;
  static constexpr int OFF_Q = NK * TILE;
  static constexpr int OFF_LSE = OFF_Q + NQ * TILE;
  static constexpr int OFF_BAR = OFF_LSE + NQ * 128 * 4;
  // k_full[NK], k_empty[NK], q_full[NQ], q_empty[NQ], l_full[NQ], l_empty[NQ], s_full[4], s_empty[4]
  static constexpr int NBAR = 2 * NK + 4 * NQ + 8;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 48 + 1024;      // (TMEM slot, abort flag, start[5], out[NQ])
  static_assert(SMEM_BYTES <= 232448, "shared memory budget (227 KB per CTA)");
  static constexpr int PAIRS = NK / 2;                        // few rows: pairs of K tiles in flight
  static constexpr int FEW_THREADS = 384, MANY_THREADS = 640;
  static constexpr uint32_t BAR_S = 1, BAR_S_THREADS = 128 + 32;   // many rows: S of key tile a has been read
};
constexpr int kWeighKeys = 512;                               // of a piece with many rows

struct WeighParams {
  CUtensorMap tk, tq;
  PagedCache cache;
  const float* lse;
  float *weights, *part;                                      // part: sums of cut pieces, two of 512 keys a CTA
  const int *cu, *seqlens, *weighed;
  int n_seqs, H, G, total, max_q, max_k;
  int tokens, rows;                                           // rows of a tile: ``tokens`` whole tokens
  float c2, decay;                                            // scale * log2 e
};

// Where a weight lies, or null (a page that is not there is reported by the copying warp).
__device__ __forceinline__ float* weigh_place(const WeighParams& p, int b, int hkv, int key) {
  const int blk = key / p.cache.block_size;
  const int page = __ldg(p.cache.table + static_cast<size_t>(b) * p.cache.max_blocks + blk);
  if (page < 0 || page >= p.cache.num_blocks) return nullptr;
  return p.weights + (static_cast<size_t>(page) * p.cache.H_kv + hkv) * p.cache.block_size + (key - blk * p.cache.block_size);
}

__device__ __forceinline__ int weigh_pairs(const PagedSeq& s) { return s.nq ? (s.len + 255) / 256 : 0; }

// Few rows: a stretch of key pairs [kt0, kt1) of a key head of a sequence.
struct WeighStretch {
  int b, hkv, kt0, kt1, tiles;                                // (row tiles)
  PagedSeq seq;
};
struct WeighWalk {
  const WeighParams& p;
  int b, off, left;                                           // sequence, unit in it, units left
  PagedSeq seq;
  int pairs;

  __device__ __forceinline__ bool next(WeighStretch& x) {
    if (left <= 0) return false;
    while (off >= pairs * p.cache.H_kv) {
      if (++b >= p.n_seqs) return false;
      off = 0;
      seq = paged_seq(p.cu, p.seqlens, b, p.total, p.max_q, p.max_k, false, 0);
      pairs = weigh_pairs(seq);
    }
    x.b = b;
    x.seq = seq;
    x.tiles = (seq.nq + p.tokens - 1) / p.tokens;
    x.hkv = off / pairs;
    x.kt0 = off - x.hkv * pairs;
    const int n = min(left, pairs - x.kt0);
    x.kt1 = x.kt0 + n;
    off += n;
    left -= n;
    return true;
  }
};

// Many rows: pieces of 512 keys of a sequence against its row tiles.  Piece j has units(j) units: one for bringing its
// keys, and as many as row tiles see them, or nearly (whole multiples of 512 keys are taken for so many whole row tiles,
// which makes their sum a closed form); its row tiles [first, tiles) are shared out in proportion to units.
struct WeighPieces {
  int pieces, tiles, step, skip, base, tokens;                // row tiles; of 512 keys; that begin before the step's tokens end
  __device__ __forceinline__ WeighPieces(const WeighParams& p, const PagedSeq& s) {
    pieces = s.nq ? (s.len + kWeighKeys - 1) / kWeighKeys : 0;
    tokens = p.tokens;
    tiles = (s.nq + tokens - 1) / tokens;
    step = kWeighKeys / tokens;
    base = s.base();
    skip = (base + tokens - 1) / tokens;
  }
  __device__ __forceinline__ int units(int j) const { return tiles - max(0, j * step - skip) + 1; }
  __device__ __forceinline__ long long total() const {        // of a key head
    const long long from = skip / step + 1, n = max(0LL, pieces - from);
    return static_cast<long long>(pieces) * (tiles + 1) - (step * (from + pieces - 1) * n / 2 - skip * n);
  }
  // First row tile behind the first k units of piece j.
  __device__ __forceinline__ int row_tile(int j, int k) const {
    const int first = max(0, j * kWeighKeys - base) / tokens;
    return first + static_cast<int>(static_cast<long long>(max(0, k - 1)) * (tiles - first) / (units(j) - 1));
  }
};

template <typename F>
__device__ __forceinline__ Q4Share weigh_share(const WeighParams& p, int ctas, bool report, F u_of, int* b, long long* before) {
  return paged_share(p.n_seqs, ctas, [&](int i, bool first) {
    return WeighPieces(p, paged_seq(p.cu, p.seqlens, i, p.total, p.max_q, p.max_k, report && first, 600)).total() * p.cache.H_kv;
  }, u_of, -1, b, before);
}

// Key head and piece of unit u of sequence ``x``; u becomes the unit in the piece.
__device__ __forceinline__ void weigh_piece_of(const WeighPieces& x, long long* u, int* hkv, int* j) {
  const long long all = x.total();
  *hkv = static_cast<int>(*u / all);
  *u -= *hkv * all;
  *j = 0;
  while (*u >= x.units(*j)) *u -= x.units((*j)++);
}

// Piece kt of a key head of a sequence against row tiles [q0, q1).  slot: -1 all of them, else the place of their sums.
struct WeighPiece {
  int b, hkv, kt, q0, q1, slot;
  PagedSeq seq;
};
struct WeighParts {
  const WeighParams& p;
  int b, hkv, kt, k;                                          // next unit: sequence, key head, piece, unit in it
  long long left;

  __device__ __forceinline__ bool next(WeighPiece& x) {
    while (left > 0) {
      x.seq = paged_seq(p.cu, p.seqlens, b, p.total, p.max_q, p.max_k, false, 0);
      const WeighPieces y(p, x.seq);
      if (kt >= y.pieces) {
        kt = k = 0;
        if (++hkv >= p.cache.H_kv || y.pieces == 0) {
          hkv = 0;
          if (++b >= p.n_seqs) return false;
        }
        continue;
      }
      const int units = y.units(kt), n = static_cast<int>(min(left, static_cast<long long>(units - k)));
      x.b = b;
      x.hkv = hkv;
      x.kt = kt;
      x.q0 = y.row_tile(kt, k);
      x.q1 = y.row_tile(kt, k + n);
      x.slot = n == units ? -1 : 2 * static_cast<int>(blockIdx.x) + (k == 0 ? 1 : 0);
      left -= n;
      k += n;
      if (k == units) {
        k = 0;
        ++kt;
      }
      if (x.q0 < x.q1) return true;
    }
    return false;
  }

  // Key tiles of the piece that hold keys, and of these the first ones that row tile qt sees (one at least).
  __device__ __forceinline__ int tiles(const WeighPiece& x) const { return min(4, (x.seq.len - x.kt * kWeighKeys + 127) / 128); }
  __device__ __forceinline__ int seen(const WeighPiece& x, int qt, int n) const {
    return min(n, ((min(x.seq.nq, (qt + 1) * p.tokens) - 1 + x.seq.base() - x.kt * kWeighKeys) >> 7) + 1);
  }
};

// Shared memory of a CTA.
template <int D>
struct WeighShared {
  using C = WeighCfg<D>;
  uint8_t *k, *q;
  float* lse;
  uint64_t *k_full, *k_empty, *q_full, *q_empty, *l_full, *l_empty, *s_full, *s_empty;
  uint32_t* tmem_slot;
  volatile int* abort_flag;
  int *start, *out;                                           // out: whether some row of a tile's lse is -inf
  __device__ __forceinline__ explicit WeighShared(uint8_t* smem) {
    k = smem + C::OFF_K;
    q = smem + C::OFF_Q;
    lse = reinterpret_cast<float*>(smem + C::OFF_LSE);
    k_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    k_empty = k_full + C::NK;
    q_full = k_empty + C::NK;
    q_empty = q_full + C::NQ;
    l_full = q_empty + C::NQ;
    l_empty = l_full + C::NQ;
    s_full = l_empty + C::NQ;
    s_empty = s_full + 4;
    tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
    start = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);
    out = start + 5;
  }
  // By one thread: ``k_arrivals`` copies make a K slot full, ``sum_warps`` give lse back, four warps an S buffer.
  __device__ __forceinline__ void init(int k_arrivals, int sum_warps) const {
    for (int s = 0; s < C::NK; ++s) {
      mbar_init(&k_full[s], k_arrivals);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < C::NQ; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
      mbar_init(&l_full[s], 1);
      mbar_init(&l_empty[s], sum_warps);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&s_empty[s], 4);
    }
    *abort_flag = 0;
    fence_mbarrier_init();
  }
};

// One row tile of Q: by one lane.
template <int D>
__device__ __forceinline__ void weigh_load_q(const WeighParams& p, const WeighShared<D>& m, int slot, int hkv, int token) {
  using C = WeighCfg<D>;
  mbar_arrive_expect_tx(&m.q_full[slot], p.rows * D * 2);
#pragma unroll
  for (int ch = 0; ch < D / 64; ++ch)
    tma_load_4d(m.q + slot * C::TILE + ch * C::CHUNK, &p.tq, &m.q_full[slot], ch * 64, 0, hkv, token);
}

// -lse log2 e of the rows of tiles, by a warp, four rows a lane.  The next tile's is asked for before this one's is
// written (with a load behind each wait 242 us for 2 x 4096 tokens at the time, 148 without).
struct WeighLse {
  const WeighParams& p;
  int token_of[4], head_of[4];
  float e[4];
  __device__ __forceinline__ explicit WeighLse(const WeighParams& p_) : p(p_) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 32 + (threadIdx.x & 31);
      token_of[i] = r / p.G;
      head_of[i] = r - token_of[i] * p.G;
      e[i] = 0.f;
    }
  }
  __device__ __forceinline__ void ask(const PagedSeq& s, int hkv, int qt, float (&v)[4]) const {
    const int n = min(p.tokens, s.nq - qt * p.tokens);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = token_of[i] < n ? __ldg(p.lse + static_cast<size_t>(hkv * p.G + head_of[i]) * p.total + s.first + qt * p.tokens + token_of[i])
                             : -INFINITY;
  }
  // ``n``: tokens of the tile.  (Rows that see nothing weigh nothing, and ``out`` is set: -inf and a score that is no
  // finite number would not add up to -inf.)
  __device__ __forceinline__ void write(int n, float* to, int* out) const {
    bool some = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      some |= token_of[i] < n && e[i] == -INFINITY;
      to[i * 32 + (threadIdx.x & 31)] = e[i] == -INFINITY ? -INFINITY : e[i] * -1.4426950408889634f;
    }
    some = __any_sync(0xffffffffu, some);
    if ((threadIdx.x & 31) == 0) *out = some;
  }
};

// S^T = K Q^T of one tile each, by the converged warp.
template <int D>
__device__ __forceinline__ void weigh_product(uint32_t to, uint64_t dk, uint64_t dq, uint32_t idesc, uint64_t* done) {
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const uint32_t off = (ks >> 2) * WeighCfg<D>::CHUNK + (ks & 3) * 32;
    umma_ss_w(to, desc_advance(dk, off), desc_advance(dq, off), idesc, ks > 0);
  }
  umma_commit_w(done);
}

// Which of a tile's columns count for a key: [lo, hi), lo between lo_min and lo_max in all lanes.
struct WeighSpan {
  int lo, lo_min, lo_max, hi;
  // of key ``key`` (this lane's) against rows [r0, r0 + n) of its sequence
  __device__ __forceinline__ WeighSpan(const WeighParams& p, const PagedSeq& s, int key, int r0, int n) {
    const int first = key - (threadIdx.x & 31);
    lo = max(0, key - s.base()) * p.G - r0;
    lo_min = max(0, first - s.base()) * p.G - r0;
    lo_max = max(0, first + 31 - s.base()) * p.G - r0;
    hi = n;
  }
};

// Adds up the weights of a tile's columns, W from tensor memory at a time up to ``cols``; ``nl``: -lse log2 e, -inf among
// them where ``out``.  ``read`` is called when all has been read, before the last of it is added up.
template <int W, typename F>
__device__ __forceinline__ float weigh_tile(uint32_t t_s, const float* __restrict__ nl, bool out, int cols, const WeighSpan& x, float c2, F read) {
  float2 sum[W / 16];
#pragma unroll
  for (int i = 0; i < W / 16; ++i) sum[i] = make_float2(0.f, 0.f);
  const float2 c = make_float2(c2, c2);
#pragma unroll 1
  for (int c0 = 0; c0 < cols; c0 += W) {
    uint32_t s[W / 32][32];
#pragma unroll
    for (int y = 0; y < W / 32; ++y) tmem_ld32(t_s + c0 + 32 * y, s[y]);
    tmem_wait_ld();
    if (c0 + W >= cols) {
      tc_fence_before();
      __syncwarp();
      read();
    }
    if (c0 + W <= x.lo_min || c0 >= x.hi) continue;
    if (out) {                                                // (a pass of its own: 32 single tokens 62 us, a test of each weight 64)
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (nl[c0 + i] == -INFINITY) s[i / 32][i % 32] = 0u;
    }
    if (c0 < x.lo_max || c0 + W > x.hi) {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float e = fast_exp2(fmaf(__uint_as_float(s[i / 32][i % 32]), c2, nl[c0 + i]));
        sum[i % (W / 16)].x += c0 + i >= x.lo && c0 + i < x.hi ? e : 0.f;
      }
      __syncwarp();                                           // (tensor memory is read by the whole warp at once)
    } else {
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const float4 n = *reinterpret_cast<const float4*>(nl + c0 + i);
        const uint32_t* v4 = &s[i / 32][i % 32];
        const float2 u = ffma2(make_float2(__uint_as_float(v4[0]), __uint_as_float(v4[1])), c, make_float2(n.x, n.y));
        const float2 v = ffma2(make_float2(__uint_as_float(v4[2]), __uint_as_float(v4[3])), c, make_float2(n.z, n.w));
        sum[i / 2 % (W / 16)] = fadd2(sum[i / 2 % (W / 16)], make_float2(fast_exp2(u.x), fast_exp2(u.y)));
        sum[(i / 2 + 1) % (W / 16)] = fadd2(sum[(i / 2 + 1) % (W / 16)], make_float2(fast_exp2(v.x), fast_exp2(v.y)));
      }
    }
  }
#pragma unroll
  for (int i = W / 32; i >= 1; i /= 2)
#pragma unroll
    for (int y = 0; y < i; ++y) sum[y] = fadd2(sum[y], sum[y + i]);
  return sum[0].x + sum[0].y;
}

template <int D>
__global__ void __launch_bounds__(WeighCfg<D>::FEW_THREADS, 1) weigh_few_kernel(const __grid_constant__ WeighParams p) {
  using C = WeighCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const WeighShared<D> m(align_smem_1k(smem_raw));
  volatile int* abort_flag = m.abort_flag;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (warp == 0) {
    if (lane == 0) m.init(2, 8);                              // (a slot of K: a pair of tiles)
    if (lane < 2) tma_prefetch_desc(lane ? &p.tq : &p.tk);
    // this CTA's share of the key pairs
    int b;
    long long before = 0;
    const int c = blockIdx.x;
    const Q4Share sh = paged_share(p.n_seqs, gridDim.x, [&](int i, bool first) {
      return static_cast<long long>(weigh_pairs(paged_seq(p.cu, p.seqlens, i, p.total, p.max_q, p.max_k, c == 0 && first, 601))) * p.cache.H_kv;
    }, [&](const Q4Share& y) { return c < y.n && y.total > 0 ? y.begin(c) : -1LL; }, -1, &b, &before);
    if (lane == 0) {
      m.start[0] = b;
      m.start[1] = b < 0 ? 0 : static_cast<int>(sh.begin(c) - before);
      m.start[2] = b < 0 ? 0 : static_cast<int>(sh.begin(c + 1) - sh.begin(c));
    }
  } else if (warp == 1) {
    tmem_alloc(m.tmem_slot, 512);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *m.tmem_slot;

  WeighWalk walk{p, m.start[0], m.start[1], m.start[2], {}, 0};
  if (walk.left > 0) {
    walk.seq = paged_seq(p.cu, p.seqlens, walk.b, p.total, p.max_q, p.max_k, false, 0);
    walk.pairs = weigh_pairs(walk.seq);
  }
  WeighStretch x;
  bool ok = true;
  int kc = 0, qc = 0;                                         // key pairs, stretches so far

  if (warp == 0) {
    // ---------------------------------------------------------------- copies of K
    PagedStream<D> keys(p.cache);
    while (ok && walk.next(x)) {
      keys.begin(p.cache, x.b, x.kt0 * 256, x.seq.len);
      for (int kt = x.kt0; ok && kt < x.kt1; ++kt, ++kc) {
        const int s = kc % C::PAIRS, u = kc / C::PAIRS;
        if (u > 0 && !(ok = mbar_wait_warp(&m.k_empty[s], (u - 1) & 1, abort_flag, 610))) break;
        uint8_t* dst = m.k + s * 2 * C::TILE;
        // (a tile behind the last key brings nothing)
#pragma unroll 1
        for (int i = 0; i < 2; ++i) keys.load(p.cache, &p.tk, dst + i * C::TILE, &m.k_full[s], x.hkv, keys.next(p.cache, 602));
      }
    }
    for (int i = max(0, kc - C::PAIRS); ok && i < kc; ++i) ok = mbar_wait_warp(&m.k_empty[i % C::PAIRS], (i / C::PAIRS) & 1, abort_flag, 611);
    if (!ok)
      for (int i = max(0, kc - C::PAIRS); i < kc; ++i) mbar_wait_warp(&m.k_full[i % C::PAIRS], (i / C::PAIRS) & 1, nullptr, 612);
  } else if (warp == 2) {
    // ---------------------------------------------------------------- copies of Q
    while (ok && walk.next(x))
      for (int r = 0; r < x.tiles; ++r, ++qc) {
        const int s = qc % C::NQ, u = qc / C::NQ;
        if (u > 0 && !(ok = mbar_wait_warp(&m.q_empty[s], (u - 1) & 1, abort_flag, 613))) break;
        if (lane == 0) weigh_load_q<D>(p, m, s, x.hkv, x.seq.first + r * p.tokens);
        __syncwarp();
      }
    for (int i = max(0, qc - C::NQ); ok && i < qc; ++i) ok = mbar_wait_warp(&m.q_empty[i % C::NQ], (i / C::NQ) & 1, abort_flag, 614);
    if (!ok)
      for (int i = max(0, qc - C::NQ); i < qc; ++i) mbar_wait_warp(&m.q_full[i % C::NQ], (i / C::NQ) & 1, nullptr, 615);
  } else if (warp == 3) {
    // ---------------------------------------------------------------- lse
    WeighLse lse(p);
    while (ok && walk.next(x))
      for (int r = 0; r < x.tiles; ++r, ++qc) {
        const int s = qc % C::NQ, u = qc / C::NQ;
        lse.ask(x.seq, x.hkv, r, lse.e);
        if (u > 0 && !(ok = mbar_wait_warp(&m.l_empty[s], (u - 1) & 1, abort_flag, 616))) break;
        lse.write(x.seq.nq - r * p.tokens, m.lse + s * 128, m.out + s);
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.l_full[s]);
      }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- products
    const uint32_t idesc = idesc_bf16_f32(128, (p.rows + 15) / 16 * 16, 0, 0);
    const uint64_t dk0 = smem_desc_sw128(smem_u32(m.k), 0, 1024);
    const uint64_t dq0 = smem_desc_sw128(smem_u32(m.q), 0, 1024);
    int sc = 0;                                               // products of each tile of a pair so far
    while (ok && walk.next(x)) {
      for (int r = 0; ok && r < x.tiles; ++r) ok = mbar_wait_warp(&m.q_full[(qc + r) % C::NQ], ((qc + r) / C::NQ) & 1, abort_flag, 621);
      for (int kt = x.kt0; ok && kt < x.kt1; ++kt, ++kc) {
        ok = mbar_wait_warp(&m.k_full[kc % C::PAIRS], (kc / C::PAIRS) & 1, abort_flag, 620);
        for (int r = 0; ok && r < x.tiles; ++r, ++sc) {
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            const int buf = 2 * a + (sc & 1);
            if (ok && sc >= 2) ok = mbar_wait_warp(&m.s_empty[buf], ((sc >> 1) - 1) & 1, abort_flag, 622);
            if (!ok) break;
            tc_fence_after();
            weigh_product<D>(tbase + buf * 128, desc_advance(dk0, ((kc % C::PAIRS) * 2 + a) * C::TILE),
                             desc_advance(dq0, ((qc + r) % C::NQ) * C::TILE), idesc, &m.s_full[buf]);
          }
        }
        if (ok) umma_commit_w(&m.k_empty[kc % C::PAIRS]);
      }
      for (int r = 0; r < x.tiles; ++r, ++qc)
        if (ok) umma_commit_w(&m.q_empty[qc % C::NQ]);
    }
  } else {
    // ---------------------------------------------------------------- sums
    const int a = (warp - 4) >> 2, sub = warp & 3;
    const uint32_t t_lane = tbase + (static_cast<uint32_t>(sub * 32) << 16);
    const int cols = (p.rows + 31) / 32 * 32;
    int sc = 0;
    while (ok && walk.next(x)) {
      const int weighed = p.weighed ? __ldg(p.weighed + x.b) : x.seq.base();
      uint32_t out = 0;                                       // by row tile
      for (int r = 0; ok && r < x.tiles; ++r) {
        ok = mbar_wait_warp(&m.l_full[(qc + r) % C::NQ], ((qc + r) / C::NQ) & 1, abort_flag, 630);
        out |= static_cast<uint32_t>(m.out[(qc + r) % C::NQ]) << r;
      }
      for (int kt = x.kt0; ok && kt < x.kt1; ++kt) {
        const int key = kt * 256 + a * 128 + sub * 32 + lane;
        float* at = key < x.seq.len ? weigh_place(p, x.b, x.hkv, key) : nullptr;
        const float old = at && key < weighed ? *at * p.decay : 0.f;
        float sum = 0.f;
        for (int r = 0; r < x.tiles; ++r, ++sc) {
          const int buf = 2 * a + (sc & 1);
          if (!(ok = mbar_wait_warp(&m.s_full[buf], (sc >> 1) & 1, abort_flag, 631))) break;
          tc_fence_after();
          const int r0 = r * p.rows;
          const float* nl = m.lse + ((qc + r) % C::NQ) * 128;
          const WeighSpan span(p, x.seq, key, r0, min(p.rows, x.seq.nq * p.G - r0));
          auto read = [&] {
            if (lane == 0) mbar_arrive(&m.s_empty[buf]);
          };
          // (64 columns at a time where there are as many: 16 x 64 tokens over 8000 87 us with 32, 82 with 64, 140 with 128;
          // 32 single tokens, four columns, 62 with 32 and 68 with 64)
          sum += cols > 32 ? weigh_tile<64>(t_lane + buf * 128, nl, out >> r & 1u, cols, span, p.c2, read) 
                            : weigh_tile<32>(t_lane + buf * 128, nl, out >> r & 1u, cols, span, p.c2, read);
        }
        if (at && ok) *at = old + sum;
      }
      __syncwarp();
      for (int r = 0; r < x.tiles; ++r, ++qc)
        if (lane == 0 && ok) mbar_arrive(&m.l_empty[qc % C::NQ]);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <int D>
__global__ void __launch_bounds__(WeighCfg<D>::MANY_THREADS, 1) weigh_many_kernel(const __grid_constant__ WeighParams p) {
  using C = WeighCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const WeighShared<D> m(align_smem_1k(smem_raw));
  volatile int* abort_flag = m.abort_flag;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (warp == 0) {
    if (lane == 0) m.init(1, 16);
    if (lane < 2) tma_prefetch_desc(lane ? &p.tq : &p.tk);
    int b, hkv = 0, kt = 0;
    long long before = 0, u = 0, left = 0;
    const int c = blockIdx.x;
    const Q4Share sh = weigh_share(p, gridDim.x, c == 0, [&](const Q4Share& y) { return c < y.n && y.total > 0 ? y.begin(c) : -1LL; }, &b, &before);
    if (b >= 0) {
      u = sh.begin(c) - before;
      left = sh.begin(c + 1) - sh.begin(c);
      weigh_piece_of(WeighPieces(p, paged_seq(p.cu, p.seqlens, b, p.total, p.max_q, p.max_k, false, 0)), &u, &hkv, &kt);
    }
    if (lane == 0) {
      m.start[0] = b;
      m.start[1] = hkv;
      m.start[2] = kt;
      m.start[3] = static_cast<int>(u);
      m.start[4] = static_cast<int>(left);                    // (below 2^31: launch)
    }
  } else if (warp == 1) {
    tmem_alloc(m.tmem_slot, 512);
  }
  pdl_launch_dependents();
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *m.tmem_slot;

  WeighParts walk{p, m.start[0], m.start[1], m.start[2], m.start[3], m.start[4]};
  WeighPiece x;
  bool ok = true;
  int kc = 0, qc = 0;                                         // pieces, row tiles so far
  constexpr int SETS = C::NK / 4;                             // pieces of K in flight

  if (warp == 0) {
    // ---------------------------------------------------------------- copies of K: slot 4 (piece % SETS) + tile
    PagedStream<D> keys(p.cache);
    uint32_t used = 0;                                        // slots that were filled before
    uint32_t parity = 0;                                      // of the next wait for them
    while (ok && walk.next(x)) {
      const int n = walk.tiles(x);
      keys.begin(p.cache, x.b, x.kt * kWeighKeys, x.seq.len);
      for (int a = 0; ok && a < n; ++a) {
        const int s = 4 * (kc % SETS) + a;
        if (used >> s & 1u) {
          if (!(ok = mbar_wait_warp(&m.k_empty[s], parity >> s & 1u, abort_flag, 610))) break;
          parity ^= 1u << s;
        }
        used |= 1u << s;
        keys.load(p.cache, &p.tk, m.k + s * C::TILE, &m.k_full[s], x.hkv, keys.next(p.cache, 602));
      }
      ++kc;
    }
    for (int s = 0; ok && s < C::NK; ++s)
      if (used >> s & 1u) ok = mbar_wait_warp(&m.k_empty[s], parity >> s & 1u, abort_flag, 611);
    if (!ok)
      for (int s = 0; s < C::NK; ++s)
        if (used >> s & 1u) mbar_wait_warp(&m.k_full[s], parity >> s & 1u, nullptr, 612);
  } else if (warp == 2) {
    // ---------------------------------------------------------------- copies of Q
    while (ok && walk.next(x)) {
      for (int qt = x.q0; ok && qt < x.q1; ++qt, ++qc) {
        const int s = qc % C::NQ, u = qc / C::NQ;
        if (u > 0 && !(ok = mbar_wait_warp(&m.q_empty[s], (u - 1) & 1, abort_flag, 613))) break;
        if (lane == 0) weigh_load_q<D>(p, m, s, x.hkv, x.seq.first + qt * p.tokens);
        __syncwarp();
      }
    }
    for (int i = max(0, qc - C::NQ); ok && i < qc; ++i) ok = mbar_wait_warp(&m.q_empty[i % C::NQ], (i / C::NQ) & 1, abort_flag, 614);
    if (!ok)
      for (int i = max(0, qc - C::NQ); i < qc; ++i) mbar_wait_warp(&m.q_full[i % C::NQ], (i / C::NQ) & 1, nullptr, 615);
  } else if (warp == 3) {
    // ---------------------------------------------------------------- lse
    WeighLse lse(p);
    while (ok && walk.next(x)) {
      lse.ask(x.seq, x.hkv, x.q0, lse.e);
      for (int qt = x.q0; ok && qt < x.q1; ++qt, ++qc) {
        const int s = qc % C::NQ, u = qc / C::NQ;
        float next[4] = {0.f, 0.f, 0.f, 0.f};
        if (qt + 1 < x.q1) lse.ask(x.seq, x.hkv, qt + 1, next);
        if (u > 0 && !(ok = mbar_wait_warp(&m.l_empty[s], (u - 1) & 1, abort_flag, 616))) break;
        lse.write(x.seq.nq - qt * p.tokens, m.lse + s * 128, m.out + s);
#pragma unroll
        for (int i = 0; i < 4; ++i) lse.e[i] = next[i];
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.l_full[s]);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- products
    const uint32_t idesc = idesc_bf16_f32(128, (p.rows + 15) / 16 * 16, 0, 0);
    const uint64_t dk0 = smem_desc_sw128(smem_u32(m.k), 0, 1024);
    const uint64_t dq0 = smem_desc_sw128(smem_u32(m.q), 0, 1024);
    // After a failed wait the warp goes on joining every hand-back, issuing nothing.
    uint32_t k_parity = 0, s_used = 0;                        // by slot of K, by S buffer
    while (walk.next(x)) {
      const int n = walk.tiles(x), set = 4 * (kc % SETS);
      for (int qt = x.q0; qt < x.q1; ++qt, ++qc) {
        ok = ok && mbar_wait_warp(&m.q_full[qc % C::NQ], (qc / C::NQ) & 1, abort_flag, 621);
        const uint64_t dq = desc_advance(dq0, (qc % C::NQ) * C::TILE);
        if (qt == x.q0)
          for (int a = 0; a < n; ++a) {
            ok = ok && mbar_wait_warp(&m.k_full[set + a], k_parity >> (set + a) & 1u, abort_flag, 620);
            k_parity ^= 1u << (set + a);
          }
        const int seen = walk.seen(x, qt, n);
        const uint64_t dk = desc_advance(dk0, set * C::TILE);
        // (unrolled: what the warp does between two products has to fit into the few that the tensor core has queued)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          if (a >= seen) break;
          if (s_used & (1u << a)) named_bar_sync(C::BAR_S + a, C::BAR_S_THREADS);
          s_used |= 1u << a;
          if (ok) {
            tc_fence_after();
            weigh_product<D>(tbase + a * 128, desc_advance(dk, a * C::TILE), dq, idesc, &m.s_full[a]);
            if (qt + 1 == x.q1) umma_commit_w(&m.k_empty[set + a]);   // (the last row tile sees all that any sees)
          }
        }
        if (ok) umma_commit_w(&m.q_empty[qc % C::NQ]);
      }
      for (int a = walk.seen(x, x.q1 - 1, n); ok && a < n; ++a) umma_commit_w(&m.k_empty[set + a]);
      ++kc;
    }
    for (int a = 0; a < 4; ++a) {
      __syncwarp();
      if (s_used >> a & 1u) named_bar_sync(C::BAR_S + a, C::BAR_S_THREADS);
    }
  } else {
    // ---------------------------------------------------------------- sums, a warpgroup a key tile
    // (S is given back by a named barrier, which costs the issuing warp some 30 clocks where an mbarrier costs it 175)
    const int a = (warp - 4) >> 2, sub = warp & 3;
    const uint32_t t_s = tbase + (static_cast<uint32_t>(sub * 32) << 16) + a * 128;
    const int cols = (p.rows + 31) / 32 * 32;
    int sc = 0;                                               // products so far
    while (walk.next(x)) {
      const int key = x.kt * kWeighKeys + a * 128 + sub * 32 + lane, tiles = walk.tiles(x);
      float sum = 0.f;
      for (int qt = x.q0; qt < x.q1; ++qt, ++qc) {
        if (a < walk.seen(x, qt, tiles)) {
          // (both at once: most of the time neither is waited for)
          uint64_t* bars[2] = {&m.l_full[qc % C::NQ], &m.s_full[a]};
          const uint32_t there = mbar_try_wait(smem_u32(bars[0]), (qc / C::NQ) & 1), done = mbar_try_wait(smem_u32(bars[1]), sc & 1);
          if (!__all_sync(0xffffffffu, there && done))
            ok = ok && mbar_wait_warp(bars[0], (qc / C::NQ) & 1, abort_flag, 630) && mbar_wait_warp(bars[1], sc & 1, abort_flag, 631);
          ++sc;
          if (!ok) {                                          // after an abort: keep joining, blocking
            __syncwarp();
            named_bar_sync(C::BAR_S + a, C::BAR_S_THREADS);
            continue;
          }
          tc_fence_after();
          const int r0 = qt * p.tokens * p.G, rows = min(p.tokens, x.seq.nq - qt * p.tokens) * p.G;
          sum += weigh_tile<32>(t_s, m.lse + (qc % C::NQ) * 128, m.out[qc % C::NQ], cols, WeighSpan(p, x.seq, key, r0, rows), p.c2,
                            [&] { named_bar_arrive(C::BAR_S + a, C::BAR_S_THREADS); });
        } else {
          ok = ok && mbar_wait_warp(&m.l_full[qc % C::NQ], (qc / C::NQ) & 1, abort_flag, 632);
        }
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&m.l_empty[qc % C::NQ]);   // (once for each time that it was there)
      }
      if (!ok || a >= tiles || key >= x.seq.len) continue;
      if (x.slot >= 0) {
        p.part[static_cast<size_t>(x.slot) * kWeighKeys + key - x.kt * kWeighKeys] = sum;
      } else {
        float* at = weigh_place(p, x.b, x.hkv, key);
        const int weighed = p.weighed ? __ldg(p.weighed + x.b) : x.seq.base();
        if (at) *at = (key < weighed ? *at * p.decay : 0.f) + sum;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// Adds up the sums of a piece that a bound between shares cuts, if bound i + 1 is the first within it; thread = key.
__global__ void __launch_bounds__(kWeighKeys) weigh_join_kernel(const __grid_constant__ WeighParams p, int ctas) {
  __shared__ int found[4];                                    // sequence, key head, piece, CTAs
  __shared__ uint32_t has[8];                                 // by CTA of the piece: whether it has any row tiles
  const int i = blockIdx.x, lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    int b;
    long long before = 0;
    const Q4Share sh = weigh_share(p, ctas, false, [&](const Q4Share& y) { return i + 1 < y.n ? y.begin(i + 1) : -1LL; }, &b, &before);
    int n = 0, hkv = 0, kt = 0;
    if (b >= 0) {
      const WeighPieces y(p, paged_seq(p.cu, p.seqlens, b, p.total, p.max_q, p.max_k, false, 0));
      long long k = sh.begin(i + 1) - before;
      weigh_piece_of(y, &k, &hkv, &kt);
      // the bound lies k units into the piece: within it, and the first that does
      const long long u0 = sh.begin(i + 1) - k;
      if (k > 0 && sh.begin(i) <= u0) {
        const int units = y.units(kt);
        n = sh.owner(u0 + units - 1) - i + 1;
        for (int base = 0; base < n; base += 32) {
          const int c = i + base + lane;
          bool some = false;
          if (base + lane < n) {
            const int k0 = static_cast<int>(max(0LL, sh.begin(c) - u0)), k1 = static_cast<int>(min(static_cast<long long>(units), sh.begin(c + 1) - u0));
            some = y.row_tile(kt, k0) < y.row_tile(kt, k1);
          }
          const uint32_t bits = __ballot_sync(0xffffffffu, some);
          if (lane == 0) has[base / 32] = bits;
        }
      }
    }
    if (lane == 0) {
      found[0] = b; found[1] = hkv; found[2] = kt; found[3] = n;
    }
  }
  __syncthreads();
  const int n = found[3], b = found[0];
  if (n > 0) {
    const PagedSeq s = paged_seq(p.cu, p.seqlens, b, p.total, p.max_q, p.max_k, false, 0);
    const int key = found[2] * kWeighKeys + threadIdx.x;
    const int weighed = p.weighed ? __ldg(p.weighed + b) : s.base();
    float* at = key < s.len ? weigh_place(p, b, found[1], key) : nullptr;
    pdl_wait();
    if (!at) return;
    const float old = key < weighed ? *at * p.decay : 0.f;
    float drawn = 0.f;
    for (int c = 0; c < n; ++c)                               // (the first CTA's second place, the others' first one)
      if (has[c >> 5] >> (c & 31) & 1u) drawn += p.part[static_cast<size_t>(2 * (i + c) + (c == 0 ? 1 : 0)) * kWeighKeys + threadIdx.x];
    *at = old + drawn;
  } else {
    pdl_wait();
  }
}

template <int D>
static cudaError_t launch_weigh_d(const WeighArgs& a, cudaStream_t stream) {
  using C = WeighCfg<D>;
  WeighParams p{};
  const int piece = paged_piece(a.block_size);
  const uint64_t rows = static_cast<uint64_t>(a.num_blocks) * a.block_size;
  p.G = a.H / a.H_kv;
  p.tokens = weigh_tokens(a.H, a.H_kv, a.max_q);
  p.rows = p.tokens * p.G;
  if (!make_map_bf16_tok(&p.tk, a.k_cache, D, a.H_kv, rows, 64, piece) ||
      !make_map_bf16_group(&p.tq, a.q, D, p.G, a.H_kv, a.total, 64, p.G, p.tokens))
    return cudaErrorInvalidValue;
  p.cache = paged_cache(a.block_table, a.H_kv, a.num_blocks, a.block_size, a.max_blocks);
  p.lse = a.lse; p.weights = a.weights; p.part = a.part; p.cu = a.cu; p.seqlens = a.seqlens; p.weighed = a.weighed;
  p.n_seqs = a.n_seqs; p.H = a.H; p.total = a.total; p.max_q = a.max_q; p.max_k = a.max_k;
  p.c2 = a.scale * 1.4426950408889634f; p.decay = a.decay;
  const bool few = weigh_few(p.tokens, a.max_q);
  static int few_done[64] = {0}, many_done[64] = {0};
  cudaError_t e = few ? ensure_smem_attr(weigh_few_kernel<D>, C::SMEM_BYTES, few_done) : ensure_smem_attr(weigh_many_kernel<D>, C::SMEM_BYTES, many_done);
  if (e != cudaSuccess) return e;
  const long long heads = static_cast<long long>(a.n_seqs) * a.H_kv;
  // (of no keys one CTA: it checks lengths and boundaries)
  const int pieces = few ? (a.max_k + 255) / 256 : (a.max_k + kWeighKeys - 1) / kWeighKeys;
  const long long items = heads * max(1, pieces) * (few ? 1 : (a.max_q + p.tokens - 1) / p.tokens);
  const long long grid = min(static_cast<long long>(min(paged_sm_count(), kWeighMaxCtas)), items);
  const unsigned threads = few ? C::FEW_THREADS : C::MANY_THREADS;
  log_launch(few ? "weigh_few_kernel<D>" : "weigh_many_kernel<D>", static_cast<unsigned long long>(grid), threads, static_cast<unsigned long long>(C::SMEM_BYTES));
  if (few) weigh_few_kernel<D><<<static_cast<unsigned>(grid), threads, C::SMEM_BYTES, stream>>>(p);
  else weigh_many_kernel<D><<<static_cast<unsigned>(grid), threads, C::SMEM_BYTES, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || few || grid == 1) return e;
  log_launch("weigh_join_kernel", static_cast<unsigned long long>(grid - 1), kWeighKeys, 0ull);
  return launch_join(weigh_join_kernel, static_cast<unsigned>(grid - 1), kWeighKeys, stream, p, static_cast<int>(grid));
}

cudaError_t launch_weigh(const WeighArgs& a, cudaStream_t stream) {
  return a.d == 64 ? launch_weigh_d<64>(a, stream) : launch_weigh_d<128>(a, stream);
}

}  // namespace fa

FA_DEFINE_STATUS_FETCH(status_fetch_weigh)
