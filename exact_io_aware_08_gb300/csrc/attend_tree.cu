// Attention of a step's query tokens over the bf16 paged cache: any number of query heads a key head, one
// token a sequence or many, and a mask among the step's own tokens (trees of drafted tokens).
//
// Mathematics.  The rows of a key head are its query heads times the step's tokens, (token, head) by token.
// Row (i, h) sees every token in front of the step's, and of these the ones whose bits are set in tree[i]
// (without a tree those up to i).  S = Q K^T, w = 2^(c S - m) with c = scale log2 e, l = sum w, O = sum w V / l
// with the online softmax; m is at most 8 below the running maximum.  Weights are rounded to bf16 for the
// product with V (the tensor core takes both operands in one type, and V has bf16's range): by 2^-8 of
// themselves.  O is divided by the sum of the rounded weights, so that a row which one key dominates is that
// key's value; lse comes from the unrounded sum.  Both sums are fp32.
//
// What bounds it.  4 d flops a (row, key) and 4 d bytes a key of a key head: up to some 278 rows the reading
// of the cache, above it the tensor core.
//
// Layout.  A CTA an SM takes NT tiles of up to 128 rows of one key head (whole tokens, so that TMA brings them), and
// runs over keys 128 at a time:
//   warp 0       copies K and V tiles by TMA into one ring, in the order in which they are used.
//   warp 1       issues the products (the whole warp converged, one elected lane): S = Q K^T from shared
//                memory, O += P V with P from tensor memory.
//   warp 2       joins the hand-off of P once V is there.
//   warp 3       brings Q in, the next item's as soon as the last S of one is done.
//   warps 4-11   softmax.  NT = 2: thread = row, a warpgroup a row tile.  NT = 1: two threads a row, 64 keys each,
//                which exchange their maxima in tensor memory.  They write O out, or states, a state's rows side by
//                side, and clean V's tile where some row does not see all of it: 0 * NaN is NaN.
// Two S buffers are in flight: of the two row tiles (NT = 2, more than 128 rows), or of two key tiles in a
// row (NT = 1).
//
// Where one row block holds all rows of a sequence and key head, each CTA gets an equal share of all key steps,
// whatever the sequences' lengths, and what is cut is joined from states (Q4Share).  With more row blocks a
// CTA takes whole ones, all row blocks of a key head side by side so that its keys are read from memory once, as
// many rounds as all CTAs can; the key steps of the rest are shared out equally (4 x 512 tokens over 16384 keys, 256 row
// blocks: 451 us in two rounds).
//
// Measured, d = 128, caches flushed before each call: 16 single tokens over 32768 keys, 32 heads over 4, 180 us (6.0 TB/s;
// the fastest CTA has its equal share done after 142); 16 trees of 1 to 60 tokens over 500 to 8188, 32 over 8, 84; 4 x 512
// tokens over 16384 407 (1.33 PFLOP/s; not flushed 388); one tree of 8 over 1000 12.3.
//
// A sequence of more than two row tiles beside short ones: row blocks are counted for the longest, and the only one that a
// single token has falls to the same few CTAs and is not cut (63 single tokens and 512 in one call, all over 8192 keys: 1.4
// ms, the single tokens alone 0.35; 64 single tokens with max_seqlen_q of 512: 1.3).  Two calls are the faster way.
//
// Short calls are bound by latencies, of fetching instructions among them (a first pass over unrolled code that
// streamed caches have driven out of L2 takes microseconds): the rarer paths are loops.
#include "fa_kernels.h"
#include "paged_tile.cuh"

namespace fa {

template <int D, int NT>
struct TreeCfg {
  static constexpr int BN = kPagedTile;
  static constexpr int CH = D / 64;
  static constexpr int CHUNK = 128 * 128;
  static constexpr int TILE = 128 * D * 2;
  static constexpr int NST = D == 128 ? (NT == 1 ? 6 : 5) : 11;   // K and V tiles of the ring
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = NT * TILE;
  static constexpr int OFF_BAR = OFF_KV + NST * TILE;
  // full[NST], empty[NST], q_full, q_empty, s_full[2], pv_done[2]; then the TMEM slot, abort flag, start[3], spoilt[4]
  static constexpr int NBAR = 2 * NST + 6;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int OFF_TAIL = OFF_MISC + 48;              // kTreeMaxCtas + 1 running counts (rests)
  static constexpr int SMEM_BYTES = OFF_TAIL + (NT == 2 ? (kTreeMaxCtas + 1) * 4 : 0) + 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget (227 KB per CTA)");
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t T_S = 0, T_O = 256, T_X = 384;    // T_X: exchanged maxima and sums (NT = 1)
  static constexpr int THREADS = 384;
  static constexpr int STATE = 32 * (D + 3);                  // of 32 rows: each column, reference, sum, rounded sum
  // named barriers: start, hand-off of P by S buffer, pairs of warps (NT = 1)
  static constexpr uint32_t BAR_START = 1, BAR_P = 2, BAR_PAIR = 4;
  static constexpr uint32_t BAR_P_THREADS = (NT == 1 ? 256 : 128) + 32 + 32;
};
constexpr float kTreeRescale = 8.f;

struct TreeParams {
  CUtensorMap tk, tv, tq;
  PagedCache cache;
  const uint16_t* v;
  uint16_t* o;
  float *lse, *part;
  const int *tree, *cu, *seqlens;
  // A key head's G query heads are taken ``group`` at a time (all of them where a tile holds them): heads of
  // that kind are called key heads below, ``heads`` of them, ``per_kv`` to a key head of the cache.
  int group, heads, per_kv, tokens;                           // tokens of a row tile
  int words, n_seqs, H, total, max_q, max_k;
  int shares, whole;                                          // equal shares of key steps (of whole row blocks or not)
  int leave;                                                  // what a row block costs beside its steps
  int row_blocks, rounds, rest, state_rows;                   // else: rounds of whole row blocks, and the rest in shares
  float c2;
};

// One stretch of work: row block rb of a key head of a sequence over keys [key0, key_end).
struct TreeItem {
  int b, head, rb, key0, key_end, slot;                       // slot: -1 results, else the state's place
  PagedSeq seq;
};

// Units of a (sequence, key head) in equal shares: its key steps, and in front of them what leaving one row block for
// the next costs, in steps.
__device__ __forceinline__ int tree_steps(const PagedSeq& s) { return (s.len + kPagedTile - 1) / kPagedTile; }
__device__ __forceinline__ int tree_units(const TreeParams& p, const PagedSeq& s) { return s.nq ? p.leave + tree_steps(s) : 0; }

// Row block ``index`` of those that are taken whole or rest: (sequence, key head) pairs, and within one the last rows,
// which see the most, first.
template <int NT>
struct TreeBlock {
  int b, head, rb;
  __device__ __forceinline__ TreeBlock(const TreeParams& p, int index) {
    rb = p.row_blocks - 1 - index % p.row_blocks;
    const int w = index / p.row_blocks;
    head = w % p.heads;
    b = w / p.heads;
  }
  __device__ __forceinline__ static int seen(const TreeParams& p, const PagedSeq& s, int token) {
    return p.tree ? s.len : s.base() + min(token, s.nq - 1) + 1;
  }
  // Its keys (0: no rows).
  __device__ __forceinline__ int keys(const TreeParams& p, const PagedSeq& s) const {
    return rb * NT * p.tokens >= s.nq ? 0 : seen(p, s, (rb + 1) * NT * p.tokens - 1);
  }
};

// By a whole warp: running counts of the rest's key steps, counts[0] = 0 to counts[p.rest].
__device__ __forceinline__ void tree_rest(const TreeParams& p, int ctas, bool report, int* counts) {
  const int lane = threadIdx.x & 31;
  int sum = 0;
  for (int base = 0; base < p.rest; base += 32) {
    int steps = 0;
    if (base + lane < p.rest) {
      const TreeBlock<2> x(p, p.rounds * ctas + base + lane);
      const PagedSeq s = paged_seq(p.cu, p.seqlens, x.b, p.total, p.max_q, p.max_k, report, 503);
      steps = (x.keys(p, s) + kPagedTile - 1) / kPagedTile;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, steps, o);
      if (lane >= o) steps += y;
    }
    if (base + lane < p.rest) counts[base + lane + 1] = sum + steps;
    sum += __shfl_sync(0xffffffffu, steps, 31);
  }
  if (lane == 0) counts[0] = 0;
  __syncwarp();
}

// Their place in the workspace, for the join: in front of the states.
__device__ __forceinline__ int* tree_counts(const TreeParams& p) { return reinterpret_cast<int*>(p.part) - (kTreeMaxCtas + 8); }

// The rest's shares: CTA c's first unit of ``units``, and the CTA that has unit u (no share is empty: of few units
// each of the first CTAs has one).
__device__ __forceinline__ int rest_begin(int units, int c, int ctas) {
  const int n = min(ctas, units);
  return c >= n ? units : static_cast<int>(static_cast<long long>(units) * c / n);
}
__device__ __forceinline__ int rest_owner(int units, int u, int ctas) {
  return static_cast<int>((static_cast<long long>(u + 1) * min(ctas, units) - 1) / units);
}

template <int NT>
struct TreeWalk {
  const TreeParams& p;
  const int* counts;                                          // (rests)
  int b, off, left;                                           // shares: sequence, unit in it, units left
  int round;                                                  // else: round; of the rest row block b, first unit off
  PagedSeq seq;
  int units;                                                  // of a key head of it

  // Tokens up to ``token`` of the sequence see keys below this.
  __device__ __forceinline__ static int seen(const TreeParams& p, const PagedSeq& s, int token) { return TreeBlock<NT>::seen(p, s, token); }

  __device__ __forceinline__ void block(TreeItem& x, int index) const {
    const TreeBlock<NT> y(p, index);
    x.b = y.b;
    x.head = y.head;
    x.rb = y.rb;
    x.seq = paged_seq(p.cu, p.seqlens, x.b, p.total, p.max_q, p.max_k, x.rb == 0 && x.head == 0 && threadIdx.x == 0, 500);
    x.key0 = 0;
    x.key_end = y.keys(p, x.seq);
    x.slot = -1;
  }

  // The share: whose first unit is unit ``u`` of sequence ``at``.
  __device__ __forceinline__ void begin(int at, int u, int n) {
    b = at;
    off = u;
    left = n;
    if (left <= 0) return;
    seq = paged_seq(p.cu, p.seqlens, b, p.total, p.max_q, p.max_k, false, 0);
    units = tree_units(p, seq);
    if (p.whole) {                                            // the row blocks that begin in it
      const int behind = off % units, skip = behind ? units - behind : 0;
      off += skip;
      left -= skip;
    }
  }

  __device__ __forceinline__ bool next(TreeItem& x) {
    if (NT == 2 && !p.shares) {
      const int ctas = gridDim.x;
      for (; round < p.rounds; ++round) {
        block(x, pers_item(round, ctas));
        if (x.key_end == 0) continue;
        ++round;
        return true;
      }
      if (round == p.rounds) {                                // the share of the rest
        ++round;
        off = rest_begin(counts[p.rest], blockIdx.x, ctas);
        left = rest_begin(counts[p.rest], blockIdx.x + 1, ctas) - off;
        b = 0;
      }
      if (left <= 0) return false;
      while (counts[b + 1] <= off) ++b;
      block(x, p.rounds * ctas + b);
      const int step0 = off - counts[b], all = counts[b + 1] - counts[b], n = min(left, all - step0);
      x.key0 = step0 * kPagedTile;
      x.key_end = min(x.key_end, x.key0 + n * kPagedTile);
      x.slot = n == all ? -1 : 2 * static_cast<int>(blockIdx.x) + (step0 == 0 ? 1 : 0);
      off += n;
      left -= n;
      return true;
    }
    while (left > 0) {
      while (off >= units * p.heads) {                        // (a sequence with work follows: left > 0)
        if (++b >= p.n_seqs) return false;
        off = 0;
        seq = paged_seq(p.cu, p.seqlens, b, p.total, p.max_q, p.max_k, false, 0);
        units = tree_units(p, seq);
      }
      x.head = off / units;
      const int u0 = off - x.head * units, n = p.whole ? units : min(left, units - u0);
      off += n;
      left -= n;
      const int step0 = max(0, u0 - p.leave), step1 = u0 + n - p.leave;
      if (step1 <= step0) continue;
      x.b = b;
      x.seq = seq;
      x.rb = 0;
      x.key0 = step0 * kPagedTile;
      x.key_end = min(step1 * kPagedTile, seq.len);
      x.slot = step1 - step0 == units - p.leave ? -1 : 2 * static_cast<int>(blockIdx.x) + (step0 == 0 ? 1 : 0);
      return true;
    }
    return false;
  }
};

template <typename F>
__device__ __forceinline__ Q4Share tree_share(const TreeParams& p, int ctas, bool report, F u_of, int at, int* b, long long* before) {
  return paged_share(p.n_seqs, ctas, [&](int i, bool first) {
    return static_cast<long long>(tree_units(p, paged_seq(p.cu, p.seqlens, i, p.total, p.max_q, p.max_k, report && first, 501))) * p.heads;
  }, u_of, at, b, before);
}

// Bit k of word w: the row's token sees key k0 + 32 w + k.
template <int W>
__device__ __forceinline__ void tree_mask(const TreeParams& p, const PagedSeq& s, int token, int k0, uint32_t (&w)[W]) {
  auto first_bits = [](int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; };
  const int end = p.tree ? s.len : s.base() + token + 1;
#pragma unroll
  for (int m = 0; m < W; ++m) w[m] = first_bits(end - (k0 + 32 * m));
  if (!p.tree) return;
  const int* row = p.tree + static_cast<size_t>(s.first + token) * p.words;
  auto word = [&](int i) { return i >= 0 && i < p.words ? static_cast<uint32_t>(__ldg(row + i)) : 0u; };
#pragma unroll
  for (int m = 0; m < W; ++m) {
    const int x = k0 + 32 * m - s.base();                     // the step's token of bit 0
    uint32_t bits = first_bits(-x);                           // tokens in front of the step's
    if (x > -32 && w[m]) {
      const int i = x >> 5;
      bits |= __funnelshift_r(word(i), word(i + 1), x & 31);
    }
    w[m] &= bits;
  }
}

__device__ __forceinline__ float max32(const float* s) {
  float a = fmax3(s[0], s[1], s[2]);
#pragma unroll
  for (int k = 3; k < 31; k += 2) a = fmax3(a, s[k], s[k + 1]);
  return fmaxf(a, s[31]);
}

// Multiplies COLS columns of a row of O.
template <int COLS>
__device__ __forceinline__ void tree_rescale(uint32_t t_o, float alpha) {
#pragma unroll 1
  for (int k = 0; k < COLS; k += 32) {
    uint32_t rr[32];
    tmem_ld32(t_o + k, rr);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float2 v = fmul2(make_float2(__uint_as_float(rr[i]), __uint_as_float(rr[i + 1])), make_float2(alpha, alpha));
      rr[i] = __float_as_uint(v.x);
      rr[i + 1] = __float_as_uint(v.y);
    }
    tmem_st32(t_o + k, rr);
  }
}

// Reference and sums of a row (or of one thread's half of it).
struct TreeRow {
  float m = -INFINITY, l = 0.f, lh = 0.f;

  // The reference follows ``cand`` (the largest score so far) where that is far above it: the factor of what has been
  // added up.  ``any``: some row of the warp moves.
  __device__ __forceinline__ float follow(float cand, float c2, bool valid, bool* any) {
    // a row that sees none of the keys so far has nothing to move
    const bool move = valid && cand != -INFINITY && (m == -INFINITY || (cand - m) * c2 > kTreeRescale);
    *any = __any_sync(0xffffffffu, move);
    const float alpha = move ? fast_exp2((m - cand) * c2) : 1.f;
    if (move) {
      l *= alpha;
      lh *= alpha;
      m = cand;
    }
    __syncwarp();                                             // (tensor memory is accessed by the whole warp at once)
    return alpha;
  }
};

// Weights of 32 scores, as 16 words of bf16 pairs; x = (s - ref) c2.
__device__ __forceinline__ void tree_weights(const float* s, float ref, float c2, TreeRow& r, uint32_t* pk) {
  float2 rs = make_float2(0.f, 0.f), hs = rs;
  const float2 nr = make_float2(-ref, -ref), c = make_float2(c2, c2);
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float2 x = fmul2(fadd2(make_float2(s[2 * k], s[2 * k + 1]), nr), c);
    const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
    pk[k] = pack_bf16x2(e.x, e.y);
    rs = fadd2(rs, e);
    hs = add_bf16x2_f32(hs, pk[k]);
  }
  r.l += rs.x + rs.y;
  r.lh += hs.x + hs.y;
}

// One key tile of a row, thread = row, where some keys are not seen or the reference is large: S in tensor memory
// (columns t_s) becomes P over its first half, O (t_o) is rescaled where the row's reference moves.  All rows of the
// warp see columns below ``all``, and none those from ``end`` on.
template <int D>
__device__ __forceinline__ void tree_softmax_masked(uint32_t t_s, uint32_t t_o, const uint32_t (&w)[4], int all, int end, bool first, bool valid,
                                                    float c2, TreeRow& r) {
  float s[32];
  auto load = [&](int k) {
    uint32_t rr[32];
    tmem_ld32(t_s + k * 32, rr);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) s[i] = __uint_as_float(rr[i]);
    if (k * 32 + 32 > all) {
      const uint32_t bits = k < 2 ? (k == 0 ? w[0] : w[1]) : (k == 2 ? w[2] : w[3]);
#pragma unroll
      for (int i = 0; i < 32; ++i) s[i] = bits >> i & 1u ? s[i] : -INFINITY;
    }
  };
  float cand = r.m;
#pragma unroll 1
  for (int k = 0; k < 4 && k * 32 < end; ++k) {
    load(k);
    cand = fmaxf(cand, max32(s));
  }
  bool any;
  const float alpha = r.follow(cand, c2, valid, &any);
  if (any && !first) tree_rescale<D>(t_o, alpha);
  const float ref = r.m == -INFINITY ? 0.f : r.m;
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {                               // (P of a quarter lies over S of quarters that were read)
    uint32_t pk[16];
    if (k * 32 < end) {
      load(k);
      tree_weights(s, ref, c2, r, pk);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) pk[i] = 0u;
    }
    tmem_st16(t_s + k * 16, pk);
  }
}

// The same where the row sees all keys, and c s - c m may be formed at once: false where c m has become so large that
// its rounding could matter (the tile is then done by the form above).
template <int D>
__device__ __forceinline__ bool tree_softmax_plain(uint32_t t_s, uint32_t t_o, bool first, bool valid, float c2, TreeRow& r) {
  // Weights are formed by a loop of two halves, the second one read again: less code (16 sequences of 1 to 60 tokens over
  // 500 to 8188, all 128 scores held and no loop: 92.8 us, this way 89; 4 x 512 tokens over 16384: 398 and 396), and no registers have to be moved to
  // these warps, which left the others too few (then 85 and 385).
  float s[64];
  auto load = [&](int k) {
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      uint32_t rr[32];
      tmem_ld32(t_s + 64 * k + 32 * y, rr);
#pragma unroll
      for (int i = 0; i < 32; ++i) s[32 * y + i] = __uint_as_float(rr[i]);
    }
    tmem_wait_ld();
  };
  float cand = r.m;
#pragma unroll
  for (int k = 1; k >= 0; --k) {                              // (half 0 stays)
    load(k);
#pragma unroll
    for (int y = 0; y < 2; ++y) cand = fmaxf(cand, max32(s + 32 * y));
  }
  bool any;
  const float alpha = r.follow(cand, c2, valid, &any);
  if (any) {
    if (!first) tree_rescale<D>(t_o, alpha);
    if (__any_sync(0xffffffffu, valid && fabsf(r.m * c2) > 4096.f && r.m != -INFINITY)) return false;
  }
  const float up = r.m == -INFINITY ? 0.f : -r.m * c2;
  const float2 c2v = make_float2(c2, c2), nms = make_float2(up, up);
  float2 rs[2], hs[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) rs[k] = hs[k] = make_float2(0.f, 0.f);
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    if (h) load(h);
    uint32_t pk[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float2 x = ffma2(make_float2(s[2 * k], s[2 * k + 1]), c2v, nms);
      const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
      pk[k] = pack_bf16x2(e.x, e.y);
      rs[k & 1] = fadd2(rs[k & 1], e);
      hs[k & 1] = add_bf16x2_f32(hs[k & 1], pk[k]);
    }
    tmem_st32(t_s + 32 * h, pk);
  }
  const float2 sum = fadd2(rs[0], rs[1]), sumh = fadd2(hs[0], hs[1]);
  r.l += sum.x + sum.y;
  r.lh += sumh.x + sumh.y;
  return true;
}

// Values that are no finite numbers were taken out of V's tiles where some row does not see their key (0 * NaN
// is NaN).  A row that does see one gets it here: the weight is positive, whatever it rounds to.
template <int D>
__device__ __forceinline__ void tree_spoil(const TreeParams& p, const TreeItem& x, int from, int token, int col, float (&acc)[32]) {
  for (int k = max(from, x.key0); k < x.key_end; ++k) {
    const int j = k - x.seq.base();
    const bool sees = p.tree ? j < 0 || (__ldg(p.tree + static_cast<size_t>(x.seq.first + token) * p.words + (j >> 5)) >> (j & 31) & 1)
                             : j <= token;
    if (!sees) continue;
    const int blk = k / p.cache.block_size;
    const int page = __ldg(p.cache.table + static_cast<size_t>(x.b) * p.cache.max_blocks + blk);
    if (page < 0 || page >= p.cache.num_blocks) continue;
    const uint16_t* v = p.v + ((static_cast<size_t>(page) * p.cache.block_size + (k - blk * p.cache.block_size)) * p.cache.H_kv + x.head / p.per_kv) * D + col;
    for (int i = 0; i < 32; ++i) {
      const uint32_t bits = __ldg(v + i);
      if ((bits & 0x7f80u) == 0x7f80u) acc[i] += __uint_as_float(bits << 16);
    }
  }
}

// By THREADS threads: of a tile of V rows from ``live`` on become 0, and of those from ``lo`` on what is no finite number.
// Whether this thread found any.
template <int D, int THREADS>
__device__ __forceinline__ bool clean_values(uint8_t* tile, int thread, int lo, int live) {
  constexpr int L = D / 8, RS = THREADS / L;                  // threads of a row, rows at a time (whole periods of the swizzle)
  static_assert(RS % 8 == 0, "rows of a thread share their swizzle");
  const int c = thread % L, r0 = thread / L;
  const int skip = min(lo, live) / RS * RS;
  uint8_t* mine = tile + (c >> 3) * 128 * 128 + sw128_offset(r0, (c & 7) * 8) + skip * 128;
  bool found = false;
#pragma unroll 4
  for (int r = r0 + skip; r < 128; r += RS, mine += RS * 128) {
    uint4* at = reinterpret_cast<uint4*>(mine);
    if (r >= live) {
      *at = make_uint4(0u, 0u, 0u, 0u);
    } else if (r >= lo) {
      uint4 v = *at;
      uint32_t* e = reinterpret_cast<uint32_t*>(&v);
      // an exponent of all ones carries into the sign's place
      uint32_t carry = 0;
#pragma unroll
      for (int y = 0; y < 4; ++y) carry |= ((e[y] & 0x7fff7fffu) + 0x00800080u) & 0x80008000u;
      if (carry) {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          if ((e[y] & 0x7f80u) == 0x7f80u) e[y] &= 0xffff0000u;
          if ((e[y] & 0x7f800000u) == 0x7f800000u) e[y] &= 0xffffu;
        }
        *at = v;
        found = true;
      }
    }
  }
  return found;
}

template <int D, int NT>
__global__ void __launch_bounds__(TreeCfg<D, NT>::THREADS, 1) attend_tree_kernel(const __grid_constant__ TreeParams p) {
  using C = TreeCfg<D, NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1k(smem_raw);
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sKV = smem + C::OFF_KV;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::NST;
  uint64_t* q_full = empty + C::NST;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;
  uint64_t* pv_done = s_full + 2;                             // NT = 2: a row tile's last product; NT = 1: each, by turns
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* start = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);
  // [row tile][item & 1] of the items that a row tile has keys in: the item's number, from 1, if it is
  volatile int* spoilt = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 20);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  int* counts = reinterpret_cast<int*>(smem + C::OFF_TAIL);
  TreeWalk<NT> walk{p, counts, 0, 0, 0, 0, {}, 0};
  uint32_t tbase = 0;

  if (warp == 0) {
    if (lane == 0) {
      for (int s = 0; s < C::NST; ++s) {
        mbar_init(&full[s], 1);
        mbar_init(&empty[s], 1);
      }
      mbar_init(q_full, 1);
      mbar_init(q_empty, 1);
      for (int t = 0; t < 2; ++t) {
        mbar_init(&s_full[t], 1);
        mbar_init(&pv_done[t], 1);
      }
      *abort_flag = 0;
      for (int i = 0; i < 4; ++i) spoilt[i] = 0;
      fence_mbarrier_init();
    }
    if (lane < 3) tma_prefetch_desc(lane == 0 ? &p.tk : lane == 1 ? &p.tv : &p.tq);
    if (p.shares) {
      int b;
      long long before = 0;
      const Q4Share sh = tree_share(p, gridDim.x, blockIdx.x == 0,
                                    [&](const Q4Share& y) { return static_cast<int>(blockIdx.x) < y.n && y.total > 0 ? y.begin(blockIdx.x) : -1LL; },
                                    -1, &b, &before);
      const int u = b < 0 ? 0 : static_cast<int>(sh.begin(blockIdx.x) - before);
      const int n = b < 0 ? 0 : static_cast<int>(sh.begin(blockIdx.x + 1) - sh.begin(blockIdx.x));
      if (lane == 0) {
        start[0] = b;
        start[1] = u;
        start[2] = n;
      }
      walk.begin(b, u, n);
    } else if (NT == 2) {
      tree_rest(p, gridDim.x, blockIdx.x == 0, counts);
      if (blockIdx.x == 0)
        for (int i = lane; i <= p.rest; i += 32) tree_counts(p)[i] = counts[i];
    }
    __syncwarp();
    named_bar_arrive(C::BAR_START, C::THREADS);               // the copies begin at once
  } else {
    if (warp == 1) {
      tmem_alloc(tmem_slot, C::TMEM_COLS);
      __syncwarp();
      tc_fence_before();
    }
    pdl_launch_dependents();
    named_bar_sync(C::BAR_START, C::THREADS);
    tc_fence_after();
    tbase = *tmem_slot;
    if (p.shares) walk.begin(start[0], start[1], start[2]);
  }

  TreeItem x{};
  // Key tiles of row tile t: those that some row of it sees.
  auto tiles = [&](int t) {
    const int token0 = (x.rb * NT + t) * p.tokens;
    if (token0 >= x.seq.nq) return 0;
    const int end = min(x.key_end, TreeWalk<NT>::seen(p, x.seq, token0 + p.tokens - 1));
    return end <= x.key0 ? 0 : (end - x.key0 + C::BN - 1) / C::BN;
  };
  // Keys from here on are not seen by every row of the block.
  auto common = [&] { return p.tree ? x.seq.base() : x.seq.base() + x.rb * NT * p.tokens + 1; };
  // Ring places of an item's tiles, from its first one, g: K_0 V_0 K_1 V_1 ... for two row tiles, and
  // K_0 K_1 V_0 K_2 V_1 ... for one.
  auto at_k = [&](int g, int j) { return NT == 2 ? g + 2 * j : g + (j == 0 ? 0 : 2 * j - 1); };
  auto at_v = [&](int g, int j, int n) { return NT == 2 ? g + 2 * j + 1 : j + 1 < n ? g + 2 * j + 2 : g + 2 * n - 1; };

  if (warp < 4) {
    if (warp == 0) {
      // -------------------------------------------------------------- copies
      bool ok = true;
      int g = 0;
      PagedStream<D> keys(p.cache);
      int slot = 0, laps = 0;                                 // of the next tile
      while (ok && walk.next(x)) {
        const int n = NT == 2 ? max(tiles(0), tiles(1)) : tiles(0), hkv = x.head / p.per_kv;
        keys.begin(p.cache, x.b, x.key0, x.key_end);
        int at = -1, before = -1;                             // of the last K tile, and of the one before it
        // K_0 V_0 K_1 V_1 ..., or K_0 K_1 V_0 K_2 V_1 ...
        for (int i = 0; i < 2 * n; ++i) {
          const bool last = i + 1 == 2 * n, is_k = !last && (NT == 2 ? (i & 1) == 0 : i == 0 || (i & 1));
          if (is_k) {
            before = at;
            at = keys.next(p.cache, 502);
          }
          if (laps > 0 && !(ok = mbar_wait_warp(&empty[slot], (laps - 1) & 1, abort_flag, 510))) break;
          keys.load(p.cache, is_k ? &p.tk : &p.tv, sKV + slot * C::TILE, &full[slot], hkv, NT == 2 || is_k || last ? at : before);
          ++g;
          if (++slot == C::NST) {
            slot = 0;
            ++laps;
          }
        }
      }
      // every signal is awaited; after an abort: every copy that was started lands
      for (int i = max(0, g - C::NST); ok && i < g; ++i) ok = mbar_wait_warp(&empty[i % C::NST], (i / C::NST) & 1, abort_flag, 511);
      if (!ok)
        for (int i = max(0, g - C::NST); i < g; ++i) mbar_wait_warp(&full[i % C::NST], (i / C::NST) & 1, nullptr, 512);
    } else if (warp == 1) {
      // -------------------------------------------------------------- products
      // After a failed wait the warp keeps joining every hand-off, issuing nothing.
      const uint32_t idesc_s = idesc_bf16_f32(128, 128, 0, 0);
      const uint32_t idesc_o = idesc_bf16_f32(128, D, 0, 1);
      const uint64_t dq0 = smem_desc_sw128(smem_u32(sQ), 0, 1024);
      const uint64_t dk0 = smem_desc_sw128(smem_u32(sKV), 0, 1024);
      const uint64_t dv0 = smem_desc_sw128(smem_u32(sKV), C::CHUNK, 1024);
      bool ok = true;
      int g = 0, items = 0, hc = 0;                           // hc: hand-offs so far (NT = 1)
      auto wait_tile = [&](int at) {
        ok = ok && mbar_wait_warp(&full[at % C::NST], (at / C::NST) & 1, abort_flag, 520);
        tc_fence_after();
      };
      auto issue_s = [&](int t, int buf, int at) {
        const uint64_t a = desc_advance(dq0, t * C::TILE);
        const uint64_t bd = desc_advance(dk0, (at % C::NST) * C::TILE);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = (ks >> 2) * C::CHUNK + (ks & 3) * 32;
          umma_ss_w(tbase + C::T_S + buf * 128, desc_advance(a, off), desc_advance(bd, off), idesc_s, ks > 0);
        }
        umma_commit_w(&s_full[buf]);
      };
      auto issue_pv = [&](int t, int buf, int at, bool fresh) {
        const uint64_t bd = desc_advance(dv0, (at % C::NST) * C::TILE);
#pragma unroll
        for (int ks = 0; ks < C::BN / 16; ++ks)
          umma_ts_w(tbase + C::T_O + t * 128, tbase + C::T_S + buf * 128 + ks * 8, desc_advance(bd, ks * 16 * 128), idesc_o,
                    (!fresh || ks > 0) ? 1u : 0u);
      };
      while (walk.next(x)) {
        const int n0 = tiles(0), n1 = NT == 2 ? tiles(1) : 0, n = max(n0, n1);
        if (n == 0) continue;
        ok = ok && mbar_wait_warp(q_full, items & 1, abort_flag, 521);
        ++items;
        if constexpr (NT == 2) {
          wait_tile(at_k(g, 0));
          if (ok) {
            if (n0 > 0) issue_s(0, 0, at_k(g, 0));
            if (n1 > 0) issue_s(1, 1, at_k(g, 0));
            umma_commit_w(&empty[at_k(g, 0) % C::NST]);
            if (n == 1) umma_commit_w(q_empty);
          }
          for (int j = 0; j < n; ++j) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int nt = t ? n1 : n0;
              if (j < nt) {
                __syncwarp();
                named_bar_sync(C::BAR_P + t, C::BAR_P_THREADS);
                if (ok) {
                  tc_fence_after();
                  issue_pv(t, t, at_v(g, j, n), j == 0);
                  if (j + 1 == nt) umma_commit_w(&pv_done[t]);
                }
              }
              if (ok && j + 1 < nt) issue_s(t, t, at_k(g, j + 1));
            }
            if (ok) {
              umma_commit_w(&empty[at_v(g, j, n) % C::NST]);
              if (j + 1 < n) umma_commit_w(&empty[at_k(g, j + 1) % C::NST]);
              if (j + 2 == n) umma_commit_w(q_empty);
            }
          }
        } else {
          // S of tiles 0 and 1; then, j by j, O += P_j V_j and S of tile j + 2 over P_j
          for (int i = -2; i < n; ++i) {
            if (i >= 0) {
              __syncwarp();
              named_bar_sync(C::BAR_P + (hc & 1), C::BAR_P_THREADS);
              if (ok) {
                tc_fence_after();
                issue_pv(0, hc & 1, at_v(g, i, n), i == 0);
                umma_commit_w(&pv_done[hc & 1]);
                umma_commit_w(&empty[at_v(g, i, n) % C::NST]);
              }
            }
            if (i + 2 < n) {
              wait_tile(at_k(g, i + 2));
              if (ok) {
                issue_s(0, (hc + (i < 0 ? i + 2 : 0)) & 1, at_k(g, i + 2));
                umma_commit_w(&empty[at_k(g, i + 2) % C::NST]);
                if (i + 3 == n) umma_commit_w(q_empty);
              }
            }
            if (i >= 0) ++hc;
          }
        }
        g += 2 * n;
      }
    } else if (warp == 2) {
      // -------------------------------------------------------------- joins P's hand-off once V is there
      bool ok = true;
      int g = 0, hc = 0;
      while (walk.next(x)) {
        const int n0 = tiles(0), n1 = NT == 2 ? tiles(1) : 0, n = max(n0, n1);
        if (n == 0) continue;
        for (int j = 0; j < n; ++j) {
          const int at = at_v(g, j, n);
          if (ok) ok = mbar_wait_warp(&full[at % C::NST], (at / C::NST) & 1, abort_flag, 530);
          if (NT == 2 && ok && j + 1 < n)
            ok = mbar_wait_warp(&full[at_k(g, j + 1) % C::NST], (at_k(g, j + 1) / C::NST) & 1, abort_flag, 531);
#pragma unroll
          for (int t = 0; t < NT; ++t)
            if (NT == 1 || j < (t ? n1 : n0)) {
              __syncwarp();
              named_bar_sync(C::BAR_P + (NT == 2 ? t : hc & 1), C::BAR_P_THREADS);
            }
          ++hc;
        }
        g += 2 * n;
      }
    } else {
      // -------------------------------------------------------------- Q
      bool ok = true;
      int items = 0;
      while (ok && walk.next(x)) {
        const int n0 = tiles(0), n1 = NT == 2 ? tiles(1) : 0;
        if (max(n0, n1) == 0) continue;
        if (items > 0 && !(ok = mbar_wait_warp(q_empty, (items - 1) & 1, abort_flag, 535))) break;
        const bool two = NT == 2 && (x.rb * NT + 1) * p.tokens < x.seq.nq;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full, (two ? 2 : 1) * p.tokens * p.group * D * 2);
#pragma unroll
          for (int t = 0; t < NT; ++t)
            if (t == 0 || two)
#pragma unroll
              for (int ch = 0; ch < C::CH; ++ch)
                tma_load_4d(sQ + t * C::TILE + ch * C::CHUNK, &p.tq, q_full, ch * 64, 0, x.head, x.seq.first + (x.rb * NT + t) * p.tokens);
        }
        __syncwarp();
        ++items;
      }
      if (ok && items > 0) ok = mbar_wait_warp(q_empty, (items - 1) & 1, abort_flag, 536);
      if (!ok && items > 0) mbar_wait_warp(q_full, (items - 1) & 1, nullptr, 537);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int wg = (warp - 4) >> 2;                           // NT = 2: row tile; NT = 1: half of the keys, and of O's columns
    const int t = NT == 2 ? wg : 0, half = NT == 1 ? wg : 0;
    constexpr int COLS = NT == 2 ? D : D / 2;                 // columns of O that a thread writes
    const int sub = warp & 3;                                 // TMEM lane quarter this warp may access
    const int row = sub * 32 + lane;
    const uint32_t t_lane = tbase + (static_cast<uint32_t>(sub * 32) << 16);
    const uint32_t t_o = t_lane + C::T_O + t * 128 + half * COLS;
    bool ok = true;
    int mine = 0, hc = 0;                                     // items that this row tile has keys in, key tiles so far
    int g = 0, others = 0;                                    // ring tiles so far; items that the other row tile has keys in
    const float c2 = p.c2;
    const int row_token = row / p.group, row_head = row - row_token * p.group;
    while (walk.next(x)) {
      const int n = tiles(t), n_other = NT == 2 ? tiles(t ^ 1) : 0, n_all = max(n, n_other);
      if (n_other > 0) ++others;
      const int token = (x.rb * NT + t) * p.tokens + row_token, head = x.head * p.group + row_head;
      const bool valid = row_token < p.tokens && token < x.seq.nq;
      const bool idle = !__any_sync(0xffffffffu, valid);
      TreeRow r;
      if (n > 0) {
        ++mine;
        if (p.tree && valid)                                  // (the words are wanted at the last key tiles)
          asm volatile("prefetch.global.L1 [%0];" :: "l"(p.tree + static_cast<size_t>(x.seq.first + token) * p.words));
        bool far = false;
        // keys below it are all the warp's rows'
        const int from = common();
        const int full_end = min(x.key_end, __reduce_min_sync(0xffffffffu, !valid ? 1 << 30 : p.tree ? x.seq.base() : x.seq.base() + token + 1));
        for (int j = 0; j < n; ++j, ++hc) {
          const int buf = NT == 2 ? t : hc & 1;
          const uint32_t t_s = t_lane + C::T_S + buf * 128;
          if (ok) ok = mbar_wait_warp(&s_full[buf], (NT == 2 ? hc : hc >> 1) & 1, abort_flag, 540);
          tc_fence_after();
          const int k0 = x.key0 + j * C::BN;
          const bool plain = k0 + C::BN <= full_end;
          // the first row tile that has the key tile cleans V, before its hand-off of P lets the product go
          if (ok && k0 + C::BN > min(from, x.key_end) && (t == 0 || j >= n_other)) {
            const int at = at_v(g, j, n_all);
            ok = mbar_wait_warp(&full[at % C::NST], (at / C::NST) & 1, abort_flag, 543);
            if (ok && clean_values<D, NT == 1 ? 256 : 128>(sKV + (at % C::NST) * C::TILE, NT == 1 ? threadIdx.x - 128 : row,
                                                            max(0, from - k0), min(C::BN, x.key_end - k0))) {
              spoilt[2 * t + (mine & 1)] = mine;
              if (j < n_other) spoilt[2 * (t ^ 1) + (others & 1)] = others;
              __threadfence_block();
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          if constexpr (NT == 2) {
            if (ok && !idle) {
              bool done = false;
              if (plain && !far) {
                done = tree_softmax_plain<D>(t_s, t_o, j == 0, valid, c2, r);
                far = !done;
              }
              if (!done) {
                uint32_t w[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
                if (!plain && valid) tree_mask<4>(p, x.seq, token, k0, w);
                __syncwarp();
                tree_softmax_masked<D>(t_s, t_o, w, full_end - k0, x.key_end - k0, j == 0, valid, c2, r);
              }
            }
          } else if (!idle) {
            // two threads a row: both read their half of S, exchange its maximum, and then write P over the first half
            float s[64];
            float top = -INFINITY;
            if (ok) {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint32_t rr[32];
                tmem_ld32(t_s + half * 64 + k * 32, rr);
#pragma unroll
                for (int i = 0; i < 32; ++i) s[k * 32 + i] = __uint_as_float(rr[i]);
              }
              tmem_wait_ld();
              if (!plain) {
                uint32_t w[2] = {0u, 0u};
                if (valid) tree_mask<2>(p, x.seq, token, k0 + half * 64, w);
#pragma unroll
                for (int k = 0; k < 64; ++k)
                  if (!(w[k >> 5] >> (k & 31) & 1u)) s[k] = -INFINITY;
                __syncwarp();
              }
              top = fmaxf(max32(s), max32(s + 32));
              tmem_st1(t_lane + C::T_X + 2 * (hc & 1) + half, __float_as_uint(top));
              tmem_wait_st();
              tc_fence_before();
            }
            named_bar_sync(C::BAR_PAIR + sub, 64);            // (joined whatever became of a wait)
            if (ok) {
              tc_fence_after();
              const uint32_t other = tmem_ld1(t_lane + C::T_X + 2 * (hc & 1) + (half ^ 1));
              tmem_wait_ld();
              bool any;
              const float alpha = r.follow(fmaxf(r.m, fmaxf(top, __uint_as_float(other))), c2, valid, &any);
              if (any && j > 0) {
                ok = mbar_wait_warp(&pv_done[(hc - 1) & 1], (hc - 1) >> 1 & 1, abort_flag, 541);
                tc_fence_after();
                if (ok) tree_rescale<COLS>(t_o, alpha);
              }
              const float ref = r.m == -INFINITY ? 0.f : r.m;
              uint32_t pk[32];
              tree_weights(s, ref, c2, r, pk);
              tree_weights(s + 32, ref, c2, r, pk + 16);
              tmem_st32(t_s + half * 32, pk);
            }
          }
          if (ok) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            named_bar_arrive(C::BAR_P + buf, C::BAR_P_THREADS);
          } else {                                            // after an abort: keep joining, blocking
            __syncwarp();
            named_bar_sync(C::BAR_P + buf, C::BAR_P_THREADS);
          }
        }
        if constexpr (NT == 1) {
          if (!idle) {                                        // the halves' sums
            tmem_st1(t_lane + C::T_X + 4 + half, __float_as_uint(r.l));
            tmem_st1(t_lane + C::T_X + 6 + half, __float_as_uint(r.lh));
            tmem_wait_st();
            tc_fence_before();
            named_bar_sync(C::BAR_PAIR + sub, 64);
            tc_fence_after();
            const uint32_t l0 = tmem_ld1(t_lane + C::T_X + 4), l1 = tmem_ld1(t_lane + C::T_X + 5);
            const uint32_t h0 = tmem_ld1(t_lane + C::T_X + 6), h1 = tmem_ld1(t_lane + C::T_X + 7);
            tmem_wait_ld();
            r.l = __uint_as_float(l0) + __uint_as_float(l1);
            r.lh = __uint_as_float(h0) + __uint_as_float(h1);
          }
        }
        if (ok) {
          // (one row tile: the product before the last one with this barrier was done when the last S was)
          const int done = NT == 2 ? t : (hc - 1) & 1;
          ok = mbar_wait_warp(&pv_done[done], (NT == 2 ? mine - 1 : (hc - 1) >> 1) & 1, abort_flag, 542);
          tc_fence_after();
        }
      }
      g += 2 * n_all;
      if (!ok || idle) continue;
      // the row's result, or its stretch's state
      const bool none = r.l == 0.f;
      const float inv = none ? 0.f : 1.f / r.lh;
      const bool spoil = n > 0 && spoilt[2 * t + (mine & 1)] == mine;
      const size_t th = static_cast<size_t>(x.seq.first + token) * p.H + head;
      float* dst = x.slot < 0 ? nullptr : p.part + (static_cast<size_t>(x.slot) * (p.state_rows / 32) + t * 4 + sub) * C::STATE + lane;
      // (lanes without a row write nothing, but come back for the next columns: all of a warp read tensor memory together)
#pragma unroll 1
      for (int k = 0; k < COLS; k += 32) {
        const int col = half * COLS + k;
        uint32_t rr[32];
        float acc[32];
        if (n > 0) {
          tmem_ld32(t_o + k, rr);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[i] = __uint_as_float(rr[i]);
          if (spoil && valid) tree_spoil<D>(p, x, common(), token, col, acc);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[i] = 0.f;
        }
        if (valid && dst) {
#pragma unroll
          for (int i = 0; i < 32; ++i) dst[(col + i) * 32] = acc[i];
        } else if (valid) {
          // (a row that sees nothing has sums of 0, and 0 here)
          uint4* out = reinterpret_cast<uint4*>(p.o + th * D + col);
#pragma unroll
          for (int i = 0; i < 32; i += 8)
            out[i / 8] = make_uint4(pack_bf16x2(acc[i] * inv, acc[i + 1] * inv), pack_bf16x2(acc[i + 2] * inv, acc[i + 3] * inv),
                                    pack_bf16x2(acc[i + 4] * inv, acc[i + 5] * inv), pack_bf16x2(acc[i + 6] * inv, acc[i + 7] * inv));
        }
        __syncwarp();
      }
      if (valid && half == 0) {
        if (dst) {
          dst[D * 32] = none ? -INFINITY : r.m * c2;
          dst[(D + 1) * 32] = r.l;
          dst[(D + 2) * 32] = r.lh;
        } else {
          p.lse[static_cast<size_t>(head) * p.total + x.seq.first + token] = none ? -INFINITY : fmaf(r.m, c2, log2f(r.l)) * 0.6931471805599453f;
        }
      }
      // (what was read of O comes before the next item's first product, which the next hand-off lets go)
      __syncwarp();
      tc_fence_before();
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, C::TMEM_COLS);
  }
}

// Joins the states of row blocks that are cut.  A block takes RB rows of one row block: a lane has one row and eight
// columns (a state's rows lie side by side), S warps share the states of those out, and where that leaves warps for
// less than D columns, blockIdx.y tells which.  SHARES: row block of bound i + 1 between the CTAs' shares, if that is
// the first within it, or, by_pair, the i-th row block of all; else the i-th row block of the rest.  Little code:
// each part of it runs once, and is fetched while nothing else happens (64 columns a lane, in straight lines: 7.6 us
// behind 1 x 8 tokens over 1000).
constexpr int kTreeJoinWarps = 16;

template <int D, int RB, int S>
struct TreeJoinCfg {
  static constexpr int STEP = 32 / RB;                        // lanes of a row
  static constexpr int COLS = kTreeJoinWarps / S * STEP * 8;  // columns of a block
  static_assert(COLS <= D, "columns of a block");
};

template <int D, int RB, int S, bool SHARES>
__global__ void __launch_bounds__(32 * kTreeJoinWarps) attend_tree_join_kernel(const __grid_constant__ TreeParams p, int ctas, int chunks, int by_pair) {
  using J = TreeJoinCfg<D, RB, S>;
  __shared__ int found[6];                                    // first token, tokens, key head, token of row 0, states, first slot
  __shared__ float merge[S > 1 ? kTreeJoinWarps : 1][11][32]; // a lane's columns, reference, sum, rounded sum
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunk = blockIdx.x % chunks, i = blockIdx.x / chunks;
  if (warp == 0) {
    int n = 0, slot = 0, head = 0, token0 = 0;
    PagedSeq s{0, 0, 0};
    if constexpr (SHARES) {
      // with fewer row blocks than bounds a block of this kernel takes one of those, else one of these
      const int at = by_pair ? i / p.heads : -1;
      int b;
      long long before = 0;
      const Q4Share sh = tree_share(p, ctas, false, [&](const Q4Share& y) { return i + 1 < y.n ? y.begin(i + 1) : -1LL; }, at, &b, &before);
      if (b >= 0) {
        s = paged_seq(p.cu, p.seqlens, b, p.total, p.max_q, p.max_k, false, 0);
        const int units = max(1, tree_units(p, s));
        head = by_pair ? i - b * p.heads : static_cast<int>(sh.begin(i + 1) - before) / units;
        const long long u0 = before + static_cast<long long>(head) * units;
        const int c0 = sh.owner(u0 + p.leave), c1 = sh.owner(u0 + units - 1);
        if (s.nq && c0 != c1 && (by_pair || c0 == i)) {       // (c0 == i: bound i + 1 is its first)
          n = c1 - c0 + 1;
          slot = 2 * c0;
        }
      }
    } else {
      pdl_wait();
      const int* counts = tree_counts(p);                     // (written by the first CTA)
      const TreeBlock<2> x(p, p.rounds * ctas + i);
      s = paged_seq(p.cu, p.seqlens, x.b, p.total, p.max_q, p.max_k, false, 0);
      head = x.head;
      token0 = x.rb * 2 * p.tokens;
      const int units = counts[p.rest], u0 = counts[i], u1 = counts[i + 1] - 1;
      if (u1 >= u0) {
        const int c0 = rest_owner(units, u0, ctas), c1 = rest_owner(units, u1, ctas);
        if (c0 != c1) {
          n = c1 - c0 + 1;
          slot = 2 * c0;
        }
      }
    }
    if (lane == 0) {
      found[0] = s.first; found[1] = s.nq; found[2] = head; found[3] = token0; found[4] = token0 < s.nq ? n : 0; found[5] = slot;
    }
  }
  __syncthreads();
  const int n = found[4], r = chunk * RB + lane % RB;
  const int in_tile = (r & 127) / p.group, token = found[3] + (r >> 7) * p.tokens + in_tile;
  const bool some = in_tile < p.tokens && token < found[1];
  const int col = (blockIdx.y * (kTreeJoinWarps / S) + warp / S) * J::STEP * 8 + (lane / RB) * 8;
  pdl_wait();
  if (n == 0 || !__any_sync(0xffffffffu, some)) return;       // (the same for the whole block: its warps have the same rows)
  float m = -INFINITY, l = 0.f, lh = 0.f, acc[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) acc[c] = 0.f;
  // a state's, or a warp's, share of the row (sum 0: no keys, and a reference of -inf; a sum that is no number goes on)
  auto add = [&](float mk, float lk, float lhk, const float (&v)[8]) {
    const float top = fmaxf(m, mk);
    const float alpha = top == m ? 1.f : fast_exp2(m - top), wt = lk == 0.f ? 0.f : fast_exp2(mk - top);
    m = top;
    l = fmaf(l, alpha, wt * lk);
    lh = fmaf(lh, alpha, wt * lhk);
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] = fmaf(acc[c], alpha, wt * v[c]);
  };
  constexpr int AT_ONCE = S > 4 ? 4 : 2;                      // states whose loads are under way together
  for (int k0 = warp % S; k0 < n; k0 += S * AT_ONCE) {
    float v[AT_ONCE][8], mk[AT_ONCE], lk[AT_ONCE], lhk[AT_ONCE];
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
      // state k: the first CTA's second place, the others' first one
      const int k = k0 + j * S, slot = found[5] + 2 * k + (k == 0 ? 1 : 0);
      const float* st = p.part + (static_cast<size_t>(slot) * (p.state_rows / 32) + (r >> 5)) * (32 * (D + 3)) + (r & 31);
      mk[j] = -INFINITY;
      lk[j] = lhk[j] = 0.f;
#pragma unroll
      for (int c = 0; c < 8; ++c) v[j][c] = k < n ? st[(col + c) * 32] : 0.f;
      if (k < n) {
        mk[j] = st[D * 32];
        lk[j] = st[(D + 1) * 32];
        lhk[j] = st[(D + 2) * 32];
      }
    }
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) add(mk[j], lk[j], lhk[j], v[j]);
  }
  if constexpr (S > 1) {
    if (warp % S) {
#pragma unroll
      for (int c = 0; c < 8; ++c) merge[warp][c][lane] = acc[c];
      merge[warp][8][lane] = m;
      merge[warp][9][lane] = l;
      merge[warp][10][lane] = lh;
    }
    __syncthreads();
    if (warp % S) return;
#pragma unroll 1
    for (int w = warp + 1; w < warp + S; ++w) {
      float v[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] = merge[w][c][lane];
      add(merge[w][8][lane], merge[w][9][lane], merge[w][10][lane], v);
    }
  }
  if (!some) return;
  const bool none = l == 0.f;
  const float inv = none ? 0.f : 1.f / lh;
  const int head = found[2] * p.group + (r & 127) - in_tile * p.group;
  uint32_t h[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) h[c] = none ? 0u : pack_bf16x2(acc[2 * c] * inv, acc[2 * c + 1] * inv);
  *reinterpret_cast<uint4*>(p.o + (static_cast<size_t>(found[0] + token) * p.H + head) * D + col) = make_uint4(h[0], h[1], h[2], h[3]);
  if (col == 0) p.lse[static_cast<size_t>(head) * p.total + found[0] + token] = none ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

template <int D, int RB, int S>
static cudaError_t launch_tree_join(const TreeParams& p, long long grid, long long cut, int by_pair, cudaStream_t stream) {
  const int chunks = RB == 8 ? 1 : p.state_rows / RB;
  const dim3 blocks(static_cast<unsigned>(cut * chunks), D / TreeJoinCfg<D, RB, S>::COLS);
  log_launch("attend_tree_join_kernel<D, RB, S, SHARES>", static_cast<unsigned long long>(blocks.x) * blocks.y, 32 * kTreeJoinWarps, 0ull);
  if constexpr (RB == 32)
    if (!p.shares)
      return launch_join(attend_tree_join_kernel<D, RB, S, false>, blocks, 32 * kTreeJoinWarps, stream, p, static_cast<int>(grid), chunks, 0);
  return launch_join(attend_tree_join_kernel<D, RB, S, true>, blocks, 32 * kTreeJoinWarps, stream, p, static_cast<int>(grid), chunks, by_pair);
}

template <int D, int NT>
static cudaError_t launch_attend_tree_d(const PagedTreeArgs& a, const TreeRows& t, cudaStream_t stream) {
  using C = TreeCfg<D, NT>;
  TreeParams p{};
  const int piece = paged_piece(a.block_size);
  const uint64_t rows = static_cast<uint64_t>(a.num_blocks) * a.block_size;
  if (!make_map_bf16_tok(&p.tk, a.k_cache, D, a.H_kv, rows, 64, piece) || !make_map_bf16_tok(&p.tv, a.v_cache, D, a.H_kv, rows, 64, piece) ||
      !make_map_bf16_group(&p.tq, a.q, D, t.group, a.H / t.group, a.total, 64, t.group, t.tokens))
    return cudaErrorInvalidValue;
  p.cache = paged_cache(a.block_table, a.H_kv, a.num_blocks, a.block_size, a.max_blocks);
  p.v = static_cast<const uint16_t*>(a.v_cache);
  p.o = static_cast<uint16_t*>(a.o); p.lse = a.lse; p.part = a.part + kTreeMaxCtas + 8;
  p.tree = a.tree; p.words = a.words; p.cu = a.cu; p.seqlens = a.seqlens;
  p.group = t.group; p.heads = a.H / t.group; p.per_kv = p.heads / a.H_kv; p.tokens = t.tokens;
  p.n_seqs = a.n_seqs; p.H = a.H; p.total = a.total; p.max_q = a.max_q; p.max_k = a.max_k;
  p.c2 = a.scale * 1.4426950408889634f;
  static int attr_done[64] = {0};
  cudaError_t e = ensure_smem_attr(attend_tree_kernel<D, NT>, C::SMEM_BYTES, attr_done);
  if (e != cudaSuccess) return e;
  const int sms = min(paged_sm_count(), kTreeMaxCtas);
  const long long pairs = static_cast<long long>(a.n_seqs) * p.heads;
  const long long steps = max(1, (a.max_k + kPagedTile - 1) / kPagedTile);
  long long grid;
  p.shares = t.tiles <= 2;
  p.state_rows = t.state_rows;
  if (p.shares) {
    p.whole = steps <= 1;
    // 16 mixed sequences of up to 60 tokens, four query heads: 120 us without, 95 with 4, 98 with 6 (their slowest CTA had
    // five short row blocks); 64 sequences of one token, up to 8192 keys, 233 us without, 227 with 1, 228 with 2
    p.leave = pairs * steps <= sms ? 0 : NT == 2 ? 4 : 1;
    grid = min(static_cast<long long>(sms), pairs * steps);
  } else {
    p.row_blocks = (t.tiles + 1) / 2;
    const long long items = pairs * p.row_blocks;
    grid = min(static_cast<long long>(sms), items * steps);
    p.rounds = static_cast<int>(items / grid);
    p.rest = static_cast<int>(items - p.rounds * grid);
  }
  log_launch("attend_tree_kernel<D, NT>", static_cast<unsigned long long>(grid), C::THREADS, static_cast<unsigned long long>(C::SMEM_BYTES));
  attend_tree_kernel<D, NT><<<static_cast<unsigned>(grid), C::THREADS, C::SMEM_BYTES, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the row blocks that a bound may cut: all, or one for each bound, or the rest
  const int by_pair = p.shares && pairs < grid;
  const long long cut = p.shares ? (p.whole ? 0 : by_pair ? pairs : grid - 1) : p.rest;
  if (cut == 0) return cudaSuccess;
  // A row block has some grid / pairs (or rest) states where the sequences are alike: with few of them a block has all columns,
  // with many each warp of eight has an eighth of them.
  const bool many = grid >= 4 * (p.shares ? pairs : p.rest);
  if (t.rows <= 8)
    return many && D == 128 ? launch_tree_join<D, 8, 8>(p, grid, cut, by_pair, stream) : launch_tree_join<D, 8, 512 / D>(p, grid, cut, by_pair, stream);
  return many ? launch_tree_join<D, 32, 8>(p, grid, cut, by_pair, stream) : launch_tree_join<D, 32, 128 / D>(p, grid, cut, by_pair, stream);
}

cudaError_t launch_attend_tree(const PagedTreeArgs& a, cudaStream_t stream) {
  const TreeRows t = tree_rows(a.H, a.H_kv, a.max_q);
  if (a.d == 64) return t.tiles == 1 ? launch_attend_tree_d<64, 1>(a, t, stream) : launch_attend_tree_d<64, 2>(a, t, stream);
  return t.tiles == 1 ? launch_attend_tree_d<128, 1>(a, t, stream) : launch_attend_tree_d<128, 2>(a, t, stream);
}

}  // namespace fa

FA_DEFINE_STATUS_FETCH(status_fetch_attend_tree)
