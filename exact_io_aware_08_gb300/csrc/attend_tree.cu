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
// Layout.  A CTA an SM takes NT tiles of 128 rows of one key head, and runs over keys 128 at a time:
//   warp 0       copies K and V tiles by TMA into one ring, in the order in which they are used.
//   warp 1       issues the products (the whole warp converged, one elected lane): S = Q K^T from shared
//                memory, O += P V with P from tensor memory.
//   warp 2       joins the hand-off of P once V is there, and cleans V's tile: rows behind the last key hold
//                anything, and 0 * NaN is NaN.
//   warps 4 on   softmax, thread = row; they bring the rows of Q in and write those of O out.
// Two S buffers are in flight: of the two row tiles (NT = 2, more than 128 rows), or of two key tiles in a
// row (NT = 1).
//
// Where one row block holds all rows of a sequence and key head, each CTA gets an equal share of all key steps,
// whatever the sequences' lengths, and what is cut is joined from states (Q4Share).  With more row blocks a
// CTA takes one, all row blocks of a key head side by side so that its keys are read from memory once.
#include "fa_kernels.h"
#include "paged_tile.cuh"
#include "q4_share.h"

namespace fa {

template <int D, int NT>
struct TreeCfg {
  static constexpr int BN = kPagedTile;
  static constexpr int CH = D / 64;
  static constexpr int CHUNK = 128 * 128;
  static constexpr int TILE = 128 * D * 2;
  static constexpr int ROWS = NT * 128;
  static constexpr int NST = D == 128 ? (NT == 1 ? 6 : 5) : 11;   // K and V tiles of the ring
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = NT * TILE;
  static constexpr int OFF_BAR = OFF_KV + NST * TILE;
  // full[NST], empty[NST], q_full[2], s_full[2], pv_done[2]; then the TMEM slot, abort flag, start[3], spoilt[4]
  static constexpr int NBAR = 2 * NST + 6;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 48 + 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget (227 KB per CTA)");
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t T_S = 0, T_O = 256;
  static constexpr int THREADS = 128 + NT * 128;
  // NT = 2: launched with 168 registers a thread, moved from the control warps
  static constexpr uint32_t REG_CTRL = 80, REG_SOFTMAX = 208;
  static constexpr int REG_NEED = NT == 2 ? 128 * (static_cast<int>(REG_CTRL) + 2 * static_cast<int>(REG_SOFTMAX)) : 0;
  static constexpr float RESCALE = 8.f;
  static constexpr uint32_t BAR_P = 2, BAR_P_THREADS = 128 + 32 + 32;
  static constexpr int STATE = D + 4;                         // O~, then reference, sum, rounded sum
};

struct TreeParams {
  CUtensorMap tk, tv;
  PagedCache cache;
  const uint16_t *q, *v;
  uint16_t* o;
  float *lse, *part;
  const int *tree, *cu, *seqlens;
  int words, n_seqs, H, G, total, max_q, max_k;
  int shares, whole;                                          // equal shares of key steps (of whole row blocks or not)
  int row_blocks, full_items, tail_splits, chunk, state_rows; // else: items from full_items on in tail_splits parts
  float c2;
};

// One stretch of work: row block rb of a key head of a sequence over keys [key0, key_end).
struct TreeItem {
  int b, hkv, rb, key0, key_end, slot;                        // slot: -1 results, else the state's place
  PagedSeq seq;
};

template <int ROWS>
struct TreeWalk {
  const TreeParams& p;
  int b, off, left;                                           // shares: sequence, unit in it, units left
  bool once;
  PagedSeq seq;
  int steps;

  __device__ __forceinline__ int seq_steps(const PagedSeq& s) const { return s.nq ? max(1, (s.len + kPagedTile - 1) / kPagedTile) : 0; }

  // Rows up to ``row`` of the sequence see keys below this.
  __device__ __forceinline__ static int seen(const TreeParams& p, const PagedSeq& s, int row) {
    return p.tree ? s.len : s.base() + min(row, s.nq * p.G - 1) / p.G + 1;
  }

  __device__ __forceinline__ bool next(TreeItem& x) {
    if (!p.shares) {
      if (once) return false;
      once = true;
      int item = blockIdx.x, split = 0, parts = 1;
      x.slot = -1;
      if (item >= p.full_items) {
        const int i = item - p.full_items;
        item = p.full_items + i / p.tail_splits;
        split = i % p.tail_splits;
        parts = p.tail_splits;
        x.slot = i;
      }
      x.rb = p.row_blocks - 1 - item % p.row_blocks;
      const int w = item / p.row_blocks;
      x.hkv = w % p.cache.H_kv;
      x.b = w / p.cache.H_kv;
      x.seq = paged_seq(p.cu, p.seqlens, x.b, p.total, p.max_q, p.max_k, x.rb == 0 && x.hkv == 0 && threadIdx.x == 0, 500);
      const int row0 = x.rb * ROWS;
      if (row0 >= x.seq.nq * p.G) return false;
      x.key0 = split * p.chunk;
      x.key_end = min(seen(p, x.seq, row0 + ROWS - 1), parts > 1 ? x.key0 + p.chunk : 1 << 30);
      return true;
    }
    if (left <= 0) return false;
    while (off >= steps * p.cache.H_kv) {                     // (a sequence with work follows: left > 0)
      if (++b >= p.n_seqs) return false;
      off = 0;
      seq = paged_seq(p.cu, p.seqlens, b, p.total, p.max_q, p.max_k, false, 0);
      steps = seq_steps(seq);
    }
    x.b = b;
    x.seq = seq;
    x.rb = 0;
    x.hkv = off / steps;
    const int step0 = off - x.hkv * steps;
    const int n = p.whole ? steps : min(left, steps - step0);
    x.key0 = step0 * kPagedTile;
    x.key_end = min(x.key0 + n * kPagedTile, seq.len);
    x.slot = n == steps ? -1 : 2 * blockIdx.x + (step0 == 0 ? 1 : 0);
    off += n;
    left -= n;
    return true;
  }
};

// By a whole warp: the shares, and the sequence that holds unit ``u_of(shares)`` with the units before it.
template <typename F>
__device__ __forceinline__ Q4Share tree_share(const TreeParams& p, int grid, bool report, F u_of, int* b, long long* before) {
  const int lane = threadIdx.x & 31;
  auto units = [&](int i, bool rep) -> long long {
    const PagedSeq s = paged_seq(p.cu, p.seqlens, i, p.total, p.max_q, p.max_k, rep, 501);
    return s.nq ? static_cast<long long>(max(1, (s.len + kPagedTile - 1) / kPagedTile)) * p.cache.H_kv : 0;
  };
  Q4Share sh;
  long long mine = 0, own = 0;
  for (int i = lane; i < p.n_seqs; i += 32) {
    const long long v = units(i, report);
    if (i == lane) own = v;
    mine += v;
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  sh.set(mine, grid);
  const long long u = u_of(sh);
  long long sum = 0;
  *b = -1;
  for (int base = 0; base < p.n_seqs && u >= 0; base += 32) {
    const long long v = base == 0 ? own : base + lane < p.n_seqs ? units(base + lane, false) : 0;
    long long inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    const uint32_t beyond = __ballot_sync(0xffffffffu, sum + inc > u);
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

// Bit k of word w: the row's token sees key k0 + 32 w + k.
__device__ __forceinline__ void tree_mask(const TreeParams& p, const PagedSeq& s, int token, int k0, uint32_t (&w)[4]) {
  // below the first n bits of a word
  auto first_bits = [](int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; };
  const int end = p.tree ? s.len : s.base() + token + 1;
#pragma unroll
  for (int m = 0; m < 4; ++m) w[m] = first_bits(end - (k0 + 32 * m));
  if (!p.tree) return;
  const int* row = p.tree + static_cast<size_t>(s.first + token) * p.words;
  auto word = [&](int i) { return i >= 0 && i < p.words ? static_cast<uint32_t>(__ldg(row + i)) : 0u; };
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int x = k0 + 32 * m - s.base();                     // the step's token of bit 0
    uint32_t bits = first_bits(-x);                           // tokens in front of the step's
    if (x > -32 && w[m]) {
      const int i = x >> 5, sh = x & 31;
      bits |= __funnelshift_r(word(i), word(i + 1), sh);
    }
    w[m] &= bits;
  }
}

// One key tile of a row: S in tensor memory (columns t_s) becomes P over its first half, O (t_o) is
// rescaled where the row's reference moves, once ``settle`` says that its last product is done.  PLAIN: the
// row sees all keys of the tile, and no reference is large (``far``); else w says which.
template <int D, bool PLAIN, typename F>
__device__ __forceinline__ bool tree_softmax(uint32_t t_s, uint32_t t_o, const uint32_t (&w)[4], bool first, float c2, float& m, float& l,
                                             float& lh, bool& far, F settle) {
  float s[128];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t rr[32];
    tmem_ld32(t_s + k * 32, rr);
#pragma unroll
    for (int i = 0; i < 32; ++i) s[k * 32 + i] = __uint_as_float(rr[i]);
  }
  tmem_wait_ld();
  if constexpr (!PLAIN) {
#pragma unroll
    for (int k = 0; k < 128; ++k)
      if (!(w[k >> 5] >> (k & 31) & 1u)) s[k] = -INFINITY;
  }
  float mx[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    mx[g] = fmax3(s[32 * g], s[32 * g + 1], s[32 * g + 2]);
#pragma unroll
    for (int k = 3; k < 31; k += 2) mx[g] = fmax3(mx[g], s[32 * g + k], s[32 * g + k + 1]);
    mx[g] = fmaxf(mx[g], s[32 * g + 31]);
  }
  const float cand = fmaxf(m, fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]));
  // a row that sees none of the tile's keys has nothing to move
  const bool move = cand != -INFINITY && (m == -INFINITY || (cand - m) * c2 > TreeCfg<D, 1>::RESCALE);
  if (__any_sync(0xffffffffu, move)) {
    const float alpha = move ? fast_exp2((m - cand) * c2) : 1.f;
    if (move) {
      l *= alpha;
      lh *= alpha;
      m = cand;
    }
    // c s - c m is off by the rounding of c m: where that could matter the reference is taken off first
    far = __any_sync(0xffffffffu, fabsf(m * c2) > 4096.f && m != -INFINITY);
    if (!first) {
      if (!settle()) return false;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        uint32_t rr[32];
        tmem_ld32(t_o + k * 32, rr);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float2 v = fmul2(make_float2(__uint_as_float(rr[i]), __uint_as_float(rr[i + 1])), make_float2(alpha, alpha));
          rr[i] = __float_as_uint(v.x);
          rr[i + 1] = __float_as_uint(v.y);
        }
        tmem_st32(t_o + k * 32, rr);
      }
    }
  }
  if (far) {
#pragma unroll
    for (int k = 0; k < 128; ++k) s[k] -= (m == -INFINITY) ? 0.f : m;
  }
  const float up = far || m == -INFINITY ? 0.f : -m * c2;
  const float2 c2v = make_float2(c2, c2), nms = make_float2(up, up);
  float2 rs[2], hs[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) rs[k] = hs[k] = make_float2(0.f, 0.f);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t pk[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float2 x = ffma2(make_float2(s[64 * h + 2 * k], s[64 * h + 2 * k + 1]), c2v, nms);
      const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
      pk[k] = pack_bf16x2(e.x, e.y);
      rs[k & 1] = fadd2(rs[k & 1], e);
      hs[k & 1] = add_bf16x2_f32(hs[k & 1], pk[k]);
    }
    tmem_st32(t_s + h * 32, pk);
  }
  const float2 sum = fadd2(rs[0], rs[1]), sumh = fadd2(hs[0], hs[1]);
  l += sum.x + sum.y;
  lh += sumh.x + sumh.y;
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
    const uint16_t* v = p.v + ((static_cast<size_t>(page) * p.cache.block_size + (k - blk * p.cache.block_size)) * p.cache.H_kv + x.hkv) * D + col;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const uint32_t bits = __ldg(v + i);
      if ((bits & 0x7f80u) == 0x7f80u) acc[i] += __uint_as_float(bits << 16);
    }
  }
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
  uint64_t* s_full = q_full + 2;
  uint64_t* pv_done = s_full + 2;                             // NT = 2: a row tile's last product; NT = 1: each, by turns
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* start = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);
  // [row tile][item & 1] of the items that a row tile has keys in: the item's number, from 1, if it is
  volatile int* spoilt = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 20);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (warp == 0) {
    if (lane == 0) {
      for (int s = 0; s < C::NST; ++s) {
        mbar_init(&full[s], 1);
        mbar_init(&empty[s], 1);
      }
      for (int t = 0; t < 2; ++t) {
        mbar_init(&q_full[t], 128);
        mbar_init(&s_full[t], 1);
        mbar_init(&pv_done[t], 1);
      }
      *abort_flag = 0;
      for (int i = 0; i < 4; ++i) spoilt[i] = 0;
      fence_mbarrier_init();
    }
    if (lane < 2) tma_prefetch_desc(lane ? &p.tv : &p.tk);
    if (p.shares) {
      int b;
      long long before = 0;
      const Q4Share sh = tree_share(p, gridDim.x, blockIdx.x == 0,
                                    [&](const Q4Share& y) { return static_cast<int>(blockIdx.x) < y.n && y.total > 0 ? y.begin(blockIdx.x) : -1LL; },
                                    &b, &before);
      if (lane == 0) {
        start[0] = b;
        start[1] = b < 0 ? 0 : static_cast<int>(sh.begin(blockIdx.x) - before);
        start[2] = b < 0 ? 0 : static_cast<int>(sh.begin(blockIdx.x + 1) - sh.begin(blockIdx.x));
      }
    }
  } else if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
  }
  pdl_launch_dependents();
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  TreeWalk<C::ROWS> walk{p, 0, 0, 0, false, {}, 0};
  if (p.shares) {
    walk.b = start[0];
    walk.off = start[1];
    walk.left = start[2];
    if (walk.left > 0) {
      walk.seq = paged_seq(p.cu, p.seqlens, walk.b, p.total, p.max_q, p.max_k, false, 0);
      walk.steps = walk.seq_steps(walk.seq);
      if (p.whole) {                                          // the row blocks that begin in the share
        const int behind = walk.off % walk.steps, skip = behind ? walk.steps - behind : 0;
        walk.off += skip;
        walk.left -= skip;
      }
    }
  }
  TreeItem x;
  // Key tiles of row tile t: those that some row of it sees.
  auto tiles = [&](int t) {
    const int row0 = x.rb * C::ROWS + t * 128;
    if (row0 >= x.seq.nq * p.G) return 0;
    const int end = min(x.key_end, TreeWalk<C::ROWS>::seen(p, x.seq, row0 + 127));
    return end <= x.key0 ? 0 : (end - x.key0 + C::BN - 1) / C::BN;
  };
  // Ring places of an item's tiles, from its first one, g: K_0 V_0 K_1 V_1 ... for two row tiles, and
  // K_0 K_1 V_0 K_2 V_1 ... for one.
  auto at_k = [&](int g, int j) { return NT == 2 ? g + 2 * j : g + (j == 0 ? 0 : 2 * j - 1); };
  auto at_v = [&](int g, int j, int n) { return NT == 2 ? g + 2 * j + 1 : j + 1 < n ? g + 2 * j + 2 : g + 2 * n - 1; };

  if (warp < 4) {
    if constexpr (NT == 2) setmaxnreg_dec<C::REG_CTRL>();
    if (warp == 0) {
      // -------------------------------------------------------------- copies
      bool ok = true;
      int g = 0;
      PageWindow win;
      auto load = [&](const CUtensorMap* map, int j) {
        const int s = g % C::NST, u = g / C::NST;
        if (u > 0 && !(ok = mbar_wait_warp(&empty[s], (u - 1) & 1, abort_flag, 510))) return;
        load_paged_tile<D>(p.cache, win, map, sKV + s * C::TILE, &full[s], x.b, x.hkv, x.key0 + j * C::BN, x.key_end, 502);
        ++g;
      };
      while (ok && walk.next(x)) {
        const int n = NT == 2 ? max(tiles(0), tiles(1)) : tiles(0);
        if (n == 0) continue;
        load(&p.tk, 0);
        for (int j = 0; ok && j < n; ++j) {
          if (NT == 1 && j + 1 < n) load(&p.tk, j + 1);
          if (ok) load(&p.tv, j);
          if (NT == 2 && ok && j + 1 < n) load(&p.tk, j + 1);
        }
      }
      // every signal is awaited; after an abort: every copy that was started lands
      if (ok) {
        for (int i = max(0, g - C::NST); ok && i < g; ++i) ok = mbar_wait_warp(&empty[i % C::NST], (i / C::NST) & 1, abort_flag, 511);
      }
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
      int g = 0, c0 = 0, c1 = 0, hc = 0;                      // items of the row tiles, hand-offs so far (NT = 1)
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
        if (n0 > 0) ok = ok && mbar_wait_warp(&q_full[0], c0++ & 1, abort_flag, 521);
        if (n1 > 0) ok = ok && mbar_wait_warp(&q_full[1], c1++ & 1, abort_flag, 522);
        if constexpr (NT == 2) {
          wait_tile(at_k(g, 0));
          if (ok) {
            if (n0 > 0) issue_s(0, 0, at_k(g, 0));
            if (n1 > 0) issue_s(1, 1, at_k(g, 0));
            umma_commit_w(&empty[at_k(g, 0) % C::NST]);
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
            }
          }
        } else {
          for (int j = 0; j < min(2, n); ++j) {
            wait_tile(at_k(g, j));
            if (ok) {
              issue_s(0, (hc + j) & 1, at_k(g, j));
              umma_commit_w(&empty[at_k(g, j) % C::NST]);
            }
          }
          for (int j = 0; j < n; ++j, ++hc) {
            __syncwarp();
            named_bar_sync(C::BAR_P + (hc & 1), C::BAR_P_THREADS);
            if (ok) {
              tc_fence_after();
              issue_pv(0, hc & 1, at_v(g, j, n), j == 0);
              umma_commit_w(&pv_done[hc & 1]);
              umma_commit_w(&empty[at_v(g, j, n) % C::NST]);
            }
            if (j + 2 < n) {
              wait_tile(at_k(g, j + 2));
              if (ok) {
                issue_s(0, hc & 1, at_k(g, j + 2));
                umma_commit_w(&empty[at_k(g, j + 2) % C::NST]);
              }
            }
          }
        }
        g += 2 * n;
      }
    } else if (warp == 2) {
      // -------------------------------------------------------------- joins P's hand-off once V is there
      bool ok = true;
      int g = 0, c0 = 0, c1 = 0, hc = 0;
      while (walk.next(x)) {
        const int n0 = tiles(0), n1 = NT == 2 ? tiles(1) : 0, n = max(n0, n1);
        if (n == 0) continue;
        if (n0 > 0) ++c0;
        if (n1 > 0) ++c1;
        // keys from ``from`` on are not seen by every row of the block
        const int from = p.tree ? x.seq.base() : x.seq.base() + x.rb * C::ROWS / p.G + 1;
        for (int j = 0; j < n; ++j) {
          const int at = at_v(g, j, n);
          if (ok) ok = mbar_wait_warp(&full[at % C::NST], (at / C::NST) & 1, abort_flag, 530);
          if (NT == 2 && ok && j + 1 < n)
            ok = mbar_wait_warp(&full[at_k(g, j + 1) % C::NST], (at_k(g, j + 1) / C::NST) & 1, abort_flag, 531);
          const int k0 = x.key0 + j * C::BN;
          if (ok && (k0 + C::BN > x.key_end || k0 + C::BN > from)) {
            uint8_t* tile = sKV + (at % C::NST) * C::TILE;
            bool found = false;
            for (int i = max(0, min(from, x.key_end) - k0) * (D / 8) + lane; i < C::BN * (D / 8); i += 32) {
              const int row = i / (D / 8), c = i % (D / 8);
              uint4* at16 = reinterpret_cast<uint4*>(tile + (c >> 3) * C::CHUNK + sw128_offset(row, (c & 7) * 8));
              if (k0 + row >= x.key_end) {
                *at16 = make_uint4(0u, 0u, 0u, 0u);
                continue;
              }
              uint4 v = *at16;
              uint32_t* e = reinterpret_cast<uint32_t*>(&v);
              bool bad = false;
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const bool lo = (e[y] & 0x7f80u) == 0x7f80u, hi = (e[y] & 0x7f800000u) == 0x7f800000u;
                bad |= lo || hi;
                if (lo) e[y] &= 0xffff0000u;
                if (hi) e[y] &= 0xffffu;
              }
              if (bad) *at16 = v;
              found |= bad;
            }
            if (found && n0 > 0) spoilt[c0 & 1] = c0;
            if (found && n1 > 0) spoilt[2 + (c1 & 1)] = c1;
            __threadfence_block();
            fence_proxy_async_smem();
          }
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
    }
  } else {
    // ---------------------------------------------------------------- softmax, thread = row
    if constexpr (NT == 2) setmaxnreg_inc<C::REG_SOFTMAX>();
    const int t = NT == 2 ? (warp - 4) >> 2 : 0;
    const int sub = warp & 3;                                 // TMEM lane quarter this warp may access
    const int row = sub * 32 + lane;
    const uint32_t t_lane = static_cast<uint32_t>(sub * 32) << 16;
    const uint32_t t_o = tbase + t_lane + C::T_O + t * 128;
    bool ok = true;
    int mine = 0, hc = 0;                                     // items that this row tile has keys in, key tiles so far
    const float c2 = p.c2;
    while (walk.next(x)) {
      const int n = tiles(t);
      const int rows = x.seq.nq * p.G, r = x.rb * C::ROWS + t * 128 + row;
      const int token = min(r, rows - 1) / p.G, head = x.hkv * p.G + r % p.G;
      const size_t th = static_cast<size_t>(x.seq.first + token) * p.H + head;
      float m = -INFINITY, l = 0.f, lh = 0.f;
      if (n > 0) {
        ++mine;
        // (this tile's products of the item before are done: their S has been read)
        uint4 q[D / 8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          q[i] = make_uint4(0u, 0u, 0u, 0u);
          if (r < rows) q[i] = __ldg(reinterpret_cast<const uint4*>(p.q + th * D) + i);
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          *reinterpret_cast<uint4*>(sQ + t * C::TILE + (i >> 3) * C::CHUNK + sw128_offset(row, (i & 7) * 8)) = q[i];
        fence_proxy_async_smem();
        mbar_arrive(&q_full[t]);
        bool far = false;
        // keys below it are all the warp's rows'
        const int full_end = __reduce_min_sync(0xffffffffu, r >= rows ? 1 << 30 : p.tree ? x.seq.base() : x.seq.base() + token + 1);
        const bool idle = __all_sync(0xffffffffu, r >= rows);
        for (int j = 0; j < n; ++j, ++hc) {
          const int buf = NT == 2 ? t : hc & 1;
          const uint32_t t_s = tbase + t_lane + C::T_S + buf * 128;
          if (ok) ok = mbar_wait_warp(&s_full[buf], (NT == 2 ? hc : hc >> 1) & 1, abort_flag, 540);
          if (ok && !idle) {
            tc_fence_after();
            const int k0 = x.key0 + j * C::BN;
            uint32_t w[4] = {0u, 0u, 0u, 0u};
            auto settle = [&] {
              if (NT == 2) return true;                       // S came behind the tile's last product
              const bool done = mbar_wait_warp(&pv_done[(hc - 1) & 1], (hc - 1) >> 1 & 1, abort_flag, 541);
              tc_fence_after();
              return done;
            };
            if (!far && k0 + C::BN <= min(full_end, x.key_end)) {
              ok = tree_softmax<D, true>(t_s, t_o, w, j == 0, c2, m, l, lh, far, settle);
            } else {
              if (r < rows) tree_mask(p, x.seq, token, k0, w);
              ok = tree_softmax<D, false>(t_s, t_o, w, j == 0, c2, m, l, lh, far, settle);
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
        if (ok) {
          // (one row tile: the product before the last one with this barrier was done when the last S was)
          const int done = NT == 2 ? t : (hc - 1) & 1;
          ok = mbar_wait_warp(&pv_done[done], (NT == 2 ? mine - 1 : (hc - 1) >> 1) & 1, abort_flag, 542);
          tc_fence_after();
        }
      }
      if (!ok || __all_sync(0xffffffffu, r >= rows)) continue;
      // the row's result, or its stretch's state
      const bool none = l == 0.f;
      const float inv = none ? 0.f : 1.f / lh;
      const bool spoil = n > 0 && spoilt[2 * t + (mine & 1)] == mine;
      float* dst = x.slot < 0 ? nullptr : p.part + (static_cast<size_t>(x.slot) * p.state_rows + (t * 128 + row)) * C::STATE;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        float acc[32];
        if (n > 0) {
          uint32_t rr[32];
          tmem_ld32(t_o + k * 32, rr);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[i] = __uint_as_float(rr[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[i] = 0.f;
        }
        if (r < rows) {
          if (spoil) tree_spoil<D>(p, x, p.tree ? x.seq.base() : x.seq.base() + x.rb * C::ROWS / p.G + 1, token, k * 32, acc);
          if (dst) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) *reinterpret_cast<float4*>(dst + k * 32 + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint32_t h[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) h[e] = none ? 0u : pack_bf16x2(acc[i + 2 * e] * inv, acc[i + 2 * e + 1] * inv);
              *reinterpret_cast<uint4*>(p.o + th * D + k * 32 + i) = make_uint4(h[0], h[1], h[2], h[3]);
            }
          }
        }
      }
      if (r < rows) {
        if (dst) *reinterpret_cast<float4*>(dst + D) = make_float4(none ? -INFINITY : m * c2, l, lh, 0.f);
        else
          p.lse[static_cast<size_t>(head) * p.total + x.seq.first + token] = none ? -INFINITY : fmaf(m, c2, log2f(l)) * 0.6931471805599453f;
      }
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

// Joins the n states of a row, ``stride`` floats apart (the first one ``skip`` further on), by one warp.
template <int D>
__device__ __forceinline__ void tree_join(const float* base, size_t stride, size_t skip, int n, uint16_t* o, float* lse) {
  constexpr int V = D / 32;                                   // consecutive elements a lane
  constexpr int AT_ONCE = 8;
  const int lane = threadIdx.x & 31;
  float M = -INFINITY, L = 0.f, LH = 0.f, acc[V];
#pragma unroll
  for (int k = 0; k < V; ++k) acc[k] = 0.f;
  for (int i0 = 0; i0 < n; i0 += AT_ONCE) {
    float4 ml[AT_ONCE];
    float v[AT_ONCE][V];
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
      ml[j] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
      if (i0 + j < n) {
        const float* st = base + (i0 + j) * stride + (i0 + j == 0 ? skip : 0);
        ml[j] = *reinterpret_cast<const float4*>(st + D);
#pragma unroll
        for (int k = 0; k < V; k += 2) {
          const float2 y = *reinterpret_cast<const float2*>(st + V * lane + k);
          v[j][k] = y.x;
          v[j][k + 1] = y.y;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
      if (ml[j].y == 0.f) continue;                           // no keys (a sum that is no number goes on)
      const float top = fmaxf(M, ml[j].x);
      const float alpha = top == M ? 1.f : fast_exp2(M - top), wt = fast_exp2(ml[j].x - top);
      M = top;
      L = fmaf(L, alpha, wt * ml[j].y);
      LH = fmaf(LH, alpha, wt * ml[j].z);
#pragma unroll
      for (int k = 0; k < V; ++k) acc[k] = fmaf(acc[k], alpha, wt * v[j][k]);
    }
  }
  const bool none = L == 0.f;
  const float inv = none ? 0.f : 1.f / LH;
#pragma unroll
  for (int k = 0; k < V; k += 2)
    *reinterpret_cast<uint32_t*>(o + V * lane + k) = none ? 0u : pack_bf16x2(acc[k] * inv, acc[k + 1] * inv);
  if (lane == 0) *lse = none ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// Rows whose row block lies in several CTAs' shares, a warp a row.
template <int D>
__global__ void __launch_bounds__(128) attend_tree_join_kernel(const __grid_constant__ TreeParams p, int ctas) {
  constexpr int STATE = TreeCfg<D, 1>::STATE;
  const long long th = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const bool some = th < static_cast<long long>(p.total) * p.H;
  const int tok = some ? static_cast<int>(th / p.H) : 0, head = static_cast<int>(th - static_cast<long long>(tok) * p.H);
  // (every sequence whose boundaries are sound has its rows, also where those of others are not)
  int b = -1;
  long long total = 0, before = 0;
  for (int i = threadIdx.x & 31; i < p.n_seqs; i += 32) {
    const PagedSeq s = paged_seq(p.cu, p.seqlens, i, p.total, p.max_q, p.max_k, false, 0);
    total += s.nq ? static_cast<long long>(max(1, (s.len + kPagedTile - 1) / kPagedTile)) * p.cache.H_kv : 0;
    if (some && s.first <= tok && tok < s.first + s.nq && b < 0) b = i;
  }
  const uint32_t has = __ballot_sync(0xffffffffu, b >= 0);
  if (has) b = static_cast<int>(__reduce_min_sync(0xffffffffu, static_cast<unsigned>(b < 0 ? 0x7fffffff : b)));
  for (int i = threadIdx.x & 31; i < b; i += 32) {
    const PagedSeq s = paged_seq(p.cu, p.seqlens, i, p.total, p.max_q, p.max_k, false, 0);
    before += s.nq ? static_cast<long long>(max(1, (s.len + kPagedTile - 1) / kPagedTile)) * p.cache.H_kv : 0;
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, off);
    before += __shfl_xor_sync(0xffffffffu, before, off);
  }
  int n = 0;
  size_t base = 0;
  if (b >= 0) {
    const PagedSeq s = paged_seq(p.cu, p.seqlens, b, p.total, p.max_q, p.max_k, false, 0);
    const int steps = max(1, (s.len + kPagedTile - 1) / kPagedTile);
    Q4Share sh;
    sh.set(total, ctas);
    const long long u0 = before + static_cast<long long>(head / p.G) * steps;
    const int c0 = sh.owner(u0), c1 = sh.owner(u0 + steps - 1);
    if (c0 != c1) {                                           // (else its CTA wrote the result)
      n = c1 - c0 + 1;
      base = (static_cast<size_t>(2 * c0) * p.state_rows + (tok - s.first) * p.G + head % p.G) * STATE;
    }
  }
  pdl_wait();
  if (n > 0)
    tree_join<D>(p.part + base, 2 * static_cast<size_t>(p.state_rows) * STATE, static_cast<size_t>(p.state_rows) * STATE, n,
                 p.o + static_cast<size_t>(th) * D, p.lse + static_cast<size_t>(head) * p.total + tok);
}

// Rows of the row blocks whose keys were split, a warp a row.
template <int D>
__global__ void __launch_bounds__(128) attend_tree_tail_kernel(const __grid_constant__ TreeParams p, int n_rows) {
  constexpr int STATE = TreeCfg<D, 2>::STATE, ROWS = TreeCfg<D, 2>::ROWS;
  const int i = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int it = i / ROWS, row = i - it * ROWS, item = p.full_items + it;
  const int rb = p.row_blocks - 1 - item % p.row_blocks, w = item / p.row_blocks;
  const int hkv = w % p.cache.H_kv, b = w / p.cache.H_kv;
  bool some = i < n_rows;
  PagedSeq s{0, 0, 0};
  if (some) s = paged_seq(p.cu, p.seqlens, b, p.total, p.max_q, p.max_k, false, 0);
  const int r = rb * ROWS + row;
  some = some && r < s.nq * p.G;
  pdl_wait();
  if (!some) return;
  const int tok = s.first + r / p.G, head = hkv * p.G + r % p.G;
  tree_join<D>(p.part + (static_cast<size_t>(it) * p.tail_splits * p.state_rows + row) * STATE, static_cast<size_t>(p.state_rows) * STATE, 0,
               p.tail_splits, p.o + (static_cast<size_t>(tok) * p.H + head) * D, p.lse + static_cast<size_t>(head) * p.total + tok);
}

template <int D, int NT>
static cudaError_t launch_attend_tree_d(const PagedTreeArgs& a, cudaStream_t stream) {
  using C = TreeCfg<D, NT>;
  TreeParams p{};
  const int piece = paged_piece(a.block_size);
  const uint64_t rows = static_cast<uint64_t>(a.num_blocks) * a.block_size;
  if (!make_map_bf16_tok(&p.tk, a.k_cache, D, a.H_kv, rows, 64, piece) || !make_map_bf16_tok(&p.tv, a.v_cache, D, a.H_kv, rows, 64, piece))
    return cudaErrorInvalidValue;
  p.cache = {a.block_table, a.H_kv, a.num_blocks, a.block_size, a.max_blocks, piece};
  p.q = static_cast<const uint16_t*>(a.q); p.v = static_cast<const uint16_t*>(a.v_cache);
  p.o = static_cast<uint16_t*>(a.o); p.lse = a.lse; p.part = a.part;
  p.tree = a.tree; p.words = a.words; p.cu = a.cu; p.seqlens = a.seqlens;
  p.n_seqs = a.n_seqs; p.H = a.H; p.G = a.H / a.H_kv; p.total = a.total; p.max_q = a.max_q; p.max_k = a.max_k;
  p.c2 = a.scale * 1.4426950408889634f;
  static int attr_done[64] = {0};
  cudaError_t e = ensure_smem_attr(attend_tree_kernel<D, NT>, C::SMEM_BYTES, attr_done, C::THREADS, C::REG_NEED);
  if (e != cudaSuccess) return e;
  const long long all_rows = static_cast<long long>(p.G) * a.max_q;
  const int sms = min(paged_sm_count(), kTreeMaxCtas);
  const long long pairs = static_cast<long long>(a.n_seqs) * a.H_kv;
  const long long steps = max(1, (a.max_k + kPagedTile - 1) / kPagedTile);
  long long grid;
  p.shares = all_rows <= C::ROWS;
  if (p.shares) {
    p.whole = steps <= 1;
    p.state_rows = static_cast<int>(all_rows);
    grid = min(static_cast<long long>(sms), pairs * steps);
  } else {
    p.state_rows = C::ROWS;
    p.row_blocks = static_cast<int>((all_rows + C::ROWS - 1) / C::ROWS);
    const long long items = pairs * p.row_blocks;
    const int tail = static_cast<int>(items % sms);
    const int s = tail ? static_cast<int>(min(static_cast<long long>(sms / tail), steps / 4)) : 1;
    p.full_items = static_cast<int>(items);
    p.tail_splits = 1;
    grid = items;
    if (s >= 2) {
      p.full_items = static_cast<int>(items - tail);
      p.tail_splits = s;
      p.chunk = static_cast<int>((steps + s - 1) / s) * kPagedTile;
      grid = p.full_items + static_cast<long long>(tail) * s;
    }
  }
  log_launch("attend_tree_kernel<D, NT>", static_cast<unsigned long long>(grid), C::THREADS, static_cast<unsigned long long>(C::SMEM_BYTES));
  attend_tree_kernel<D, NT><<<static_cast<unsigned>(grid), C::THREADS, C::SMEM_BYTES, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (p.shares) {
    if (p.whole) return cudaSuccess;
    const unsigned blocks = static_cast<unsigned>((static_cast<long long>(a.total) * a.H + 3) / 4);
    log_launch("attend_tree_join_kernel<D>", blocks, 128, 0ull);
    return launch_join(attend_tree_join_kernel<D>, blocks, 128, stream, p, static_cast<int>(grid));
  }
  if (p.tail_splits == 1) return cudaSuccess;
  const int n_rows = static_cast<int>((grid - p.full_items) / p.tail_splits) * C::ROWS;
  log_launch("attend_tree_tail_kernel<D>", n_rows / 4, 128, 0ull);
  return launch_join(attend_tree_tail_kernel<D>, static_cast<unsigned>(n_rows / 4), 128, stream, p, n_rows);
}

cudaError_t launch_attend_tree(const PagedTreeArgs& a, cudaStream_t stream) {
  const bool one = static_cast<long long>(a.H / a.H_kv) * a.max_q <= 128;
  if (a.d == 64) return one ? launch_attend_tree_d<64, 1>(a, stream) : launch_attend_tree_d<64, 2>(a, stream);
  return one ? launch_attend_tree_d<128, 1>(a, stream) : launch_attend_tree_d<128, 2>(a, stream);
}

}  // namespace fa

FA_DEFINE_STATUS_FETCH(status_fetch_attend_tree)
