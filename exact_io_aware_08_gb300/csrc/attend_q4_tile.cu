// Attention of many query rows over a paged cache held in 4 bits, on the tensor core that reads
// shared memory (the form for parts of prompts; attend_q4.cu has the one for single tokens).
//
// A CTA owns 256 rows of one key head, in two tiles of 128.  Rows are (query token, query head of the
// group) pairs, token by token, so that a tile is full whatever the group's size, and the rows of a
// token lie side by side in memory.  The mathematics is attend_q4.cu's: codes * scales are exact fp16
// numbers, query rows are brought to fp16 by a power of two, weights <= 2^15 are rounded to fp16, sums
// are fp32.  The reference m is at most 8 below the running maximum here, and weights are 2^(s - m + 7).
//
// Roles (512 threads, one CTA an SM):
//   warp 0       copies codes and scales, 64 keys a stage, by bulk copies.
//   warp 1       issues the products (the whole warp converged, one elected lane):
//                  S_t = Q_t K_j^T   both operands from shared memory
//                  O_t += P_t V_j    P_t from tensor memory
//                in the order PV_0(j), S_0(j+1), PV_1(j), S_1(j+1).
//   warp 2       joins the hand-off of P_t once V_j and K_(j+1) are there (warp 3 idles).
//   warps 4-11   softmax, thread = row; they also bring the rows of Q in and write those of O out.
//   warps 12-15  unpack: a lane takes 16 elements (8 code bytes, one scale), and writes 32 bytes of
//                fp16 into the 128-byte-swizzled tile, from where K is read K-major and V MN-major.
// Tensor memory: S_0, S_1 (P_t over the first half of S_t), O_0, O_1.
//
// Unpacking costs about 1.6 instructions an element and is shared by 256 rows: some 400 issue slots of
// each SM quarter a 128-key tile, and leaving it out (in a copy) changes no time.  What bounds the
// kernels is each tile's chain: softmax (1250 to 1650 clocks), hand-over, 1024 clocks of its products,
// landing of S; two tiles in flight (tensor memory is full) hide half of it.  A 128-key step of 256 rows
// takes some 3400 clocks where its products alone take 2048.  Measured and not kept, us for 4 x 1024
// tokens over 16384 keys with the forms of their day: two softmax threads a row 1312 against 1135; P
// handed over in two halves 830 against 792; S in halves of 64 keys, two in flight a tile, 1434 against
// 779 (their products issue at 91 clocks each instead of 50); part of the exponentials by polynomial 812
// against 792; products of a step in one asm block 733 against 712.  And for up to 128 rows, both tiles of
// a CTA over the same rows with the key tiles by turns: 118 against 99 us for 16 x 12 tokens over 8000
// keys, and as fast as before at d = 64 (two K and two V tiles are too few for it).
#include "fa_kernels.h"
#include "q4.cuh"

namespace fa {

template <int D>
struct Q4TCfg {
  static constexpr int BM = 128, BN = 128;
  static constexpr int CH = D / 64;                           // 64-column chunks of a tile
  static constexpr int CHUNK = 128 * 128;
  static constexpr int TILE = 128 * D * 2;                    // fp16 tile of Q, K or V
  static constexpr int NS = 2;                                // K and V tiles each
  static constexpr int CB = D / 2, SB = D / 16;
  static constexpr int CKEYS = 64;                            // keys of a code stage
  static constexpr int OFF_CV = CKEYS * CB;                   // inside a code stage
  static constexpr int OFF_CKS = 2 * CKEYS * CB;
  static constexpr int OFF_CVS = OFF_CKS + CKEYS * SB;
  static constexpr int CSTAGE = OFF_CVS + CKEYS * SB;
  static constexpr int NC = D == 128 ? 3 : 6;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = 2 * TILE;
  static constexpr int OFF_V = OFF_K + NS * TILE;
  static constexpr int OFF_C = OFF_V + NS * TILE;
  static constexpr int OFF_BAR = OFF_C + NC * CSTAGE;
  // q_full, k_full[NS], k_empty[NS], v_full[NS], v_empty[NS], s_full[2], o_done[2], c_full[NC], c_empty[NC]
  static constexpr int NBAR = 1 + 4 * NS + 4 + 2 * NC;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget (227 KB per CTA)");
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t T_S = 0, T_O = 256;
  static constexpr int THREADS = 512;
  static constexpr int UNPACK_WARPS = 4;
  // launched with 128 registers a thread, all of which the split uses
  static constexpr uint32_t REG_CTRL = 56, REG_SOFTMAX = 208, REG_UNPACK = 40;
  static constexpr int REG_NEED = 128 * (static_cast<int>(REG_CTRL) + 2 * static_cast<int>(REG_SOFTMAX) + static_cast<int>(REG_UNPACK));
  static constexpr float RESCALE = 8.f;
  static constexpr uint32_t BAR_START = 1, BAR_P = 3, BAR_P_THREADS = 128 + 32 + 32;
};

struct Q4TParams {
  const uint16_t* q;
  const uint8_t *kc, *ks, *vc, *vs;
  uint16_t* o;
  float *lse, *part;
  const int *cu_q, *seqlens, *table;
  int n_seqs, H, H_kv, G, total_q, max_q, max_k, causal, num_blocks, block_size, max_blocks, piece;
  int n_splits, chunk, row_blocks;                            // n_splits 0: the items from ``whole`` on in
  int whole, tail_splits, block_rows;                         // tail_splits parts; rows of an item
  float score, descale_v;
};

// fp16 A and B, fp32 accumulator
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int a_mn, int b_mn) {
  return idesc_bf16_f32(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10));
}

// Item of a CTA (or pair) by its index: row blocks with the most keys first over all sequences and
// heads, then the next.  ``parts``: chunks of the item's keys; ``state``: place of its first row's state.
struct Q4TItem {
  int b, hkv, rb, split, parts, chunk;
  size_t state;
};

__device__ __forceinline__ Q4TItem q4_tile_item(const Q4TParams& p, int index) {
  Q4TItem x;
  int item = index;
  x.split = 0;
  x.parts = 1;
  x.chunk = p.chunk;
  x.state = 0;
  if (p.n_splits) {
    x.parts = p.n_splits;
    item = index / p.n_splits;
    x.split = index - item * p.n_splits;
  } else if (index >= p.whole) {
    const int q = index - p.whole;
    x.parts = p.tail_splits;
    item = p.whole + q / p.tail_splits;
    x.split = q % p.tail_splits;
    x.state = static_cast<size_t>(q) * p.block_rows;
  }
  if (x.parts == 1) x.chunk = 1 << 30;                        // (all keys)
  const int per_rb = p.n_seqs * p.H_kv;
  x.rb = p.row_blocks - 1 - item / per_rb;
  const int w = item % per_rb;
  x.hkv = w % p.H_kv;
  x.b = w / p.H_kv;
  return x;
}

// Brings query row ``th`` (none: zeros) as row ``row`` of the tile, in fp16, and returns its score factor.
template <int D>
__device__ __forceinline__ float q4_query_row(const Q4TParams& p, bool has, size_t th, uint8_t* tile, int row) {
  uint4 x[D / 8];
  float big = 0.f;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (has) x[i] = __ldg(reinterpret_cast<const uint4*>(p.q + th * D) + i);
    const uint32_t ww[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) big = fmaxf(big, fmaxf(fabsf(bf16_lo(ww[k])), fabsf(bf16_hi(ww[k]))));
  }
  // the largest element goes to [2^14, 2^15); exponents such that the power and its inverse are normal
  const int ex = big == 0.f ? 14 : max(-100, static_cast<int>(__float_as_uint(big) >> 23) - 127);
  const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - ex) << 23);
  // (a factor that vanished would make 0 * -inf of a masked score; 2^-126 leaves every weight at 1 too)
  const float c2 = fmaxf(p.score * __uint_as_float(static_cast<uint32_t>(127 - 14 + ex) << 23), 0x1p-126f);
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    const uint32_t ww[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t h[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = pack_f16x2(bf16_lo(ww[k]) * up, bf16_hi(ww[k]) * up);
    *reinterpret_cast<uint4*>(tile + (i >> 3) * Q4TCfg<D>::CHUNK + sw128_offset(row, (i & 7) * 8)) =
        make_uint4(h[0], h[1], h[2], h[3]);
  }
  return c2;
}

// A value that the compiler forms again rather than hold what follows from it in registers.
__device__ __forceinline__ int again(int x) {
  asm volatile("" : "+r"(x));
  return x;
}

// One key tile of a row: S in tensor memory (columns t_s) becomes P over its first half, O (t_o) is
// rescaled where the row's reference moves.  Keys from ``lim`` on are not the row's.  ``far``: a
// reference of the warp is large.  PLAIN: all keys are the rows' and none was far; written out twice
// since the two tests stood as instructions of every element (794 instead of 758 us for 4x1024 tokens
// over 16384 keys).
template <int D, bool PLAIN>
__device__ __forceinline__ void q4_softmax_tile(uint32_t t_s, uint32_t t_o, int k0, int lim, bool first, float c2, float& m, float& l,
                                                bool& far) {
  // The row's 128 scores stay in registers: with 208 of them a thread nothing of this spills (kept in
  // quarters, two of them loaded twice, in 168 registers: 957 instead of 781 us for 4x1024 tokens over
  // 16384 keys; in 168 registers all 128: 1558).
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
      if (k0 + k >= lim) s[k] = -INFINITY;
  }
  float mx[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    mx[g] = fmax3(s[32 * g], s[32 * g + 1], s[32 * g + 2]);
#pragma unroll
    for (int k = 3; k < 31; k += 2) mx[g] = fmax3(mx[g], s[32 * g + k], s[32 * g + k + 1]);
    mx[g] = fmaxf(mx[g], s[32 * g + 31]);
  }
  const float mq = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]);
  const float cand = fmaxf(m, mq);
  // a row that sees none of the tile's keys has nothing to move
  const bool move = (PLAIN || cand != -INFINITY) && (m == -INFINITY || (cand - m) * c2 > Q4TCfg<D>::RESCALE);
  if (__any_sync(0xffffffffu, move)) {
    const float alpha = move ? fast_exp2((m - cand) * c2) : 1.f;
    if (move) {
      l *= alpha;
      m = cand;
    }
    // s c2 - m c2 + 7 is off by the rounding of 7 - m c2: where that could matter the reference is taken off
    // the scores first
    far = __any_sync(0xffffffffu, fabsf(m * c2) > 4096.f && m != -INFINITY);
    if (PLAIN && far) {
#pragma unroll
      for (int k = 0; k < 128; ++k) s[k] -= (m == -INFINITY) ? 0.f : m;
    }
    if (!first) {
      // O_t is settled: PV_t(j-1) completed before S_t(j) (same issuing thread, in order)
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
  if (!PLAIN && far) {
#pragma unroll
    for (int k = 0; k < 128; ++k) s[k] -= (m == -INFINITY) ? 0.f : m;
  }
  const float up = far || (!PLAIN && m == -INFINITY) ? kQ4Lift : fmaf(-m, c2, kQ4Lift);
  const float2 c2v = make_float2(c2, c2), nms = make_float2(up, up);
  float2 rs[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) rs[k] = make_float2(0.f, 0.f);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t pk[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float2 x = ffma2(make_float2(s[64 * h + 2 * k], s[64 * h + 2 * k + 1]), c2v, nms);
      const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
      pk[k] = pack_f16x2(e.x, e.y);
      rs[k & 3] = fadd2(rs[k & 3], e);
    }
    tmem_st32(t_s + h * 32, pk);
  }
  const float2 sum = fadd2(fadd2(rs[0], rs[1]), fadd2(rs[2], rs[3]));
  l += sum.x + sum.y;
}

// The row's result, or its chunk's state: O of columns t_o over l (``any``: some key tile was run).
template <int D>
__device__ __forceinline__ void q4_store_row(const Q4TParams& p, uint32_t t_o, bool any, bool has, size_t th, int tok, int head, const Q4TItem& item,
                                             int row, float c2, float m, float l) {
  const bool none = l == 0.f;                             // a row that sees no key (of the chunk)
  const float inv = none ? 0.f : p.descale_v / l;
  float* dst = nullptr;                                   // the chunk's state: [row][chunk], or [part][row of the block]
  if (item.parts > 1) dst = p.part + (p.n_splits ? th * p.n_splits + item.split : item.state + row) * (D + 2);
#pragma unroll
  for (int k = 0; k < D / 32; ++k) {
    uint32_t rr[32];
    if (any) {
      tmem_ld32(t_o + k * 32, rr);
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) rr[i] = 0u;
    }
    if (has) {
      if (dst) {
#pragma unroll
        for (int i = 0; i < 32; i += 2)
          *reinterpret_cast<float2*>(dst + k * 32 + i) = make_float2(__uint_as_float(rr[i]), __uint_as_float(rr[i + 1]));
      } else {
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            h[e] = none ? 0u : pack_bf16x2(__uint_as_float(rr[i + 2 * e]) * inv, __uint_as_float(rr[i + 2 * e + 1]) * inv);
          *reinterpret_cast<uint4*>(p.o + th * D + k * 32 + i) = make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
    }
  }
  if (has) {
    if (dst)
      *reinterpret_cast<float2*>(dst + D) = make_float2(none ? -INFINITY : fmaf(m, c2, -kQ4Lift), l);
    else
      p.lse[p.cu_q ? static_cast<size_t>(head) * p.total_q + tok : th] =
          none ? -INFINITY : fmaf(m, c2, log2f(l * 0x1p-7f)) * 0.6931471805599453f;
  }
}

template <int D>
__global__ void __launch_bounds__(Q4TCfg<D>::THREADS, 1) attend_q4_tile_kernel(const __grid_constant__ Q4TParams p) {
  using C = Q4TCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1k(smem_raw);
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  uint8_t* sC = smem + C::OFF_C;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* k_full = q_full + 1;
  uint64_t* k_empty = k_full + C::NS;
  uint64_t* v_full = k_empty + C::NS;
  uint64_t* v_empty = v_full + C::NS;
  uint64_t* s_full = v_empty + C::NS;
  uint64_t* o_done = s_full + 2;
  uint64_t* c_full = o_done + 2;
  uint64_t* c_empty = c_full + C::NC;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  const Q4TItem item = q4_tile_item(p, blockIdx.x);
  const int key0 = item.parts > 1 ? item.split * item.chunk : 0;
  // the copying warp's first 32 table entries, asked for before anything that decides which are used
  int window = key0 / p.block_size, tab = 0;
  if (warp == 0 && window + lane < p.max_blocks) tab = __ldg(p.table + static_cast<size_t>(item.b) * p.max_blocks + window + lane);
  const int rb = item.rb, hkv = item.hkv, b = item.b;
  int first = b, nq = 1;
  if (p.cu_q) {
    first = __ldg(p.cu_q + b);
    const int end = __ldg(p.cu_q + b + 1);
    nq = end - first;
    if (first < 0 || end < first || end > p.total_q || nq > p.max_q) {
      if (threadIdx.x == 0 && rb == 0) report_device_error(FA_DEV_BAD_CONFIG, 440);
      return;
    }
  }
  int len = __ldg(p.seqlens + b);
  if (len < 0 || len > p.max_k) {
    if (threadIdx.x == 0 && rb == 0) report_device_error(FA_DEV_BAD_CONFIG, 441);
    len = 0;
  }
  const int rows = nq * p.G;
  const int row0 = rb * 2 * C::BM;
  if (row0 >= rows) return;                                   // whole CTA, before any shared state
  // Row r of the sequence sees its first seen(r) keys; the item's keys are [key0, key_end), tile t
  // runs n_t[t] key tiles of 128.
  auto seen = [&](int r) { return p.causal ? max(0, len - nq + min(r, rows - 1) / p.G + 1) : len; };
  int n_t[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int last = min(key0 + item.chunk, seen(row0 + (t + 1) * C::BM - 1));
    n_t[t] = (row0 + t * C::BM >= rows || last <= key0) ? 0 : (last - key0 + C::BN - 1) / C::BN;
  }
  const int n_max = max(n_t[0], n_t[1]);
  const int key_end = min(key0 + item.chunk, seen(rows - 1 < row0 + 2 * C::BM - 1 ? rows - 1 : row0 + 2 * C::BM - 1));

  if (threadIdx.x == 0) {
    mbar_init(q_full, 256);
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(&k_full[s], C::UNPACK_WARPS);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], C::UNPACK_WARPS);
      mbar_init(&v_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&o_done[t], 1);
    }
    for (int s = 0; s < C::NC; ++s) {
      mbar_init(&c_full[s], 1);
      mbar_init(&c_empty[s], C::UNPACK_WARPS);
    }
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  pdl_launch_dependents();
  uint32_t tbase = 0;
  if (warp == 0) {                                            // the copies begin at once
    __syncwarp();
    named_bar_arrive(C::BAR_START, C::THREADS);
  } else {
    if (warp == 1) tmem_alloc(tmem_slot, C::TMEM_COLS);
    named_bar_sync(C::BAR_START, C::THREADS);
    tc_fence_after();
    tbase = *tmem_slot;
  }

  if (warp < 4) {
    setmaxnreg_dec<C::REG_CTRL>();
    if (warp == 0) {
      // -------------------------------------------------------------- copies of codes and scales
      const int pieces = C::CKEYS / p.piece;
      bool ok = true;
      int g = 0;
      const int n_st = 2 * n_max;                             // code stages (the last may hold no key)
      for (; ok && g < n_st; ++g) {
        const int s = g % C::NC, u = g / C::NC;
        const int kk = key0 + g * C::CKEYS;
        const int last = (min(kk + C::CKEYS, key_end) - 1) / p.block_size;
        if (kk < key_end && last >= window + 32) {
          window = kk / p.block_size;
          const int blk = window + lane;
          tab = blk <= (key_end - 1) / p.block_size ? __ldg(p.table + static_cast<size_t>(b) * p.max_blocks + blk) : 0;
        }
        const int key = kk + (lane < pieces ? lane : 0) * p.piece;
        const int blk = key / p.block_size;
        int page = __shfl_sync(0xffffffffu, tab, (blk - window) & 31);
        const bool mine = lane < pieces && key < key_end;
        if (mine && (page < 0 || page >= p.num_blocks)) {
          report_device_error(FA_DEV_BAD_CONFIG, 442);
          page = 0;                                           // stays in bounds; the result is reported invalid
        }
        if (u > 0 && !(ok = mbar_wait_warp(&c_empty[s], (u - 1) & 1, abort_flag, 450))) break;
        const int live = __popc(__ballot_sync(0xffffffffu, mine));
        if (lane == 0) mbar_arrive_expect_tx(&c_full[s], live * p.piece * 2 * (C::CB + C::SB));
        __syncwarp();
        if (mine) {
          uint8_t* st = sC + s * C::CSTAGE;
          const size_t row = (static_cast<size_t>(page) * p.H_kv + hkv) * p.block_size + (key - blk * p.block_size);
          const int at = lane * p.piece;
          bulk_load(st + at * C::CB, p.kc + row * C::CB, p.piece * C::CB, &c_full[s]);
          bulk_load(st + C::OFF_CKS + at * C::SB, p.ks + row * C::SB, p.piece * C::SB, &c_full[s]);
          bulk_load(st + C::OFF_CV + at * C::CB, p.vc + row * C::CB, p.piece * C::CB, &c_full[s]);
          bulk_load(st + C::OFF_CVS + at * C::SB, p.vs + row * C::SB, p.piece * C::SB, &c_full[s]);
        }
        __syncwarp();
      }
      // After an abort: let every copy land that was started.
      if (!ok)
        for (int x = max(0, g - C::NC); x < g; ++x) mbar_wait_warp(&c_full[x % C::NC], (x / C::NC) & 1, nullptr, 451);
    } else if (warp == 1) {
      // -------------------------------------------------------------- products
      // After a failed wait the warp keeps joining every hand-off, issuing nothing.
      if (n_max > 0) {
        const uint32_t idesc_s = idesc_f16_f32(128, 128, 0, 0);
        const uint32_t idesc_o = idesc_f16_f32(128, D, 0, 1);
        const uint64_t dq0 = smem_desc_sw128(smem_u32(sQ), 0, 1024);
        const uint64_t dk0 = smem_desc_sw128(smem_u32(sK), 0, 1024);
        const uint64_t dv0 = smem_desc_sw128(smem_u32(sV), C::CHUNK, 1024);
        auto issue_s = [&](int t, int j) {
          const uint64_t a = desc_advance(dq0, t * C::TILE);
          const uint64_t bd = desc_advance(dk0, (j % C::NS) * C::TILE);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = (ks >> 2) * C::CHUNK + (ks & 3) * 32;
            umma_ss_w(tbase + C::T_S + t * 128, desc_advance(a, off), desc_advance(bd, off), idesc_s, ks > 0);
          }
          umma_commit_w(&s_full[t]);
        };
        auto issue_pv = [&](int t, int j, bool fresh) {
          const uint64_t bd = desc_advance(dv0, (j % C::NS) * C::TILE);
#pragma unroll
          for (int ks = 0; ks < C::BN / 16; ++ks)
            umma_ts_w(tbase + C::T_O + t * 128, tbase + C::T_S + t * 128 + ks * 8, desc_advance(bd, ks * 16 * 128), idesc_o,
                      (!fresh || ks > 0) ? 1u : 0u);
        };
        bool ok = mbar_wait_warp(q_full, 0, abort_flag, 452) && mbar_wait_warp(&k_full[0], 0, abort_flag, 453);
        if (ok) {
          tc_fence_after();
          if (n_t[0] > 0) issue_s(0, 0);
          if (n_t[1] > 0) issue_s(1, 0);
          // (a tile is given back only where another follows in its place: no signal stays unawaited)
          if (C::NS < n_max) umma_commit_w(&k_empty[0]);
        }
        for (int j = 0; j < n_max; ++j) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (j < n_t[t]) {
              __syncwarp();
              named_bar_sync(C::BAR_P + t, C::BAR_P_THREADS);
              if (ok) {
                tc_fence_after();
                issue_pv(t, j, j == 0);
                if (j + 1 == n_t[t]) umma_commit_w(&o_done[t]);
              }
            }
            if (ok && j + 1 < n_t[t]) issue_s(t, j + 1);
          }
          if (ok) {
            if (j + C::NS < n_max) umma_commit_w(&v_empty[j % C::NS]);
            if (j + 1 + C::NS < n_max) umma_commit_w(&k_empty[(j + 1) % C::NS]);
          }
        }
      }
    } else if (warp == 2) {
      // -------------------------------------------------------------- joins P's hand-off once V_j, K_(j+1) are there
      bool ok = true;
      for (int j = 0; j < n_max; ++j) {
        if (ok) ok = mbar_wait_warp(&v_full[j % C::NS], (j / C::NS) & 1, abort_flag, 454);
        if (ok && j + 1 < n_max) ok = mbar_wait_warp(&k_full[(j + 1) % C::NS], ((j + 1) / C::NS) & 1, abort_flag, 455);
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (j < n_t[t]) {
            __syncwarp();
            named_bar_sync(C::BAR_P + t, C::BAR_P_THREADS);
          }
      }
    }
  } else if (warp >= 12) {
    // ---------------------------------------------------------------- unpacking
    setmaxnreg_dec<C::REG_UNPACK>();
    constexpr int BLK = D / 16;                               // scale blocks of a row
    constexpr int RPW = 32 / BLK;                             // rows a warp takes at once
    const int blk = lane % BLK, rsub = lane / BLK;
    // D = 128: the blocks of the second chunk write their two 16-byte units the other way round, so
    // that the eight lanes of a row reach eight different bank groups
    const int flip = (D == 128 && blk >= 4) ? 1 : 0;
    // A lane's rows are RSTEP apart, a multiple of 8: one swizzle, and constant strides.
    constexpr int RSTEP = RPW * C::UNPACK_WARPS;
    static_assert(RSTEP % 8 == 0, "rows of a lane share their swizzle");
    const int r0 = (warp - 12) * RPW + rsub;
    const uint32_t u0 = (blk >> 2) * C::CHUNK + sw128_offset(r0, ((blk & 3) * 2 + flip) * 8);
    const uint32_t u1 = (blk >> 2) * C::CHUNK + sw128_offset(r0, ((blk & 3) * 2 + (flip ^ 1)) * 8);
    auto unpack = [&](const uint8_t* codes, const uint8_t* scales, uint8_t* tile, int key_base) {
      uint2 cd[C::CKEYS / RSTEP];
      uint32_t e[C::CKEYS / RSTEP];
#pragma unroll
      for (int i = 0; i < C::CKEYS / RSTEP; ++i) {
        cd[i] = *reinterpret_cast<const uint2*>(codes + (r0 + i * RSTEP) * C::CB + blk * 8);
        e[i] = scales[(r0 + i * RSTEP) * C::SB + blk];
      }
      if (key_base + C::CKEYS > key_end) {
        // behind the item's keys lies anything, a scale that is no number among it
#pragma unroll
        for (int i = 0; i < C::CKEYS / RSTEP; ++i)
          if (key_base + r0 + i * RSTEP >= key_end) e[i] = 0;
      }
#pragma unroll
      for (int i = 0; i < C::CKEYS / RSTEP; ++i) {
        const uint32_t s = e4m3x2_to_f16(e[i] * 0x0101u);
        uint32_t h[2][4];
        e2m1x8_to_f16(flip ? cd[i].y : cd[i].x, h[0]);
        e2m1x8_to_f16(flip ? cd[i].x : cd[i].y, h[1]);
#pragma unroll
        for (int k = 0; k < 8; ++k) h[k >> 2][k & 3] = hmul2(h[k >> 2][k & 3], s);
        *reinterpret_cast<uint4*>(tile + u0 + i * RSTEP * 128) = make_uint4(h[0][0], h[0][1], h[0][2], h[0][3]);
        *reinterpret_cast<uint4*>(tile + u1 + i * RSTEP * 128) = make_uint4(h[1][0], h[1][1], h[1][2], h[1][3]);
      }
    };
    auto done = [&](uint64_t* bar) {                          // this warp's part is written: hand it to the tensor core
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    bool ok = true;
    for (int j = 0; ok && j < n_max; ++j) {
      const int s = j % C::NS, u = j / C::NS;
      const int g0 = 2 * j, g1 = 2 * j + 1;
      uint8_t* c0 = sC + (g0 % C::NC) * C::CSTAGE;
      uint8_t* c1 = sC + (g1 % C::NC) * C::CSTAGE;
      const int kk = key0 + j * C::BN;
      if (!(ok = mbar_wait_warp(&c_full[g0 % C::NC], (g0 / C::NC) & 1, abort_flag, 456))) break;
      if (u > 0 && !(ok = mbar_wait_warp(&k_empty[s], (u - 1) & 1, abort_flag, 457))) break;
      unpack(c0, c0 + C::OFF_CKS, sK + s * C::TILE, kk);
      if (!(ok = mbar_wait_warp(&c_full[g1 % C::NC], (g1 / C::NC) & 1, abort_flag, 458))) break;
      unpack(c1, c1 + C::OFF_CKS, sK + s * C::TILE + C::CKEYS * 128, kk + C::CKEYS);
      done(&k_full[s]);
      if (u > 0 && !(ok = mbar_wait_warp(&v_empty[s], (u - 1) & 1, abort_flag, 459))) break;
      unpack(c0 + C::OFF_CV, c0 + C::OFF_CVS, sV + s * C::TILE, kk);
      __syncwarp();
      if (lane == 0) mbar_arrive(&c_empty[g0 % C::NC]);
      unpack(c1 + C::OFF_CV, c1 + C::OFF_CVS, sV + s * C::TILE + C::CKEYS * 128, kk + C::CKEYS);
      done(&v_full[s]);
      if (lane == 0) mbar_arrive(&c_empty[g1 % C::NC]);
    }
  } else {
    // ---------------------------------------------------------------- softmax, thread = row
    setmaxnreg_inc<C::REG_SOFTMAX>();
    const int t = (warp - 4) >> 2;
    const int sub = warp & 3;                                 // TMEM lane quarter this warp may access
    const int row = sub * 32 + lane;
    const int r = row0 + t * C::BM + row;
    const uint32_t t_lane = static_cast<uint32_t>(sub * 32) << 16;
    const uint32_t t_s = tbase + t_lane + C::T_S + t * 128;
    const uint32_t t_o = tbase + t_lane + C::T_O + t * 128;
    const int n = t == 0 ? n_t[0] : n_t[1];
    const size_t th = static_cast<size_t>(first + r / p.G) * p.H + hkv * p.G + r % p.G;
    const float c2 = q4_query_row<D>(p, r < rows, th, sQ + t * C::TILE, row);
    fence_proxy_async_smem();
    mbar_arrive(q_full);
    const int lim = min(key_end, seen(r));                    // keys below it are this row's
    const int lim_low = __reduce_min_sync(0xffffffffu, lim);  // keys below it are all the warp's rows'
    bool far = false;
    float m = -INFINITY, l = 0.f;                             // reference (raw units) and sum of the weights
    bool ok = true;
    int j = 0;
    auto hand_over = [&] {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      named_bar_arrive(C::BAR_P + t, C::BAR_P_THREADS);
    };
    for (const int plain = min(n, (lim_low - key0) / C::BN); !far && j < plain; ++j) {
      if (!(ok = mbar_wait_warp(&s_full[t], j & 1, abort_flag, 460))) break;
      tc_fence_after();
      q4_softmax_tile<D, true>(t_s, t_o, key0 + j * C::BN, lim, j == 0, c2, m, l, far);
      hand_over();
    }
    for (; ok && j < n; ++j) {
      if (!(ok = mbar_wait_warp(&s_full[t], j & 1, abort_flag, 460))) break;
      tc_fence_after();
      q4_softmax_tile<D, false>(t_s, t_o, key0 + j * C::BN, lim, j == 0, c2, m, l, far);
      hand_over();
    }
    // after an abort: keep joining (blocking) the remaining hand-offs
    for (; j < n; ++j) {
      __syncwarp();
      named_bar_sync(C::BAR_P + t, C::BAR_P_THREADS);
    }
    if (ok && n > 0) {
      ok = mbar_wait_warp(&o_done[t], 0, abort_flag, 461);
      tc_fence_after();
    }
    if (ok && row0 + t * C::BM < rows) {
      const int x = again(r), tok = first + x / p.G, head = hkv * p.G + x % p.G;
      q4_store_row<D>(p, t_o, n > 0, x < rows, static_cast<size_t>(tok) * p.H + head, tok, head, item, x - row0, c2, m, l);
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

// ------------------------------------------------------------------------------------------
// The same for 512 rows of a key head on a pair of SMs (d = 128): a cluster of two CTAs whose tensor
// cores work on one product.  Tile t is 256 rows, 128 in each CTA, and each CTA holds half of the
// other operand: 64 of a key tile's 128 keys for S, 64 of the 128 columns of V for O.  So each
// unpacks half as much a row (K: its 64 keys whole, V: its half of every key), and the tensor core
// reads half as much of it from each shared memory.  4 x 1024 tokens over 16384 keys: 717 us, 809
// by CTAs of their own.
//
// The even CTA's warp 1 issues all products; the barriers it waits on are its own and both CTAs arrive
// there, and a product's completion is signalled to both.
// ------------------------------------------------------------------------------------------
struct Q4PCfg {
  static constexpr int D = 128, BN = 128;
  static constexpr int CHUNK = 128 * 128;                     // 64 columns of a Q tile, or V's half
  static constexpr int QTILE = 2 * CHUNK;
  static constexpr int HALF = 16384;                          // half a K tile [2 chunks][64 keys], or of V [128 keys]
  static constexpr int NS = 3;
  static constexpr int CB = 64, SB = 8;
  static constexpr int OFF_CV = 64 * CB;                      // inside a code stage: K of 64 keys, V of 128, scales
  static constexpr int OFF_CKS = OFF_CV + 128 * CB;
  static constexpr int OFF_CVS = OFF_CKS + 64 * SB;
  static constexpr int CSTAGE = OFF_CVS + 128 * SB;
  static constexpr int NC = 3;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = 2 * QTILE;
  static constexpr int OFF_V = OFF_K + NS * HALF;
  static constexpr int OFF_C = OFF_V + NS * HALF;
  static constexpr int OFF_BAR = OFF_C + NC * CSTAGE;
  // q_full, k_full[NS], v_full[NS], p_full[2] (of the even CTA); k_empty[NS], v_empty[NS], s_full[2],
  // o_done[2], c_full[NC], c_empty[NC]
  static constexpr int NBAR = 1 + 4 * NS + 6 + 2 * NC;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget (227 KB per CTA)");
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t T_S = 0, T_O = 256;
  static constexpr int THREADS = 512;
  static constexpr int UNPACK_WARPS = 4;
  static constexpr uint32_t BAR_START = 1;
  // (4 x 1024 tokens over 16384 keys with 48, 208 and 48 721 us; with 56, 208, 40 717; with 72, 200, 40 794)
  static constexpr uint32_t REG_CTRL = 56, REG_SOFTMAX = 208, REG_UNPACK = 40;
  static constexpr int REG_NEED = 128 * (static_cast<int>(REG_CTRL) + 2 * static_cast<int>(REG_SOFTMAX) + static_cast<int>(REG_UNPACK));
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Q4PCfg::THREADS, 1)
attend_q4_pair_kernel(const __grid_constant__ Q4TParams p) {
  using C = Q4PCfg;
  constexpr int D = C::D;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1k(smem_raw);                    // (the same address in both CTAs)
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  uint8_t* sC = smem + C::OFF_C;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* k_full = q_full + 1;
  uint64_t* v_full = k_full + C::NS;
  uint64_t* p_full = v_full + C::NS;
  uint64_t* k_empty = p_full + 2;
  uint64_t* v_empty = k_empty + C::NS;
  uint64_t* s_full = v_empty + C::NS;
  uint64_t* o_done = s_full + 2;
  uint64_t* c_full = o_done + 2;
  uint64_t* c_empty = c_full + C::NC;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());

  const Q4TItem item = q4_tile_item(p, blockIdx.x >> 1);      // of 512 rows
  const int key0 = item.parts > 1 ? item.split * item.chunk : 0;
  // the copying warp's first 32 table entries, asked for before anything that decides which are used
  int window = key0 / p.block_size, tab = 0;
  if (warp == 0 && window + lane < p.max_blocks) tab = __ldg(p.table + static_cast<size_t>(item.b) * p.max_blocks + window + lane);
  const int rb = item.rb, hkv = item.hkv, b = item.b;
  int first = b, nq = 1;
  if (p.cu_q) {
    first = __ldg(p.cu_q + b);
    const int end = __ldg(p.cu_q + b + 1);
    nq = end - first;
    if (first < 0 || end < first || end > p.total_q || nq > p.max_q) {
      if (threadIdx.x == 0 && rb == 0) report_device_error(FA_DEV_BAD_CONFIG, 470);
      return;
    }
  }
  int len = __ldg(p.seqlens + b);
  if (len < 0 || len > p.max_k) {
    if (threadIdx.x == 0 && rb == 0) report_device_error(FA_DEV_BAD_CONFIG, 471);
    len = 0;
  }
  const int rows = nq * p.G;
  const int row0 = rb * 512;
  if (row0 >= rows) return;                                   // both CTAs, before any shared state
  auto seen = [&](int r) { return p.causal ? max(0, len - nq + min(r, rows - 1) / p.G + 1) : len; };
  int n_t[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int last = min(key0 + item.chunk, seen(row0 + t * 256 + 255));
    n_t[t] = (row0 + t * 256 >= rows || last <= key0) ? 0 : (last - key0 + C::BN - 1) / C::BN;
  }
  const int n_max = max(n_t[0], n_t[1]);
  const int key_end = min(key0 + item.chunk, seen(row0 + 511));

  if (threadIdx.x == 0) {
    mbar_init(q_full, 16);                                    // softmax warps of both CTAs
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(&k_full[s], 2 * C::UNPACK_WARPS);
      mbar_init(&v_full[s], 2 * C::UNPACK_WARPS);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&p_full[t], 8 + 1);                           // the tile's softmax warps of both CTAs, and the helper
      mbar_init(&s_full[t], 1);
      mbar_init(&o_done[t], 1);
    }
    for (int s = 0; s < C::NC; ++s) {
      mbar_init(&c_full[s], 1);
      mbar_init(&c_empty[s], C::UNPACK_WARPS);
    }
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  pdl_launch_dependents();
  uint32_t tbase = 0;
  if (warp == 0) {                                            // the copies, into this CTA, begin at once
    __syncwarp();
    named_bar_arrive(C::BAR_START, C::THREADS);
    cluster_arrive();
  } else {
    if (warp == 1) tmem_alloc_pair(tmem_slot, C::TMEM_COLS);
    named_bar_sync(C::BAR_START, C::THREADS);
    cluster_sync();                                           // barriers and tensor memory of both are there
    tc_fence_after();
    tbase = *tmem_slot;
  }

  if (warp < 4) {
    setmaxnreg_dec<C::REG_CTRL>();
    if (warp == 0) {
      // -------------------------------------------------------------- copies: K of this CTA's 64 keys, V of all 128
      const int kp = 64 / p.piece, vp = 128 / p.piece;        // at most 4 and 8 pieces: lanes 8 to 11, 0 to 7
      bool ok = true;
      int g = 0;
      for (; ok && g < n_max; ++g) {
        const int s = g % C::NC, u = g / C::NC;
        const int kk = key0 + g * C::BN;                      // (< key_end)
        const int blk0 = kk / p.block_size;
        if (blk0 + 8 >= window + 32) {
          window = blk0;
          tab = window + lane <= (key_end - 1) / p.block_size
                    ? __ldg(p.table + static_cast<size_t>(b) * p.max_blocks + window + lane) : 0;
        }
        const bool is_v = lane < 8;
        const int piece = is_v ? lane : lane - 8;
        const bool role = is_v ? piece < vp : (lane < 12 && piece < kp);
        const int at = role ? piece * p.piece : 0;            // key of the stage's part
        const int key = kk + (is_v ? 0 : rank * 64) + at;
        const int blk = key / p.block_size;
        int page = __shfl_sync(0xffffffffu, tab, (blk - window) & 31);
        const bool mine = role && key < key_end;
        if (mine && (page < 0 || page >= p.num_blocks)) {
          report_device_error(FA_DEV_BAD_CONFIG, 472);
          page = 0;                                           // stays in bounds; the result is reported invalid
        }
        if (u > 0 && !(ok = mbar_wait_warp(&c_empty[s], (u - 1) & 1, abort_flag, 480))) break;
        const int live = __popc(__ballot_sync(0xffffffffu, mine));
        if (lane == 0) mbar_arrive_expect_tx(&c_full[s], live * p.piece * (C::CB + C::SB));
        __syncwarp();
        if (mine) {
          uint8_t* st = sC + s * C::CSTAGE;
          const size_t row = (static_cast<size_t>(page) * p.H_kv + hkv) * p.block_size + (key - blk * p.block_size);
          bulk_load(st + (is_v ? C::OFF_CV : 0) + at * C::CB, (is_v ? p.vc : p.kc) + row * C::CB, p.piece * C::CB, &c_full[s]);
          bulk_load(st + (is_v ? C::OFF_CVS : C::OFF_CKS) + at * C::SB, (is_v ? p.vs : p.ks) + row * C::SB, p.piece * C::SB,
                    &c_full[s]);
        }
        __syncwarp();
      }
      if (!ok)
        for (int x = max(0, g - C::NC); x < g; ++x) mbar_wait_warp(&c_full[x % C::NC], (x / C::NC) & 1, nullptr, 481);
    } else if (warp == 1 && rank == 0) {
      // -------------------------------------------------------------- products of the pair
      const uint32_t idesc = idesc_f16_f32(256, 128, 0, 0), idesc_o = idesc_f16_f32(256, 128, 0, 1);
      const uint64_t dq0 = smem_desc_sw128(smem_u32(sQ), 0, 1024);
      const uint64_t dk0 = smem_desc_sw128(smem_u32(sK), 0, 1024);
      const uint64_t dv0 = smem_desc_sw128(smem_u32(sV), C::CHUNK, 1024);
      auto issue_s = [&](int t, int j) {
        const uint64_t a = desc_advance(dq0, t * C::QTILE);
        const uint64_t bd = desc_advance(dk0, (j % C::NS) * C::HALF);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          umma_ss_pair(tbase + C::T_S + t * 128, desc_advance(a, (ks >> 2) * C::CHUNK + (ks & 3) * 32),
                       desc_advance(bd, (ks >> 2) * (C::HALF / 2) + (ks & 3) * 32), idesc, ks > 0);
        umma_commit_pair(&s_full[t]);
      };
      auto issue_pv = [&](int t, int j) {
        const uint64_t bd = desc_advance(dv0, (j % C::NS) * C::HALF);
#pragma unroll
        for (int ks = 0; ks < C::BN / 16; ++ks)
          umma_ts_pair(tbase + C::T_O + t * 128, tbase + C::T_S + t * 128 + ks * 8, desc_advance(bd, ks * 16 * 128), idesc_o,
                       (j > 0 || ks > 0) ? 1u : 0u);
      };
      bool ok = n_max > 0 && mbar_wait_warp_cluster(q_full, 0, abort_flag, 482) &&
                mbar_wait_warp_cluster(&k_full[0], 0, abort_flag, 483);
      if (ok) {
        tc_fence_after();
        if (n_t[0] > 0) issue_s(0, 0);
        if (n_t[1] > 0) issue_s(1, 0);
        // (a tile is given back only where another follows in its place: no signal stays unawaited)
        if (C::NS < n_max) umma_commit_pair(&k_empty[0]);
      }
      for (int j = 0; ok && j < n_max; ++j) {
        // V_j and K_(j+1) are there: the helper waited for them before its arrival
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (j < n_t[t]) {
            if (!(ok = mbar_wait_warp_cluster(&p_full[t], j & 1, abort_flag, 484))) break;
            tc_fence_after();
            issue_pv(t, j);
            if (j + 1 == n_t[t]) umma_commit_pair(&o_done[t]);
          }
          if (j + 1 < n_t[t]) issue_s(t, j + 1);
        }
        if (!ok) break;
        if (j + C::NS < n_max) umma_commit_pair(&v_empty[j % C::NS]);
        if (j + 1 + C::NS < n_max) umma_commit_pair(&k_empty[(j + 1) % C::NS]);
      }
    } else if (warp == 2 && rank == 0) {
      // -------------------------------------------------------------- arrives for P_t once V_j, K_(j+1) are there
      bool ok = true;
      for (int j = 0; ok && j < n_max; ++j) {
        if (!(ok = mbar_wait_warp_cluster(&v_full[j % C::NS], (j / C::NS) & 1, abort_flag, 485))) break;
        if (j + 1 < n_max && !(ok = mbar_wait_warp_cluster(&k_full[(j + 1) % C::NS], ((j + 1) / C::NS) & 1, abort_flag, 486))) break;
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (j < n_t[t]) {
            // one arrival a phase: wait for the last one's end first
            if (j > 0 && !(ok = mbar_wait_warp_cluster(&p_full[t], (j - 1) & 1, abort_flag, 487))) break;
            if (lane == 0) mbar_arrive(&p_full[t]);
            __syncwarp();
          }
      }
    }
  } else if (warp >= 12) {
    // ---------------------------------------------------------------- unpacking
    setmaxnreg_dec<C::REG_UNPACK>();
    const int uw = warp - 12;
    auto expand = [&](uint2 cd, uint32_t e, uint8_t* d0, uint8_t* d1, bool flip) {
      const uint32_t s = e4m3x2_to_f16(e * 0x0101u);
      uint32_t h[2][4];
      e2m1x8_to_f16(flip ? cd.y : cd.x, h[0]);
      e2m1x8_to_f16(flip ? cd.x : cd.y, h[1]);
#pragma unroll
      for (int k = 0; k < 8; ++k) h[k >> 2][k & 3] = hmul2(h[k >> 2][k & 3], s);
      *reinterpret_cast<uint4*>(d0) = make_uint4(h[0][0], h[0][1], h[0][2], h[0][3]);
      *reinterpret_cast<uint4*>(d1) = make_uint4(h[1][0], h[1][1], h[1][2], h[1][3]);
    };
    // K: a lane takes block lane % 8 of rows 16 apart; V: block lane % 4 of this CTA's half of rows 32 apart
    const int kb = lane & 7, kr = uw * 4 + (lane >> 3), kf = kb >> 2;
    const uint32_t k0 = kf * (C::HALF / 2) + sw128_offset(kr, ((kb & 3) * 2 + kf) * 8);
    const uint32_t k1 = kf * (C::HALF / 2) + sw128_offset(kr, ((kb & 3) * 2 + (kf ^ 1)) * 8);
    const int vb = lane & 3, vr = uw * 8 + (lane >> 2);
    const uint32_t v0 = sw128_offset(vr, vb * 16), v1 = sw128_offset(vr, vb * 16 + 8);
    auto done = [&](uint64_t* bar) {                          // this warp's part is written: tell the issuing CTA
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_release(cluster_addr(bar, 0));
    };
    bool ok = true;
    for (int j = 0; ok && j < n_max; ++j) {
      const int s = j % C::NS, u = j / C::NS;
      const uint8_t* st = sC + (j % C::NC) * C::CSTAGE;
      const int kk = key0 + j * C::BN;
      if (!(ok = mbar_wait_warp(&c_full[j % C::NC], (j / C::NC) & 1, abort_flag, 488))) break;
      if (u > 0 && !(ok = mbar_wait_warp(&k_empty[s], (u - 1) & 1, abort_flag, 489))) break;
      {
        uint2 cd[4];
        uint32_t e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          cd[i] = *reinterpret_cast<const uint2*>(st + (kr + 16 * i) * C::CB + kb * 8);
          e[i] = st[C::OFF_CKS + (kr + 16 * i) * C::SB + kb];
        }
        // behind the item's keys lies anything, a scale that is no number among it
        if (kk + C::BN > key_end) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (kk + rank * 64 + kr + 16 * i >= key_end) e[i] = 0;
        }
        uint8_t* tile = sK + s * C::HALF;
#pragma unroll
        for (int i = 0; i < 4; ++i) expand(cd[i], e[i], tile + k0 + i * 16 * 128, tile + k1 + i * 16 * 128, kf != 0);
      }
      done(&k_full[s]);
      if (u > 0 && !(ok = mbar_wait_warp(&v_empty[s], (u - 1) & 1, abort_flag, 490))) break;
      {
        uint2 cd[4];
        uint32_t e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          cd[i] = *reinterpret_cast<const uint2*>(st + C::OFF_CV + (vr + 32 * i) * C::CB + rank * 32 + vb * 8);
          e[i] = st[C::OFF_CVS + (vr + 32 * i) * C::SB + rank * 4 + vb];
        }
        if (kk + C::BN > key_end) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (kk + vr + 32 * i >= key_end) e[i] = 0;
        }
        uint8_t* tile = sV + s * C::HALF;
#pragma unroll
        for (int i = 0; i < 4; ++i) expand(cd[i], e[i], tile + v0 + i * 32 * 128, tile + v1 + i * 32 * 128, false);
      }
      done(&v_full[s]);
      if (lane == 0) mbar_arrive(&c_empty[j % C::NC]);
    }
  } else {
    // ---------------------------------------------------------------- softmax, thread = row
    setmaxnreg_inc<C::REG_SOFTMAX>();
    const int t = (warp - 4) >> 2;
    const int sub = warp & 3;
    const int row = sub * 32 + lane;
    const int r = row0 + t * 256 + rank * 128 + row;
    const uint32_t t_lane = static_cast<uint32_t>(sub * 32) << 16;
    const uint32_t t_s = tbase + t_lane + C::T_S + t * 128;
    const uint32_t t_o = tbase + t_lane + C::T_O + t * 128;
    const int n = t == 0 ? n_t[0] : n_t[1];
    const size_t th = static_cast<size_t>(first + r / p.G) * p.H + hkv * p.G + r % p.G;
    const float c2 = q4_query_row<D>(p, r < rows, th, sQ + t * C::QTILE, row);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster_release(cluster_addr(q_full, 0));
    const uint32_t hand = cluster_addr(&p_full[t], 0);
    const int lim = min(key_end, seen(r));
    const int lim_low = __reduce_min_sync(0xffffffffu, lim);  // keys below it are all the warp's rows'
    bool far = false;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    int j = 0;
    auto hand_over = [&] {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(hand);
    };
    for (const int plain = min(n, (lim_low - key0) / C::BN); !far && j < plain; ++j) {
      if (!(ok = mbar_wait_warp(&s_full[t], j & 1, abort_flag, 491))) break;
      tc_fence_after();
      q4_softmax_tile<D, true>(t_s, t_o, key0 + j * C::BN, lim, j == 0, c2, m, l, far);
      hand_over();
    }
    for (; ok && j < n; ++j) {
      if (!(ok = mbar_wait_warp(&s_full[t], j & 1, abort_flag, 491))) break;
      tc_fence_after();
      q4_softmax_tile<D, false>(t_s, t_o, key0 + j * C::BN, lim, j == 0, c2, m, l, far);
      hand_over();
    }
    if (ok && n > 0) {
      ok = mbar_wait_warp(&o_done[t], 0, abort_flag, 492);
      tc_fence_after();
    }
    if (ok && row0 + t * 256 < rows) {
      const int x = again(r), tok = first + x / p.G, head = hkv * p.G + x % p.G;
      q4_store_row<D>(p, t_o, n > 0, x < rows, static_cast<size_t>(tok) * p.H + head, tok, head, item, x - row0, c2, m, l);
    }
  }
  __syncwarp();
  tc_fence_before();
  if (warp == 0) cluster_wait();                              // (of the start)
  __syncthreads();
  cluster_sync();                                             // nothing of the other CTA reaches here any more
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tbase, C::TMEM_COLS);
  }
}

// Joins the parts of the items from ``whole`` on: WPR warps a row.
template <int D, int WPR>
__global__ void __launch_bounds__(128) attend_q4_tail_kernel(const __grid_constant__ Q4TParams p, int n_rows) {
  const int i = WPR > 1 ? blockIdx.x : blockIdx.x * 4 + (threadIdx.x >> 5);
  const int n = i / p.block_rows, row = i - n * p.block_rows;
  const Q4TItem x = q4_tile_item(p, p.whole + n * p.tail_splits);
  int first = x.b, nq = 1;
  if (i < n_rows && p.cu_q) {
    first = __ldg(p.cu_q + x.b);
    const int end = __ldg(p.cu_q + x.b + 1);
    nq = end - first;
    if (first < 0 || end < first || end > p.total_q || nq > p.max_q) nq = 0;   // reported
  }
  const int r = x.rb * p.block_rows + row;
  const bool some = i < n_rows && r < nq * p.G;
  const int tok = first + r / p.G, head = x.hkv * p.G + r % p.G;
  const size_t th = static_cast<size_t>(tok) * p.H + head;
  pdl_wait();
  q4_join<D, WPR>({p.part + (x.state + row) * (D + 2), static_cast<size_t>(p.block_rows) * (D + 2), 0, some ? p.tail_splits : 0},
                  WPR > 1 ? threadIdx.x >> 5 : 0, WPR, p.o + th * D, p.lse + (p.cu_q ? static_cast<size_t>(head) * p.total_q + tok : th), p.descale_v);
}

// Shares the items out to ``places`` (SMs, or pairs of them) at a time: all that fill them a whole
// number of times run whole, what is left over is split so that it fills them once more (4x1024 tokens
// over 16384 keys, 256 items on 76 pairs: 785 us whole, 717 us with the last 28 in two parts).  A part
// has at least 512 keys where nothing else runs (1x128 tokens over 4096 keys: 30 us, 59 whole; 35 with 1024
// keys a part against 31 at the time), else 1024 (8 prompts of up to 1024 tokens, 64 wide: 51 us whole, 62 us
// in parts of 640 at the time).  The states and their join cost some 15 us, so that at least nine key steps
// have to be saved (64 items over 1024 keys: 19 us whole, 28 in two; over 2048: 31 and 34; 16 items over
// 2048: 31 whole, 20 in four).  Returns the grid.
static long long share_tiles(Q4TParams& p, const PagedQ4Args& a, int places, int block_rows) {
  p.block_rows = block_rows;
  p.row_blocks = static_cast<int>((q4_rows(a.H, a.H_kv, a.max_seqlen_q) + block_rows - 1) / block_rows);
  const long long items = static_cast<long long>(a.n_seqs) * a.H_kv * p.row_blocks;
  p.whole = static_cast<int>(items);
  p.tail_splits = 1;
  if (a.n_splits) return items * a.n_splits;
  const int tail = static_cast<int>(items % places);
  const int s = tail ? min(places / tail, a.max_seqlen_k / (items < places ? 512 : 1024)) : 1;
  if (s < 2 || a.max_seqlen_k - a.max_seqlen_k / s < 9 * kQ4Step) return items;
  p.whole = static_cast<int>(items - tail);
  p.tail_splits = s;
  p.chunk = q4_chunk(a.max_seqlen_k, s);
  return p.whole + static_cast<long long>(tail) * s;
}

template <int D>
static cudaError_t launch_tail(const Q4TParams& p, long long grid, cudaStream_t stream) {
  if (p.tail_splits == 1) return cudaSuccess;
  const int rows = static_cast<int>((grid - p.whole) / p.tail_splits) * p.block_rows;
  const int warps = q4_join_warps(rows);
  log_launch("attend_q4_tail_kernel<D, WPR>", rows * warps / 4, 128, 0ull);
  return launch_join(warps == 1 ? attend_q4_tail_kernel<D, 1> : attend_q4_tail_kernel<D, 4>, rows * warps / 4, 128, stream, p, rows);
}

static cudaError_t launch_attend_q4_pair(Q4TParams& p, const PagedQ4Args& a, cudaStream_t stream) {
  using C = Q4PCfg;
  static int attr_done[64] = {0};
  cudaError_t e = ensure_smem_attr(attend_q4_pair_kernel, C::SMEM_BYTES, attr_done, C::THREADS, C::REG_NEED);
  if (e != cudaSuccess) return e;
  const long long pairs = share_tiles(p, a, kQ4MaxTailRows / (2 * kQ4TileRows), 2 * kQ4TileRows);
  const unsigned grid = static_cast<unsigned>(2 * pairs);
  log_launch("attend_q4_pair_kernel", grid, C::THREADS, static_cast<unsigned long long>(C::SMEM_BYTES));
  attend_q4_pair_kernel<<<grid, C::THREADS, C::SMEM_BYTES, stream>>>(p);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_tail<C::D>(p, pairs, stream) : e;
}

template <int D>
static cudaError_t launch_attend_q4_tile_d(const PagedQ4Args& a, cudaStream_t stream) {
  using C = Q4TCfg<D>;
  Q4TParams p{};
  p.q = static_cast<const uint16_t*>(a.q);
  p.kc = a.k_codes; p.ks = a.k_scales; p.vc = a.v_codes; p.vs = a.v_scales;
  p.o = static_cast<uint16_t*>(a.o); p.lse = a.lse; p.part = a.part;
  p.cu_q = a.cu_q; p.seqlens = a.seqlens; p.table = a.block_table;
  p.n_seqs = a.n_seqs; p.H = a.H; p.H_kv = a.H_kv; p.G = a.H / a.H_kv; p.total_q = a.total_q;
  p.max_q = a.max_seqlen_q; p.max_k = a.max_seqlen_k; p.causal = a.causal;
  p.num_blocks = a.num_blocks; p.block_size = a.block_size; p.max_blocks = a.max_blocks;
  p.piece = a.block_size % 64 == 0 ? 64 : a.block_size % 32 == 0 ? 32 : 16;
  p.n_splits = a.n_splits; p.chunk = a.chunk;
  p.score = a.scale * 1.4426950408889634f * a.descale_k;
  p.descale_v = a.descale_v;
  if (D == 128 && q4_rows(a.H, a.H_kv, a.max_seqlen_q) > kQ4TileRows) return launch_attend_q4_pair(p, a, stream);
  static int attr_done[64] = {0};
  cudaError_t e = ensure_smem_attr(attend_q4_tile_kernel<D>, C::SMEM_BYTES, attr_done, C::THREADS, C::REG_NEED);
  if (e != cudaSuccess) return e;
  const long long grid = share_tiles(p, a, kQ4MaxTailRows / kQ4TileRows, kQ4TileRows);
  log_launch("attend_q4_tile_kernel<D>", grid, C::THREADS, static_cast<unsigned long long>(C::SMEM_BYTES));
  attend_q4_tile_kernel<D><<<static_cast<unsigned>(grid), C::THREADS, C::SMEM_BYTES, stream>>>(p);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_tail<D>(p, grid, stream) : e;
}

cudaError_t launch_attend_q4_tile(const PagedQ4Args& a, cudaStream_t stream) {
  return a.d == 64 ? launch_attend_q4_tile_d<64>(a, stream) : launch_attend_q4_tile_d<128>(a, stream);
}

}  // namespace fa

FA_DEFINE_STATUS_FETCH(status_fetch_attend_q4_tile)
