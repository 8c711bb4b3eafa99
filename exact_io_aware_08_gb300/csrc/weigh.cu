// How much attention each cached token draws: w[k] = decay w[k] + sum over rows r of exp(scale q_r k - lse_r), where
// the rows of a key head are its query heads times the step's tokens, and a token's rows see the keys up to its own.
//
// Mathematics.  The attention's weights again, from its queries, keys and log-sum-exps, summed down the columns of
// S instead of along its rows: S^T = K Q^T puts a key on each lane of tensor memory, so that a thread adds up its own
// key's weights and nothing is exchanged.  scale s - lse is formed first and then multiplied by log2 e: the
// difference is small where the weight is not, and its rounding with it.  Products are exact, sums fp32, and each
// tile of 128 rows is summed before it is added.
//
// What bounds it.  2 d flops and an exponential a (row, key): with few rows the reading of K, with many the
// exponentials (32 a clock and SM: 1024 clocks for 256 keys times 128 rows, as many as the products take).
//
// Layout.  A CTA takes 256 keys at a time, in two tiles of 128, against tiles of up to 128 rows:
//   warp 0       copies K tiles, warp 2 tiles of Q (whole tokens, all heads of the group) and their lse.
//   warp 1       issues the products, up to two row tiles ahead of ...
//   warps 4 on   the sums, thread = key.
// FEW rows (one tile of them): Q stays, each CTA gets an equal share of all keys (Q4Share), and eight warps sum.
// Else a CTA keeps 256 keys and runs over a range of the rows that see them.  Sixteen warps sum, two threads a key with 64
// rows each (eight left most of a step to latencies: 1.6 us for 256 keys times 128 rows), and where there are too few
// pieces for the SMs the rows are divided into ranges whose sums a second kernel adds up, in order.
#include "fa_kernels.h"
#include "paged_tile.cuh"
#include "q4_share.h"

namespace fa {

template <int D, bool FEW>
struct WeighCfg {
  static constexpr int TILE = 128 * D * 2;
  static constexpr int CHUNK = 128 * 128;
  static constexpr int NK = D == 128 ? 2 : 4;                 // pairs of K tiles
  static constexpr int NQ = 3;                                // tiles of Q
  static constexpr int OFF_K = 0;
  static constexpr int OFF_Q = NK * 2 * TILE;
  static constexpr int OFF_LSE = OFF_Q + NQ * TILE;
  static constexpr int OFF_BAR = OFF_LSE + NQ * 128 * 4;
  // k_full[NK], k_empty[NK], q_full[NQ], l_full[NQ], q_empty[NQ], s_full[2][2], s_empty[2][2]
  static constexpr int NBAR = 2 * NK + 3 * NQ + 8;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 32 + 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget (227 KB per CTA)");
  static constexpr int HALVES = FEW ? 1 : 2;                  // threads of a key
  static constexpr int SUM_WARPS = 8 * HALVES;
  static constexpr int THREADS = 128 + 32 * SUM_WARPS;
  static constexpr uint32_t BAR_KEYS = 2;                     // named barriers of a key tile's warps
};

struct WeighParams {
  CUtensorMap tk, tq;
  PagedCache cache;
  const float* lse;
  float *weights, *part;                                      // part: sums of ranges [range][sequence][key head][pairs * 256]
  const int *cu, *seqlens, *weighed;
  int n_seqs, H, G, total, max_q, max_k;
  int tokens, rows;                                           // rows of a tile: ``tokens`` whole tokens
  int pairs, ranges, range;                                   // key pairs that max_k has; ranges of ``range`` row tiles
  float scale, decay;
};

// A stretch of work: key pairs [kt0, kt1) of a key head of a sequence, against row tiles [q0, q1).
struct WeighItem {
  int b, hkv, kt0, kt1, q0, q1, range, weighed;
  PagedSeq seq;
};

__device__ __forceinline__ int weigh_pairs(const PagedSeq& s) { return s.nq ? (s.len + 255) / 256 : 0; }

// First row tile whose tokens see a key of pair kt.
__device__ __forceinline__ int weigh_first(const WeighParams& p, const PagedSeq& s, int kt) { return max(0, kt * 256 - s.base()) / p.tokens; }

// Where a weight lies, or null (a page that is not there is reported by the copying warp).
__device__ __forceinline__ float* weigh_place(const WeighParams& p, int b, int hkv, int key) {
  const int blk = key / p.cache.block_size;
  const int page = __ldg(p.cache.table + static_cast<size_t>(b) * p.cache.max_blocks + blk);
  if (page < 0 || page >= p.cache.num_blocks) return nullptr;
  return p.weights + (static_cast<size_t>(page) * p.cache.H_kv + hkv) * p.cache.block_size + (key - blk * p.cache.block_size);
}

template <bool FEW>
struct WeighWalk {
  const WeighParams& p;
  int b, off, left;                                           // FEW: sequence, unit in it, units left; else: round
  PagedSeq seq;
  int pairs;

  __device__ __forceinline__ bool next(WeighItem& x) {
    if constexpr (!FEW) {
      // (range, key pair) by (range, key pair) over all sequences and heads, the last rows, which see the most, first;
      // dealt out in rounds
      const int per = p.n_seqs * p.cache.H_kv, n = per * p.pairs * p.ranges;
      for (; off * static_cast<int>(gridDim.x) < n; ++off) {
        const int item = pers_item(off, gridDim.x);
        if (item >= n) continue;
        const int i = item / per, w = item - i * per;
        x.hkv = w % p.cache.H_kv;
        x.b = w / p.cache.H_kv;
        x.range = p.ranges - 1 - i / p.pairs;
        x.kt0 = i % p.pairs;
        x.kt1 = x.kt0 + 1;
        x.seq = paged_seq(p.cu, p.seqlens, x.b, p.total, p.max_q, p.max_k, threadIdx.x == 0 && i == 0 && x.hkv == 0, 600);
        if (x.kt0 >= weigh_pairs(x.seq)) continue;
        x.q0 = max(x.range * p.range, weigh_first(p, x.seq, x.kt0));
        x.q1 = min((x.range + 1) * p.range, (x.seq.nq + p.tokens - 1) / p.tokens);
        if (x.q0 >= x.q1) continue;
        ++off;
        return true;
      }
      return false;
    } else {
      if (left <= 0) return false;
      while (off >= pairs * p.cache.H_kv) {
        if (++b >= p.n_seqs) return false;
        off = 0;
        seq = paged_seq(p.cu, p.seqlens, b, p.total, p.max_q, p.max_k, false, 0);
        pairs = weigh_pairs(seq);
      }
      x.b = b;
      x.seq = seq;
      x.hkv = off / pairs;
      x.kt0 = off - x.hkv * pairs;
      const int n = min(left, pairs - x.kt0);
      x.kt1 = x.kt0 + n;
      x.q0 = 0;
      x.q1 = 1;
      off += n;
      left -= n;
      return true;
    }
  }
};

// Adds up the weights of columns [lo, hi) of S^T, 32 columns from tensor memory at a time from ``from`` up to ``cols``.
template <bool MASKED>
__device__ __forceinline__ float weigh_tile(uint32_t t_s, const float* __restrict__ lse, int from, int cols, int lo, int hi, float scale) {
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  const float2 sc = make_float2(scale, scale), l2e = make_float2(1.4426950408889634f, 1.4426950408889634f);
#pragma unroll 1
  for (int c0 = from; c0 < cols; c0 += 32) {
    uint32_t rr[32];
    tmem_ld32(t_s + c0, rr);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      const float4 nl = *reinterpret_cast<const float4*>(lse + c0 + i);     // -lse
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = i + 2 * h;
        const float2 n = h ? make_float2(nl.z, nl.w) : make_float2(nl.x, nl.y);
        float2 x = fmul2(ffma2(make_float2(__uint_as_float(rr[c]), __uint_as_float(rr[c + 1])), sc, n), l2e);
        if constexpr (MASKED) {
          if (c0 + c < lo || c0 + c >= hi) x.x = -INFINITY;
          if (c0 + c + 1 < lo || c0 + c + 1 >= hi) x.y = -INFINITY;
        }
        sum[h] = fadd2(sum[h], make_float2(fast_exp2(x.x), fast_exp2(x.y)));
      }
    }
  }
  const float2 s = fadd2(sum[0], sum[1]);
  return s.x + s.y;
}

template <int D, bool FEW>
__global__ void __launch_bounds__(WeighCfg<D, FEW>::THREADS, 1) weigh_kernel(const __grid_constant__ WeighParams p) {
  using C = WeighCfg<D, FEW>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1k(smem_raw);
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sQ = smem + C::OFF_Q;
  float* sL = reinterpret_cast<float*>(smem + C::OFF_LSE);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* k_empty = k_full + C::NK;
  uint64_t* q_full = k_empty + C::NK;
  uint64_t* l_full = q_full + C::NQ;
  uint64_t* q_empty = l_full + C::NQ;
  uint64_t* s_full = q_empty + C::NQ;                         // [key tile][buffer]
  uint64_t* s_empty = s_full + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* start = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (warp == 0) {
    if (lane == 0) {
      for (int s = 0; s < C::NK; ++s) {
        mbar_init(&k_full[s], 2);                             // a key tile each
        mbar_init(&k_empty[s], 1);
      }
      for (int s = 0; s < C::NQ; ++s) {
        mbar_init(&q_full[s], 1);
        mbar_init(&l_full[s], 1);
        mbar_init(&q_empty[s], 1 + C::SUM_WARPS);             // the products, and the summing warps (lse)
      }
      for (int s = 0; s < 4; ++s) {
        mbar_init(&s_full[s], 1);
        mbar_init(&s_empty[s], 4 * C::HALVES);
      }
      *abort_flag = 0;
      fence_mbarrier_init();
    }
    if (lane < 2) tma_prefetch_desc(lane ? &p.tq : &p.tk);
    if constexpr (FEW) {
      // this CTA's share of the key pairs
      long long mine = 0;
      for (int i = lane; i < p.n_seqs; i += 32)
        mine += static_cast<long long>(weigh_pairs(paged_seq(p.cu, p.seqlens, i, p.total, p.max_q, p.max_k, blockIdx.x == 0, 601))) * p.cache.H_kv;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
      Q4Share sh;
      sh.set(mine, gridDim.x);
      const bool some = static_cast<int>(blockIdx.x) < sh.n && sh.total > 0;
      const long long u = some ? sh.begin(blockIdx.x) : -1;
      long long sum = 0, before = 0;
      int b = -1;
      for (int base = 0; base < p.n_seqs && u >= 0; base += 32) {
        const long long v = base + lane < p.n_seqs
            ? static_cast<long long>(weigh_pairs(paged_seq(p.cu, p.seqlens, base + lane, p.total, p.max_q, p.max_k, false, 0))) * p.cache.H_kv : 0;
        long long inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        const uint32_t beyond = __ballot_sync(0xffffffffu, sum + inc > u);
        if (beyond) {
          const int l = __ffs(beyond) - 1;
          b = base + l;
          before = sum + __shfl_sync(0xffffffffu, inc - v, l);
          break;
        }
        sum += __shfl_sync(0xffffffffu, inc, 31);
      }
      if (lane == 0) {
        start[0] = b;
        start[1] = b < 0 ? 0 : static_cast<int>(u - before);
        start[2] = b < 0 ? 0 : static_cast<int>(sh.begin(blockIdx.x + 1) - u);
      }
    }
  } else if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
  }
  if constexpr (!FEW) pdl_launch_dependents();
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  WeighWalk<FEW> walk{p, 0, 0, 0, {}, 0};
  if constexpr (FEW) {
    walk.b = start[0];
    walk.off = start[1];
    walk.left = start[2];
    if (walk.left > 0) {
      walk.seq = paged_seq(p.cu, p.seqlens, walk.b, p.total, p.max_q, p.max_k, false, 0);
      walk.pairs = weigh_pairs(walk.seq);
    }
  }
  WeighItem x;
  bool ok = true;
  int kc = 0, qc = 0, sc = 0;                                 // key pairs, row tiles, products (pairs of them) so far

  if (warp == 0) {
    // ---------------------------------------------------------------- copies of K
    PageWindow win;
    while (ok && walk.next(x)) {
      for (int kt = x.kt0; ok && kt < x.kt1; ++kt, ++kc) {
        const int s = kc % C::NK, u = kc / C::NK;
        if (u > 0 && !(ok = mbar_wait_warp(&k_empty[s], (u - 1) & 1, abort_flag, 610))) break;
        uint8_t* dst = sK + s * 2 * C::TILE;
        load_paged_tile<D>(p.cache, win, &p.tk, dst, &k_full[s], x.b, x.hkv, kt * 256, x.seq.len, 602);
        if (kt * 256 + 128 < x.seq.len)
          load_paged_tile<D>(p.cache, win, &p.tk, dst + C::TILE, &k_full[s], x.b, x.hkv, kt * 256 + 128, x.seq.len, 602);
        else if (lane == 0)
          mbar_arrive(&k_full[s]);
      }
    }
    for (int i = max(0, kc - C::NK); ok && i < kc; ++i) ok = mbar_wait_warp(&k_empty[i % C::NK], (i / C::NK) & 1, abort_flag, 611);
    if (!ok)
      for (int i = max(0, kc - C::NK); i < kc; ++i) mbar_wait_warp(&k_full[i % C::NK], (i / C::NK) & 1, nullptr, 612);
  } else if (warp == 2) {
    // ---------------------------------------------------------------- copies of Q and lse
    // (the next tile's lse is asked for before this one's is written: a load behind each wait bound the kernel, 126 us
    // for 1 x 4096 tokens)
    int token_of[4], head_of[4];                              // of the lane's four rows
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      token_of[i] = (i * 32 + lane) / p.G;
      head_of[i] = i * 32 + lane - token_of[i] * p.G;
    }
    while (ok && walk.next(x)) {
      auto ask = [&](int qt, float (&v)[4]) {
        const int n = min(p.tokens, x.seq.nq - qt * p.tokens);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = token_of[i] < n ? __ldg(p.lse + static_cast<size_t>(x.hkv * p.G + head_of[i]) * p.total + x.seq.first + qt * p.tokens + token_of[i])
                                 : -INFINITY;
      };
      float e[4];
      ask(x.q0, e);
      for (int qt = x.q0; ok && qt < x.q1; ++qt, ++qc) {
        const int s = qc % C::NQ, u = qc / C::NQ;
        if (u > 0 && !(ok = mbar_wait_warp(&q_empty[s], (u - 1) & 1, abort_flag, 613))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&q_full[s], p.rows * D * 2);
#pragma unroll
          for (int ch = 0; ch < D / 64; ++ch)
            tma_load_4d(sQ + s * C::TILE + ch * C::CHUNK, &p.tq, &q_full[s], ch * 64, 0, x.hkv, x.seq.first + qt * p.tokens);
        }
        __syncwarp();
        float next[4] = {0.f, 0.f, 0.f, 0.f};
        if (qt + 1 < x.q1) ask(qt + 1, next);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sL[s * 128 + i * 32 + lane] = e[i] == -INFINITY ? -INFINITY : -e[i];   // rows that see nothing weigh nothing
          e[i] = next[i];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&l_full[s]);
      }
    }
    for (int i = max(0, qc - C::NQ); ok && i < qc; ++i) ok = mbar_wait_warp(&q_empty[i % C::NQ], (i / C::NQ) & 1, abort_flag, 614);
    if (!ok)
      for (int i = max(0, qc - C::NQ); i < qc; ++i) mbar_wait_warp(&q_full[i % C::NQ], (i / C::NQ) & 1, nullptr, 615);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- products
    const uint32_t idesc = idesc_bf16_f32(128, (p.rows + 15) / 16 * 16, 0, 0);
    const uint64_t dk0 = smem_desc_sw128(smem_u32(sK), 0, 1024);
    const uint64_t dq0 = smem_desc_sw128(smem_u32(sQ), 0, 1024);
    while (ok && walk.next(x)) {
      for (int kt = x.kt0; ok && kt < x.kt1; ++kt, ++kc) {
        if (!(ok = mbar_wait_warp(&k_full[kc % C::NK], (kc / C::NK) & 1, abort_flag, 620))) break;
        for (int qt = x.q0; ok && qt < x.q1; ++qt, ++sc) {
          // FEW: the item's one tile serves all its keys
          const int q = FEW ? qc : qc++;
          ok = mbar_wait_warp(&q_full[q % C::NQ], (q / C::NQ) & 1, abort_flag, 621);
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            if (ok && sc >= 2) ok = mbar_wait_warp(&s_empty[2 * a + (sc & 1)], ((sc >> 1) - 1) & 1, abort_flag, 622);
            if (!ok) break;
            tc_fence_after();
            const uint64_t ad = desc_advance(dk0, ((kc % C::NK) * 2 + a) * C::TILE);
            const uint64_t bd = desc_advance(dq0, (q % C::NQ) * C::TILE);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t off = (ks >> 2) * C::CHUNK + (ks & 3) * 32;
              umma_ss_w(tbase + a * 256 + (sc & 1) * 128, desc_advance(ad, off), desc_advance(bd, off), idesc, ks > 0);
            }
            umma_commit_w(&s_full[2 * a + (sc & 1)]);
          }
          if (ok && !FEW) umma_commit_w(&q_empty[q % C::NQ]);
        }
        if (ok) umma_commit_w(&k_empty[kc % C::NK]);
      }
      if (FEW) {
        if (ok) umma_commit_w(&q_empty[qc % C::NQ]);
        ++qc;
      }
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- sums, thread = key (of half the rows)
    const int a = FEW ? (warp - 4) >> 2 : (warp - 4) >> 3, half = FEW ? 0 : (warp - 4) >> 2 & 1;
    const int sub = warp & 3;
    const uint32_t t_lane = tbase + (static_cast<uint32_t>(sub * 32) << 16) + a * 256;
    const int cols = (p.rows + 31) / 32 * 32;
    const int from = half * 64, to = FEW ? cols : half ? cols : min(64, cols);
    // After a failed wait the warps go on through all items without work: two halves meet once an item.
    while (walk.next(x)) {
      if constexpr (FEW) x.weighed = p.weighed ? __ldg(p.weighed + x.b) : x.seq.base();
      for (int kt = x.kt0; kt < x.kt1; ++kt) {
        const int key = kt * 256 + a * 128 + sub * 32 + lane;
        float* at = nullptr;
        float old = 0.f, sum = 0.f;
        if (FEW && key < x.seq.len) {
          at = weigh_place(p, x.b, x.hkv, key);
          if (at && key < x.weighed) old = *at * p.decay;
        }
        // the first row that sees the key, and that sees all of the warp's
        const int low = max(0, key - x.seq.base()) * p.G;
        const int low_all = max(0, key - lane + 31 - x.seq.base()) * p.G;
        for (int qt = x.q0; qt < x.q1; ++qt, ++sc) {
          const int q = FEW ? qc : qc++;
          const int r0 = qt * p.tokens * p.G, n = min(p.tokens, x.seq.nq - qt * p.tokens) * p.G;
          ok = ok && mbar_wait_warp(&l_full[q % C::NQ], (q / C::NQ) & 1, abort_flag, 630) &&
               mbar_wait_warp(&s_full[2 * a + (sc & 1)], (sc >> 1) & 1, abort_flag, 631);
          tc_fence_after();
          const uint32_t t_s = t_lane + (sc & 1) * 128;
          const float* lse = sL + (q % C::NQ) * 128;
          if (ok) {
            if (n == cols && low_all <= r0) sum += weigh_tile<false>(t_s, lse, from, to, 0, 0, p.scale);
            else sum += weigh_tile<true>(t_s, lse, from, min(to, (n + 31) / 32 * 32), low - r0, n, p.scale);
          }
          if (!FEW && qt + 1 == x.q1) {
            // the halves' sums, through a column that both have read
            tc_fence_before();
            named_bar_sync(C::BAR_KEYS + a, 256);
            tc_fence_after();
            if (half && ok) {
              tmem_st1(t_s, __float_as_uint(sum));
              tmem_wait_st();
            }
            tc_fence_before();
            named_bar_sync(C::BAR_KEYS + a, 256);
            tc_fence_after();
            if (!half && ok) {
              const uint32_t other = tmem_ld1(t_s);
              tmem_wait_ld();
              sum += __uint_as_float(other);
            }
          }
          if (!ok) continue;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&s_empty[2 * a + (sc & 1)]);
            if (!FEW) mbar_arrive(&q_empty[q % C::NQ]);
          }
        }
        if (FEW) {
          if (ok && at) *at = old + sum;
        } else if (ok && !half && key < x.seq.len) {
          if (p.ranges > 1) {
            p.part[((static_cast<size_t>(x.range) * p.n_seqs + x.b) * p.cache.H_kv + x.hkv) * p.pairs * 256 + key] = sum;
          } else {
            at = weigh_place(p, x.b, x.hkv, key);
            const int weighed = p.weighed ? __ldg(p.weighed + x.b) : x.seq.base();
            if (at) *at = (key < weighed ? *at * p.decay : 0.f) + sum;
          }
        }
      }
      if (FEW) {
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&q_empty[qc % C::NQ]);
        ++qc;
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

// Adds up the ranges' sums, thread = key.
__global__ void __launch_bounds__(256) weigh_join_kernel(const __grid_constant__ WeighParams p) {
  const int hkv = blockIdx.y % p.cache.H_kv, b = blockIdx.y / p.cache.H_kv, kt = blockIdx.x;
  const PagedSeq s = paged_seq(p.cu, p.seqlens, b, p.total, p.max_q, p.max_k, false, 0);
  const int key = kt * 256 + threadIdx.x;
  const int weighed = p.weighed ? __ldg(p.weighed + b) : s.base();
  float* at = s.nq && key < s.len ? weigh_place(p, b, hkv, key) : nullptr;
  pdl_wait();
  if (!at) return;
  const int tiles = (s.nq + p.tokens - 1) / p.tokens;
  const float* part = p.part + (static_cast<size_t>(b) * p.cache.H_kv + hkv) * p.pairs * 256 + key;
  const size_t stride = static_cast<size_t>(p.n_seqs) * p.cache.H_kv * p.pairs * 256;
  float sum = key < weighed ? *at * p.decay : 0.f, drawn = 0.f;
  for (int r = weigh_first(p, s, kt) / p.range; r * p.range < tiles; ++r) drawn += part[r * stride];
  *at = sum + drawn;
}

template <int D, bool FEW>
static cudaError_t launch_weigh_d(const WeighArgs& a, cudaStream_t stream) {
  using C = WeighCfg<D, FEW>;
  WeighParams p{};
  const int piece = paged_piece(a.block_size);
  const uint64_t rows = static_cast<uint64_t>(a.num_blocks) * a.block_size;
  const WeighSplit t = weigh_split(a.n_seqs, a.H, a.H_kv, a.max_q, a.max_k);
  p.G = a.H / a.H_kv;
  p.tokens = t.tokens;
  p.rows = p.tokens * p.G;
  if (!make_map_bf16_tok(&p.tk, a.k_cache, D, a.H_kv, rows, 64, piece) ||
      !make_map_bf16_group(&p.tq, a.q, D, p.G, a.H_kv, a.total, 64, p.G, p.tokens))
    return cudaErrorInvalidValue;
  p.cache = {a.block_table, a.H_kv, a.num_blocks, a.block_size, a.max_blocks, piece};
  p.lse = a.lse; p.weights = a.weights; p.part = a.part; p.cu = a.cu; p.seqlens = a.seqlens; p.weighed = a.weighed;
  p.n_seqs = a.n_seqs; p.H = a.H; p.total = a.total; p.max_q = a.max_q; p.max_k = a.max_k;
  p.scale = a.scale; p.decay = a.decay;
  p.pairs = (a.max_k + 255) / 256;
  p.ranges = t.ranges;
  p.range = t.range;
  static int attr_done[64] = {0};
  cudaError_t e = ensure_smem_attr(weigh_kernel<D, FEW>, C::SMEM_BYTES, attr_done);
  if (e != cudaSuccess) return e;
  const long long items = static_cast<long long>(a.n_seqs) * a.H_kv * p.pairs * p.ranges;
  const long long grid = min(static_cast<long long>(paged_sm_count()), items);
  log_launch("weigh_kernel<D, FEW>", static_cast<unsigned long long>(grid), C::THREADS, static_cast<unsigned long long>(C::SMEM_BYTES));
  weigh_kernel<D, FEW><<<static_cast<unsigned>(grid), C::THREADS, C::SMEM_BYTES, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.ranges == 1) return e;
  const dim3 blocks(static_cast<unsigned>(p.pairs), static_cast<unsigned>(a.n_seqs * a.H_kv));
  log_launch("weigh_join_kernel", static_cast<unsigned long long>(blocks.x) * blocks.y, 256, 0ull);
  return launch_join(weigh_join_kernel, blocks, 256, stream, p);
}

cudaError_t launch_weigh(const WeighArgs& a, cudaStream_t stream) {
  const bool few = weigh_split(a.n_seqs, a.H, a.H_kv, a.max_q, a.max_k).tokens >= a.max_q;
  if (a.d == 64) return few ? launch_weigh_d<64, true>(a, stream) : launch_weigh_d<64, false>(a, stream);
  return few ? launch_weigh_d<128, true>(a, stream) : launch_weigh_d<128, false>(a, stream);
}

}  // namespace fa

FA_DEFINE_STATUS_FETCH(status_fetch_weigh)
