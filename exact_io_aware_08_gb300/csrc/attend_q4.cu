// Attention over a paged key/value cache held in 4 bits: one query token a sequence (decode) or a
// few, any number of query heads to a key head.
//
// Mathematics.  The rows of a key head are the query heads that share it, times the step's query
// tokens.  Each row runs the online softmax over the sequence's keys, chunk by chunk where the key
// axis is split, and the chunks' states (m, l, o~) merge as for the bf16 decode.  Keys and values are
// code * scale * descale: code * scale is an exact fp16 number (q4.cuh), so the products run on fp16
// operands with fp32 sums, and the descales go into the score factor and the last division.  A query
// row is multiplied by a power of two that puts its largest element in [2^14, 2^15): in fp16 it keeps
// bf16's 8 bits down to 2^-28 of that element, and the power goes into the row's score factor.
// Weights are 2^(s - m) with a reference m at most 8 below the running maximum, so <= 2^8, rounded
// to fp16 for the product with V: off by at most 2^-11 each, and independently, below the output's
// own rounding to bf16; l sums the unrounded weights in fp32.
//
// What bounds it.  A key head's token is d + d/8 bytes (K and V), read once for up to kQ4Rows rows.
// At HBM rate that is some 42 elements a clock and SM, so what counts is the work of unpacking: per
// element 1/2 conversion, 1/2 multiplication with the scale, and 1/4 (V) to bring two keys' codes side
// by side.  Products are m16n8k16 warp instructions on operands unpacked in registers: the tensor
// core that reads shared memory would take a store and a load of every unpacked element first.
//   S^T = K Q^T:  A = 16 keys x 16 elements, B = 8 rows.  The order of d in a contraction is free, so
//                 lane c of a quad takes d/4 consecutive elements of its keys: one load each.
//   O^T = V^T P^T: A = 16 elements x 16 keys.  The lanes of row r take d/8 consecutive elements, and
//                 P^T comes from the S^T accumulators by an 8x8 transpose in registers.
// Keys sit in the S^T tile in the order kappa(r), which spreads the V loads over all banks.
//
// Layout.  Four warps compute, 16 keys each of a 64-key stage; a fifth copies stages by TMA (codes,
// swizzled) and bulk copies (scales) into a ring that runs on across work items.  Items are
// (sequence, key head, row block, chunk).
#include "fa_kernels.h"
#include "q4.cuh"

namespace fa {

template <int D, int NT>
struct Q4Cfg {
  static constexpr int KEYS = kDecodeKeyStep;                 // 64
  static constexpr int ROWS = 8 * NT;
  static constexpr int CB = D / 2;                            // code bytes of a row
  static constexpr int SB = D / 16;                           // scale bytes of a row
  static constexpr int CODES = KEYS * CB;
  static constexpr int SCALES = KEYS * SB;
  static constexpr int OFF_V = CODES;
  static constexpr int OFF_KS = 2 * CODES;
  static constexpr int OFF_VS = OFF_KS + SCALES;
  static constexpr int STAGE = (OFF_VS + SCALES + 1023) / 1024 * 1024;
  static constexpr int NST = 4;
  static constexpr int WARPS = 4;
  static constexpr int THREADS = 32 * (WARPS + 1);
  static constexpr int MROW = D + 4;                          // floats of a merge row (bank spread)
  static constexpr int OFF_MERGE = NST * STAGE;               // WARPS x ROWS x MROW
  static constexpr int OFF_ML = OFF_MERGE + WARPS * ROWS * MROW * 4;   // WARPS x ROWS x (m, l)
  static constexpr int OFF_BAR = OFF_ML + WARPS * ROWS * 8;
  static constexpr int SMEM_BYTES = OFF_BAR + (2 * NST + 2) * 8 + 16 + 1024;
  static constexpr int KS = D / 16;                           // k-steps of S^T
  static constexpr int MT = D / 16;                           // element tiles of O^T
  static constexpr int MIN_CTAS = NT == 1 ? 4 : 3;
};

struct Q4Params {
  CUtensorMap tk, tv;
  const uint16_t* q;
  const uint8_t *ks, *vs;
  uint16_t* o;
  float *lse, *part;
  const int *cu_q, *seqlens, *table;
  int n_seqs, H, H_kv, G, total_q, max_q, max_k, causal, num_blocks, block_size, max_blocks, piece;
  int n_splits, chunk, row_blocks, n_items;
  float score, descale_v;                                     // scale * log2 e * descale_k
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Work of one item, the same for every thread that asks.
struct Q4Item {
  int b, hkv, rb, split, first, nq, len, key0, key_end;   // key_end: keys any row of the block sees
  bool write;                                             // rows to write (false: no rows, or reported)
};

__device__ __forceinline__ Q4Item q4_item(const Q4Params& p, int item, int rows_per_block, bool report) {
  Q4Item x;
  x.split = item % p.n_splits;
  item /= p.n_splits;
  x.rb = item % p.row_blocks;
  item /= p.row_blocks;
  x.hkv = item % p.H_kv;
  x.b = item / p.H_kv;
  x.first = x.b;
  x.nq = 1;
  x.write = true;
  x.len = __ldg(p.seqlens + x.b);
  if (p.cu_q) {
    x.first = __ldg(p.cu_q + x.b);
    const int end = __ldg(p.cu_q + x.b + 1);
    x.nq = end - x.first;
    if (x.first < 0 || end < x.first || end > p.total_q || x.nq > p.max_q) {
      if (report) report_device_error(FA_DEV_BAD_CONFIG, 420);
      x.nq = 0;
    }
  }
  if (x.len < 0 || x.len > p.max_k) {
    if (report) report_device_error(FA_DEV_BAD_CONFIG, 421);
    x.len = 0;
  }
  const int rows = x.nq * p.G;
  const int row0 = x.rb * rows_per_block;
  x.write = row0 < rows;
  int seen = x.len;
  if (p.causal) seen = max(0, x.len - x.nq + (min(rows, row0 + rows_per_block) - 1) / p.G + 1);
  x.key0 = x.split * p.chunk;
  x.key_end = x.write ? min(x.key0 + p.chunk, seen) : 0;
  return x;
}

template <int D>
__device__ __forceinline__ uint32_t code_offset(int row, int chunk) {   // 16-byte chunk of a row, swizzled
  return D == 128 ? row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4) : row * 32 + ((chunk ^ ((row >> 2) & 1)) << 4);
}

template <int D, int NT>
__global__ void __launch_bounds__(Q4Cfg<D, NT>::THREADS, Q4Cfg<D, NT>::MIN_CTAS)
attend_q4_kernel(const __grid_constant__ Q4Params p) {
  using C = Q4Cfg<D, NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1k(smem_raw);
  float* merge = reinterpret_cast<float*>(smem + C::OFF_MERGE);
  float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::NST;
  uint64_t* mrg = empty + C::NST;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_BAR + (2 * C::NST + 2) * 8);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], C::WARPS);
    }
    mbar_init(&mrg[0], C::WARPS);
    mbar_init(&mrg[1], C::WARPS);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  __syncthreads();

  if (warp == C::WARPS) {
    // ---------------------------------------------------------------- copies
    // Lane j copies piece j (``piece`` keys of one page) of a stage.
    const int pieces = C::KEYS / p.piece;
    uint32_t g = 0;
    bool ok = true;
    for (int item = blockIdx.x; ok && item < p.n_items; item += gridDim.x) {
      const Q4Item x = q4_item(p, item, C::ROWS, lane == 0);
      int window = -1, tab = 0;                              // 32 table entries from block ``window`` on
      for (int kk = x.key0; kk < x.key_end; kk += C::KEYS, ++g) {
        const int s = g % C::NST;
        const uint32_t n = g / C::NST;
        // the stage's pages: at most four table entries, kept 32 at a time
        const int blk0 = kk / p.block_size;
        const int last = (min(kk + C::KEYS, x.key_end) - 1) / p.block_size;
        if (window < 0 || last >= window + 32) {
          window = blk0;
          const int blk = window + lane;
          // entries that hold the item's keys only
          tab = blk <= (x.key_end - 1) / p.block_size ? __ldg(p.table + static_cast<size_t>(x.b) * p.max_blocks + blk) : 0;
        }
        const int key = kk + (lane < pieces ? lane : 0) * p.piece;
        const int blk = key / p.block_size;
        int page = __shfl_sync(0xffffffffu, tab, (blk - window) & 31);
        const bool mine = lane < pieces && key < x.key_end;
        if (mine && (page < 0 || page >= p.num_blocks)) {
          report_device_error(FA_DEV_BAD_CONFIG, 422);
          page = 0;                                          // stays in bounds; the result is reported invalid
        }
        if (n > 0 && !(ok = mbar_wait_warp(&empty[s], (n - 1) & 1, abort_flag, 430))) break;
        const int live = __popc(__ballot_sync(0xffffffffu, mine));
        if (lane == 0) mbar_arrive_expect_tx(&full[s], live * p.piece * 2 * (C::CB + C::SB));
        __syncwarp();
        if (mine) {
          uint8_t* st = smem + s * C::STAGE;
          const int row = (page * p.H_kv + x.hkv) * p.block_size + (key - blk * p.block_size);
          const int at = lane * p.piece;
          tma_load_2d(st + at * C::CB, &p.tk, &full[s], 0, row);
          tma_load_2d(st + C::OFF_V + at * C::CB, &p.tv, &full[s], 0, row);
          bulk_load(st + C::OFF_KS + at * C::SB, p.ks + static_cast<size_t>(row) * C::SB, p.piece * C::SB, &full[s]);
          bulk_load(st + C::OFF_VS + at * C::SB, p.vs + static_cast<size_t>(row) * C::SB, p.piece * C::SB, &full[s]);
        }
        __syncwarp();
      }
    }
    if (!ok) {
      // drain the copies already issued (at most NST stages outstanding)
      for (uint32_t x = (g > C::NST ? g - C::NST : 0); x < g; ++x) mbar_wait_warp(&full[x % C::NST], (x / C::NST) & 1, nullptr, 431);
    }
  } else {
    // ---------------------------------------------------------------- products
    const int r = lane >> 2, c = lane & 3;
    const int ra = warp * 16 + (r ^ (((r >> 1) ^ (r >> 2)) & 1));     // key kappa(r) of the warp's 16; + 8
    const int e = 2 * c;
    const int v0 = warp * 16 + (e ^ (((e >> 1) ^ (e >> 2)) & 1));     // keys kappa(2c) and kappa(2c + 1)
    const int v1 = v0 ^ 1;
    uint32_t g = 0, it = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < p.n_items; item += gridDim.x) {
      const Q4Item x = q4_item(p, item, C::ROWS, false);
      if (!x.write) continue;
      const int rows = x.nq * p.G;
      // Queries: lane (r, c) holds row r's elements [c d/4, (c+1) d/4) as B operands; the factors and
      // key limits of rows 2c and 2c + 1, whose scores the lane gets, come from the lanes that hold them.
      uint32_t qb[NT][C::KS][2];
      float fac[NT][2];
      int vis[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int row = x.rb * C::ROWS + 8 * n + r;
        const int i = row / p.G;
        uint4 w[D / 32];
        float big = 0.f;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          w[j] = make_uint4(0u, 0u, 0u, 0u);
          if (row < rows) {
            const size_t at = (static_cast<size_t>(x.first + i) * p.H + x.hkv * p.G + (row - i * p.G)) * D;
            w[j] = __ldg(reinterpret_cast<const uint4*>(p.q + at + c * (D / 4)) + j);
          }
          const uint32_t ww[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) big = fmaxf(big, fmaxf(fabsf(bf16_lo(ww[k])), fabsf(bf16_hi(ww[k]))));
        }
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // exponent of the largest element, so that 2^(14 - ex) and its inverse are normal numbers
        const int ex = big == 0.f ? 14 : max(-100, static_cast<int>(__float_as_uint(big) >> 23) - 127);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - ex) << 23);
        const float f = p.score * __uint_as_float(static_cast<uint32_t>(127 - 14 + ex) << 23);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const uint32_t ww[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            qb[n][2 * j + (k >> 1)][k & 1] = pack_f16x2(bf16_lo(ww[k]) * up, bf16_hi(ww[k]) * up);
        }
        const int seen = p.causal ? x.len - x.nq + min(i, x.nq - 1) + 1 : x.len;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          fac[n][k] = __shfl_sync(0xffffffffu, f, (2 * c + k) * 4);
          vis[n][k] = __shfl_sync(0xffffffffu, seen, (2 * c + k) * 4);
        }
      }
      float m[NT][2], l[NT][2], o[NT][C::MT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int t = 0; t < C::MT; ++t) o[n][t][0] = o[n][t][1] = o[n][t][2] = o[n][t][3] = 0.f;
      }

      for (int kk = x.key0; ok && kk < x.key_end; kk += C::KEYS, ++g) {
        const int s = g % C::NST;
        if (!(ok = mbar_wait_warp(&full[s], (g / C::NST) & 1, abort_flag, 432))) break;
        const uint8_t* st = smem + s * C::STAGE;
        // S^T: this warp's 16 keys against the rows
        float sc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
        {
          uint32_t wa[D / 32], wb[D / 32];                     // the two keys' codes, 8 a word
          uint32_t sa[2], sb[2];                               // scales of their blocks, doubled
          if constexpr (D == 128) {
            const uint4 a = *reinterpret_cast<const uint4*>(st + code_offset<D>(ra, c));
            const uint4 b = *reinterpret_cast<const uint4*>(st + code_offset<D>(ra + 8, c));
            wa[0] = a.x; wa[1] = a.y; wa[2] = a.z; wa[3] = a.w;
            wb[0] = b.x; wb[1] = b.y; wb[2] = b.z; wb[3] = b.w;
            const uint32_t ea = e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(st + C::OFF_KS + ra * C::SB + 2 * c));
            const uint32_t eb = e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(st + C::OFF_KS + (ra + 8) * C::SB + 2 * c));
            sa[0] = __byte_perm(ea, ea, 0x1010); sa[1] = __byte_perm(ea, ea, 0x3232);
            sb[0] = __byte_perm(eb, eb, 0x1010); sb[1] = __byte_perm(eb, eb, 0x3232);
          } else {
            const uint2 a = *reinterpret_cast<const uint2*>(st + code_offset<D>(ra, c >> 1) + (c & 1) * 8);
            const uint2 b = *reinterpret_cast<const uint2*>(st + code_offset<D>(ra + 8, c >> 1) + (c & 1) * 8);
            wa[0] = a.x; wa[1] = a.y;
            wb[0] = b.x; wb[1] = b.y;
            sa[0] = e4m3x2_to_f16(st[C::OFF_KS + ra * C::SB + c] * 0x0101u);
            sb[0] = e4m3x2_to_f16(st[C::OFF_KS + (ra + 8) * C::SB + c] * 0x0101u);
          }
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            uint32_t a[4], b[4];
            e2m1x8_to_f16(wa[j], a);
            e2m1x8_to_f16(wb[j], b);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              a[k] = hmul2(a[k], sa[D == 128 ? j >> 1 : 0]);
              b[k] = hmul2(b[k], sb[D == 128 ? j >> 1 : 0]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma_f16(sc[n], a[0], b[0], a[1], b[1], qb[n][2 * j][0], qb[n][2 * j][1]);
              mma_f16(sc[n], a[2], b[2], a[3], b[3], qb[n][2 * j + 1][0], qb[n][2 * j + 1][1]);
            }
          }
        }
        // scores of keys kk + ra and kk + ra + 8 for rows 2c, 2c + 1, in the log2 domain
        uint32_t pb[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float t[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            t[k] = sc[n][k] * fac[n][k & 1];
            if (kk + ra + 8 * (k >> 1) >= min(x.key_end, vis[n][k & 1])) t[k] = -INFINITY;
          }
          const float t0 = fmaxf(t[0], t[2]), t1 = fmaxf(t[1], t[3]);
          if (__any_sync(0xffffffffu, t0 > m[n][0] + 8.f || t1 > m[n][1] + 8.f)) {
            // a row's maximum grew by more than 2^8: move its reference
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float top = k ? t1 : t0;
#pragma unroll
              for (int off = 4; off <= 16; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
              const float m_new = fmaxf(m[n][k], top);
              const float alpha = m_new == -INFINITY ? 1.f : fast_exp2(m[n][k] - m_new);
              m[n][k] = m_new;
              l[n][k] *= alpha;
#pragma unroll
              for (int i = 0; i < C::MT; ++i) {
                o[n][i][k] *= alpha;
                o[n][i][2 + k] *= alpha;
              }
            }
          }
          const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0];
          const float m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
          const float p0 = fast_exp2(t[0] - m0), p1 = fast_exp2(t[1] - m1);
          const float p2 = fast_exp2(t[2] - m0), p3 = fast_exp2(t[3] - m1);
          l[n][0] += p0 + p2;
          l[n][1] += p1 + p3;
          pb[n][0] = transpose8x8(pack_f16x2(p0, p1));
          pb[n][1] = transpose8x8(pack_f16x2(p2, p3));
        }
        // O^T += V^T P^T
        {
          const uint8_t* sv = st + C::OFF_V;
          const uint8_t* vs = st + C::OFF_VS;
          constexpr int W = D / 64;                            // words of a row's d/8 elements
          constexpr int SR = D == 128 ? 1 : 2;                 // lanes' rows that share a scale block
          uint32_t lo[2][W], hi[2][W], sl[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int k0 = v0 + 8 * h, k1 = v1 + 8 * h;
            uint32_t a[W], b[W];
            if constexpr (D == 128) {
              const uint2 x0 = *reinterpret_cast<const uint2*>(sv + code_offset<D>(k0, r >> 1) + (r & 1) * 8);
              const uint2 x1 = *reinterpret_cast<const uint2*>(sv + code_offset<D>(k1, r >> 1) + (r & 1) * 8);
              a[0] = x0.x; a[1] = x0.y; b[0] = x1.x; b[1] = x1.y;
            } else {
              a[0] = *reinterpret_cast<const uint32_t*>(sv + code_offset<D>(k0, r >> 2) + (r & 3) * 4);
              b[0] = *reinterpret_cast<const uint32_t*>(sv + code_offset<D>(k1, r >> 2) + (r & 3) * 4);
            }
            uint32_t e0 = vs[k0 * C::SB + r / SR], e1 = vs[k1 * C::SB + r / SR];
            // rows past the end hold anything, a scale that is no number among it: 0 * NaN is NaN
            if (kk + k0 >= x.key_end) e0 = 0;
            if (kk + k1 >= x.key_end) e1 = 0;
            sl[h] = e4m3x2_to_f16(e0 | (e1 << 8));
#pragma unroll
            for (int j = 0; j < W; ++j) {
              // byte i: the two keys' even (lo) or odd (hi) elements 2i (+1) of the word
              lo[h][j] = (a[j] & 0x0f0f0f0fu) | ((b[j] << 4) & 0xf0f0f0f0u);
              hi[h][j] = ((a[j] >> 4) & 0x0f0f0f0fu) | (b[j] & 0xf0f0f0f0u);
            }
          }
#pragma unroll
          for (int j = 0; j < W; ++j) {
            uint32_t a0[4], a1[4], a2[4], a3[4];
            e2m1x8_to_f16(lo[0][j], a0);
            e2m1x8_to_f16(hi[0][j], a1);
            e2m1x8_to_f16(lo[1][j], a2);
            e2m1x8_to_f16(hi[1][j], a3);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t w0 = hmul2(a0[i], sl[0]), w1 = hmul2(a1[i], sl[0]);
              const uint32_t w2 = hmul2(a2[i], sl[1]), w3 = hmul2(a3[i], sl[1]);
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_f16(o[n][4 * j + i], w0, w1, w2, w3, pb[n][0], pb[n][1]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
      }
      if (!ok) break;

      // The warps' states of this chunk.  o[n][t]: rows 2c, 2c + 1 at elements r d/8 + 2t (+1), kept at
      // position 16 t + 2 r (+1) of the merge row.
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int off = 4; off <= 16; off <<= 1) l[n][k] += __shfl_xor_sync(0xffffffffu, l[n][k], off);
          float* dst = merge + (warp * C::ROWS + 8 * n + 2 * c + k) * C::MROW;
#pragma unroll
          for (int t = 0; t < C::MT; ++t)
            *reinterpret_cast<float2*>(dst + 16 * t + 2 * r) = make_float2(o[n][t][k], o[n][t][2 + k]);
          if (r == 0) ml[warp * C::ROWS + 8 * n + 2 * c + k] = make_float2(m[n][k], l[n][k]);
        }
      }
      if (!(ok = warps_sync(&mrg[0], it & 1, abort_flag, 433))) break;
      for (int idx = threadIdx.x; idx < C::ROWS * (D / 2); idx += 32 * C::WARPS) {
        const int n = idx / (D / 2), dd = 2 * (idx % (D / 2));
        const int row = x.rb * C::ROWS + n;
        if (row >= rows) break;
        const int pos = D == 128 ? ((dd >> 1) & 7) * 16 + (dd >> 4) * 2 : ((dd >> 1) & 3) * 16 + (dd >> 3) * 2;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) M = fmaxf(M, ml[w * C::ROWS + n].x);
        float a0 = 0.f, a1 = 0.f, L = 0.f;
        if (M != -INFINITY) {
#pragma unroll
          for (int w = 0; w < C::WARPS; ++w) {
            const float2 st = ml[w * C::ROWS + n];
            const float wt = fast_exp2(st.x - M);
            const float2 v = *reinterpret_cast<const float2*>(merge + (w * C::ROWS + n) * C::MROW + pos);
            a0 = fmaf(wt, v.x, a0);
            a1 = fmaf(wt, v.y, a1);
            L = fmaf(wt, st.y, L);
          }
        }
        const int i = row / p.G;
        const int tok = x.first + i, head = x.hkv * p.G + (row - i * p.G);
        const size_t th = static_cast<size_t>(tok) * p.H + head;
        if (p.n_splits == 1) {
          const bool none = M == -INFINITY;                    // a row that sees no key
          const float inv = none ? 0.f : p.descale_v / L;
          *reinterpret_cast<uint32_t*>(p.o + th * D + dd) = pack_bf16x2(none ? 0.f : a0 * inv, none ? 0.f : a1 * inv);
          if (dd == 0)
            p.lse[p.cu_q ? static_cast<size_t>(head) * p.total_q + tok : th] = none ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
        } else {
          float* dst = p.part + (th * p.n_splits + x.split) * (D + 2);
          *reinterpret_cast<float2*>(dst + dd) = make_float2(a0, a1);
          if (dd == 0) *reinterpret_cast<float2*>(dst + D) = make_float2(M, L);
        }
      }
      if (!(ok = warps_sync(&mrg[1], it & 1, abort_flag, 434))) break;
      ++it;
    }
  }
  __syncwarp();
  __syncthreads();
}

// Joins a row's chunk states: one warp a row.
template <int D>
__global__ void __launch_bounds__(128) attend_q4_merge_kernel(const float* __restrict__ part, uint16_t* __restrict__ o,
                                                             float* __restrict__ lse, const int* __restrict__ cu_q,
                                                             int n_seqs, int H, int total_q, int n_splits, float descale_v) {
  const long long th = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (th >= static_cast<long long>(total_q) * H) return;
  const int tok = static_cast<int>(th / H), head = static_cast<int>(th - static_cast<long long>(tok) * H);
  if (cu_q && tok >= __ldg(cu_q + n_seqs)) return;             // rows behind the last sequence stay as they are
  const float* base = part + static_cast<size_t>(th) * n_splits * (D + 2);
  float M = -INFINITY;
  for (int c = lane; c < n_splits; c += 32) M = fmaxf(M, base[static_cast<size_t>(c) * (D + 2) + D]);
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  constexpr int V = D / 32;
  float acc[V], L = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  for (int c = 0; c < n_splits; ++c) {
    const float* st = base + static_cast<size_t>(c) * (D + 2);
    const float mc = st[D];
    if (mc == -INFINITY) continue;                             // empty chunk: weight 0
    const float wt = fast_exp2(mc - M);
    L = fmaf(wt, st[D + 1], L);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 v = *reinterpret_cast<const float2*>(st + 64 * i + 2 * lane);
      acc[2 * i] = fmaf(wt, v.x, acc[2 * i]);
      acc[2 * i + 1] = fmaf(wt, v.y, acc[2 * i + 1]);
    }
  }
  const bool none = M == -INFINITY;
  const float inv = none ? 0.f : descale_v / L;
#pragma unroll
  for (int i = 0; i < V / 2; ++i)
    *reinterpret_cast<uint32_t*>(o + static_cast<size_t>(th) * D + 64 * i + 2 * lane) =
        pack_bf16x2(none ? 0.f : acc[2 * i] * inv, none ? 0.f : acc[2 * i + 1] * inv);
  if (lane == 0)
    lse[cu_q ? static_cast<size_t>(head) * total_q + tok : static_cast<size_t>(th)] =
        none ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

static int q4_sm_count() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 152;
  if (dev < 64 && cached[dev]) return cached[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 152;
  if (dev < 64) cached[dev] = n;
  return n;
}

template <int D, int NT>
static cudaError_t launch_attend_q4_d(const PagedQ4Args& a, cudaStream_t stream) {
  using C = Q4Cfg<D, NT>;
  Q4Params p{};
  const uint64_t rows = static_cast<uint64_t>(a.num_blocks) * a.H_kv * a.block_size;
  // a stage's 64 keys in pieces that never cross a page
  p.piece = a.block_size % 64 == 0 ? 64 : a.block_size % 32 == 0 ? 32 : 16;
  const CUtensorMapSwizzle sw = D == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
  if (!make_map_u8_2d(&p.tk, a.k_codes, C::CB, rows, p.piece, sw) || !make_map_u8_2d(&p.tv, a.v_codes, C::CB, rows, p.piece, sw))
    return cudaErrorInvalidValue;
  p.q = static_cast<const uint16_t*>(a.q); p.ks = a.k_scales; p.vs = a.v_scales;
  p.o = static_cast<uint16_t*>(a.o); p.lse = a.lse; p.part = a.part;
  p.cu_q = a.cu_q; p.seqlens = a.seqlens; p.table = a.block_table;
  p.n_seqs = a.n_seqs; p.H = a.H; p.H_kv = a.H_kv; p.G = a.H / a.H_kv; p.total_q = a.total_q;
  p.max_q = a.max_seqlen_q; p.max_k = a.max_seqlen_k; p.causal = a.causal;
  p.num_blocks = a.num_blocks; p.block_size = a.block_size; p.max_blocks = a.max_blocks;
  p.n_splits = a.n_splits; p.chunk = a.chunk;
  p.row_blocks = static_cast<int>((static_cast<long long>(p.G) * a.max_seqlen_q + C::ROWS - 1) / C::ROWS);
  p.n_items = static_cast<int>(static_cast<long long>(a.n_seqs) * a.H_kv * p.row_blocks * a.n_splits);
  p.score = a.scale * 1.4426950408889634f * a.descale_k;
  p.descale_v = a.descale_v;
  static int attr_done[64] = {0};
  cudaError_t e = ensure_smem_attr(attend_q4_kernel<D, NT>, C::SMEM_BYTES, attr_done);
  if (e != cudaSuccess) return e;
  const int grid = min(p.n_items, C::MIN_CTAS * q4_sm_count());
  log_launch("attend_q4_kernel<D, NT>", static_cast<unsigned long long>(grid), C::THREADS, static_cast<unsigned long long>(C::SMEM_BYTES));
  attend_q4_kernel<D, NT><<<grid, C::THREADS, C::SMEM_BYTES, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
static cudaError_t launch_attend_q4_merge(const PagedQ4Args& a, cudaStream_t stream) {
  const long long warps = static_cast<long long>(a.total_q) * a.H;
  const unsigned blocks = static_cast<unsigned>((warps + 3) / 4);
  log_launch("attend_q4_merge_kernel<D>", blocks, 128, 0ull);
  attend_q4_merge_kernel<D><<<blocks, 128, 0, stream>>>(a.part, static_cast<uint16_t*>(a.o), a.lse, a.cu_q, a.n_seqs, a.H,
                                                        a.total_q, a.n_splits, a.descale_v);
  return cudaGetLastError();
}

cudaError_t launch_attend_q4(const PagedQ4Args& a, cudaStream_t stream) {
  cudaError_t e;
  if (q4_use_tiles(a.H, a.H_kv, a.max_seqlen_q)) {
    e = launch_attend_q4_tile(a, stream);
  } else {
    // 8 rows suffice for up to 8 query heads a key head at one token; else 16 share the unpacked keys
    const bool small = q4_rows(a.H, a.H_kv, a.max_seqlen_q) <= 8;
    if (a.d == 64) e = small ? launch_attend_q4_d<64, 1>(a, stream) : launch_attend_q4_d<64, 2>(a, stream);
    else e = small ? launch_attend_q4_d<128, 1>(a, stream) : launch_attend_q4_d<128, 2>(a, stream);
  }
  if (e != cudaSuccess || a.n_splits == 1) return e;
  return a.d == 64 ? launch_attend_q4_merge<64>(a, stream) : launch_attend_q4_merge<128>(a, stream);
}

}  // namespace fa

FA_DEFINE_STATUS_FETCH(status_fetch_attend_q4)
