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
// Weights are 2^(s - m) with a reference m 7 to 15 below the running maximum, so <= 2^15, rounded to
// fp16 for the product with V: off by at most 2^-11 of themselves, and independently, or half of fp16's
// smallest step, 2^-25, which is at most 2^-32 of the weight that the maximum has.  (A reference at the
// maximum left fp16's upper half unused and lost what lies 2^-25 below a row's largest weight; keys that
// many, behind one that draws most of the attention, add up.)  Bf16 weights would keep the range and
// be off by 2^-9 each.  l sums the unrounded weights in fp32.
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
// Layout.  One CTA an SM, of three or four teams.  A team's four warps compute, 32 keys each of a
// 128-key stage, 16 at a time; a fifth copies stages by TMA (codes, swizzled) and bulk copies (scales,
// query rows) into a ring that runs on across work items, and its registers go to the others.  Each
// team gets an equal share of all sequences' key steps (Q4Share), whatever their lengths; with an
// explicit split count the items are (sequence, key head, row block, chunk).
//
// Measured on the GPU, without the call's host time: 64 x 32768 tokens, 4 query heads a key head: 384 us,
// 2.42 GB at 6.3 TB/s (93% of the copy rate).  Short calls are bound by latencies: 4 us from the launch to
// the first keys (place in the work, query rows, page table, stage: each waits for the last), 1.4 us a step,
// 1.3 to leave a row block, 3 for the join behind; 1 x 1000 tokens 7.7 us.
#include "fa_kernels.h"
#include "q4.cuh"
#include "q4_share.h"

namespace fa {

constexpr float kNone = -3.402823466e38f;                     // -FLT_MAX: a reference below every score

template <int D, int NT>
struct Q4Cfg {
  static constexpr int KEYS = kQ4Step;                        // 128: 32 a warp, in two halves
  static constexpr int ROWS = 8 * NT;
  static constexpr int CB = D / 2;                            // code bytes of a row
  static constexpr int SB = D / 16;                           // scale bytes of a row
  static constexpr int CODES = KEYS * CB;
  static constexpr int SCALES = KEYS * SB;
  static constexpr int OFF_V = CODES;
  static constexpr int OFF_KS = 2 * CODES;
  static constexpr int OFF_VS = OFF_KS + SCALES;
  static constexpr int STAGE = (OFF_VS + SCALES + 1023) / 1024 * 1024;
  static constexpr int NST = D == 128 ? 2 : 3;
  static constexpr int WARPS = 4;                             // computing warps of a team
  static constexpr int TEAMS = NT == 1 ? 4 : 3;
  static constexpr int THREADS = 128 * (TEAMS + 1);           // a warpgroup a team, and one that copies
  static constexpr int QBUF = ROWS * D * 2;
  static constexpr int OFF_Q = NST * STAGE;                   // an item's query rows
  static constexpr int MROW = D + 4;                          // floats of a merge row (bank spread)
  static constexpr int OFF_MERGE = OFF_Q + QBUF;              // WARPS x ROWS x MROW
  static constexpr int OFF_ML = OFF_MERGE + WARPS * ROWS * MROW * 4;   // WARPS x ROWS x (m, l)
  static constexpr int OFF_BAR = OFF_ML + WARPS * ROWS * 8;
  // full[NST], empty[NST], q_full, q_empty, merge written, merge read; then start[3], abort flag
  static constexpr int NBAR = 2 * NST + 4;
  static constexpr int TEAM_BYTES = (OFF_BAR + NBAR * 8 + 16 + 1023) / 1024 * 1024;
  static constexpr int SMEM_BYTES = TEAMS * TEAM_BYTES + 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget (227 KB per CTA)");
  static constexpr int KS = D / 16;                           // k-steps of S^T
  static constexpr int MT = D / 16;                           // element tiles of O^T
  // Launched with 96 (640 threads) or 128 (512) registers a thread, moved from the copying warps.
  static constexpr uint32_t REG_COPY = 32;
  static constexpr uint32_t REG_TEAM = NT == 1 ? 112 : 160;
  static constexpr int REG_NEED = 128 * (static_cast<int>(REG_COPY) + TEAMS * static_cast<int>(REG_TEAM));
};

struct Q4Params {
  CUtensorMap tk, tv;
  const uint16_t* q;
  const uint8_t *ks, *vs;
  uint16_t* o;
  float *lse, *part;
  const int *cu_q, *seqlens, *table;
  int n_seqs, H, H_kv, G, total_q, max_q, max_k, causal, num_blocks, block_size, max_blocks, piece;
  int n_splits, chunk, row_blocks, n_items;                   // n_splits 0: shares of equal length,
  int whole;                                                  // each of whole row blocks or not
  float score, descale_v, one;                                // scale * log2 e * descale_k; 1
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

// What a sequence brings: its query tokens [first, first + nq), its keys, and its work in units of
// one key step of one row block of one key head.  A sequence without keys still has one
// (empty) unit a row block, which writes O = 0 and lse = -inf.
struct Q4Seq {
  int first, nq, len, blocks, steps;                          // row blocks a key head, units a row block
  __device__ __forceinline__ long long units(int H_kv) const { return static_cast<long long>(blocks) * H_kv * steps; }
};

// Bad contents are reported where ``report`` is set and leave the sequence without rows (boundaries)
// or without keys (lengths).
__device__ __forceinline__ Q4Seq q4_seq(const Q4Params& p, int b, int rows_per_block, bool report) {
  Q4Seq x;
  x.first = b;
  x.nq = 1;
  x.len = __ldg(p.seqlens + b);
  if (p.cu_q) {
    x.first = __ldg(p.cu_q + b);
    const int end = __ldg(p.cu_q + b + 1);
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
  x.blocks = (x.nq * p.G + rows_per_block - 1) / rows_per_block;
  x.steps = max(1, (x.len + kQ4Step - 1) / kQ4Step);
  return x;
}

// By a whole warp: the total, and the sequence that holds unit ``u_of(share)`` with the units before
// it (b = -1 where there is none).
template <typename F>
__device__ __forceinline__ Q4Share q4_share(const Q4Params& p, int rows_per_block, int grid, bool report, F u_of, int* b,
                                            long long* before) {
  const int lane = threadIdx.x & 31;
  Q4Share sh;
  long long mine = 0, own = 0;                                // of all the lane's sequences, of its first
  for (int i = lane; i < p.n_seqs; i += 32) {
    const long long v = q4_seq(p, i, rows_per_block, report).units(p.H_kv);
    if (i == lane) own = v;
    mine += v;
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, off);
  sh.set(mine, grid);
  const long long u = u_of(sh);
  long long sum = 0;
  *b = -1;
  for (int base = 0; base < p.n_seqs && u >= 0; base += 32) {
    const long long v = base == 0 ? own : base + lane < p.n_seqs ? q4_seq(p, base + lane, rows_per_block, false).units(p.H_kv) : 0;
    long long inc = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += x;
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

// One stretch of work: rows [row0, row0 + rows_per_block) of a key head of a sequence over the keys
// [key0, key_end); every row sees the keys below ``full``.
struct Q4Item {
  int b, hkv, rb, first, nq, len, key0, key_end, full;
  int out;                                                    // -1: results; else the place of the state
};

struct Q4Walk {
  const Q4Params& p;
  int rows_per_block, id, stride, item;                       // this team, all teams; chunks: the next item
  int b;                                                      // shares: sequence, unit in it, units left
  int off, left;
  bool report;
  Q4Seq seq;

  __device__ __forceinline__ void finish(Q4Item& x, int step0, int steps) const {
    const int row0 = x.rb * rows_per_block;
    int seen = x.len;
    x.full = x.len;
    if (p.causal) {
      seen = max(0, x.len - x.nq + (min(x.nq * p.G, row0 + rows_per_block) - 1) / p.G + 1);
      x.full = x.len - x.nq + row0 / p.G + 1;
    }
    x.key0 = step0 * kQ4Step;
    x.key_end = min(x.key0 + steps * kQ4Step, seen);
    x.full = min(x.full, x.key_end);
  }

  __device__ __forceinline__ bool next(Q4Item& x) {
    if (p.n_splits) {
      for (; item < p.n_items; item += stride) {
        int i = item;
        const int split = i % p.n_splits;
        i /= p.n_splits;
        x.rb = i % p.row_blocks;
        i /= p.row_blocks;
        x.hkv = i % p.H_kv;
        x.b = i / p.H_kv;
        seq = q4_seq(p, x.b, rows_per_block, report);
        if (x.rb >= seq.blocks) continue;
        x.first = seq.first;
        x.nq = seq.nq;
        x.len = seq.len;
        finish(x, split * (p.chunk / kQ4Step), p.chunk / kQ4Step);
        x.out = p.n_splits == 1 ? -1 : split;
        item += stride;
        return true;
      }
      return false;
    }
    if (left <= 0) return false;
    while (off >= seq.blocks * p.H_kv * seq.steps) {          // (a sequence with work follows: left > 0)
      if (++b >= p.n_seqs) return false;
      off = 0;
      seq = q4_seq(p, b, rows_per_block, false);
    }
    const int pair = off / seq.steps;
    const int step0 = off - pair * seq.steps;
    const int steps = p.whole ? seq.steps : min(left, seq.steps - step0);
    x.b = b;
    x.hkv = pair % p.H_kv;
    x.rb = pair / p.H_kv;
    x.first = seq.first;
    x.nq = seq.nq;
    x.len = seq.len;
    finish(x, step0, steps);
    // a row block that a team has from its first to its last key is done; else the team keeps one state
    // of a row block that began before its share (0) and one of one that goes on behind it (1)
    x.out = steps == seq.steps ? -1 : 2 * id + (step0 == 0 ? 1 : 0);
    off += steps;
    left -= steps;
    return true;
  }
};

template <int D>
__device__ __forceinline__ uint32_t code_offset(int row, int chunk) {   // 16-byte chunk of a row, swizzled
  return D == 128 ? row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4) : row * 32 + ((chunk ^ ((row >> 2) & 1)) << 4);
}

template <int D, int NT>
__global__ void __launch_bounds__(Q4Cfg<D, NT>::THREADS, 1) attend_q4_kernel(const __grid_constant__ Q4Params p) {
  using C = Q4Cfg<D, NT>;
  extern __shared__ uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // Warps 4 t to 4 t + 3 compute for team t, warp 4 TEAMS + t copies for it (others of that group idle).
  const bool copies = warp >= 4 * C::TEAMS;
  const int team = min(copies ? warp - 4 * C::TEAMS : warp >> 2, C::TEAMS - 1);
  const bool idle = copies && warp - 4 * C::TEAMS >= C::TEAMS;
  uint8_t* smem = align_smem_1k(smem_raw) + team * C::TEAM_BYTES;
  float* merge = reinterpret_cast<float*>(smem + C::OFF_MERGE);
  float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::NST;
  uint64_t* q_full = empty + C::NST;
  uint64_t* q_empty = q_full + 1;
  uint64_t* mrg = q_empty + 1;                                // [0]: the warps' states are written, [1]: read
  int* start = reinterpret_cast<int*>(mrg + 2);               // sequence, unit in it, units of the share
  volatile int* abort_flag = start + 3;
  const int id = team * gridDim.x + blockIdx.x, teams = C::TEAMS * gridDim.x;   // few shares: one an SM first
  if (copies && !idle) {
    if (lane == 0) {
      for (int s = 0; s < C::NST; ++s) {
        mbar_init(&full[s], 1);
        mbar_init(&empty[s], C::WARPS);
      }
      mbar_init(q_full, 1);
      mbar_init(q_empty, C::WARPS);
      mbar_init(&mrg[0], C::WARPS);
      mbar_init(&mrg[1], C::WARPS);
      *abort_flag = 0;
      fence_mbarrier_init();
    }
    if (lane < 2) tma_prefetch_desc(lane ? &p.tv : &p.tk);
    if (p.n_splits == 0) {
      int b;
      long long before = 0;
      const Q4Share sh = q4_share(p, C::ROWS, teams, id == 0,
                                  [&](const Q4Share& y) { return id < y.n && y.total > 0 ? y.begin(id) : -1LL; }, &b, &before);
      if (lane == 0) {
        start[0] = b;
        start[1] = b < 0 ? 0 : static_cast<int>(sh.begin(id) - before);
        start[2] = b < 0 ? 0 : static_cast<int>(sh.begin(id + 1) - sh.begin(id));
      }
    }
  }
  pdl_launch_dependents();
  __syncthreads();
  Q4Walk walk{p, C::ROWS, id, teams, id, 0, 0, 0, copies && lane == 0, {}};
  if (p.n_splits == 0) {
    walk.b = start[0];
    walk.off = start[1];
    walk.left = start[2];
    if (walk.left > 0) {
      walk.seq = q4_seq(p, walk.b, C::ROWS, false);
      if (p.whole) {
        const int behind = walk.off % walk.seq.steps, skip = behind ? walk.seq.steps - behind : 0;
        walk.off += skip;
        walk.left -= skip;
      }
    }
  }
  Q4Item x;

  if (copies) {
    setmaxnreg_dec<C::REG_COPY>();
    // ---------------------------------------------------------------- copies
    // Lane j copies piece j (``piece`` keys of one page) of a stage.
    const int pieces = C::KEYS / p.piece;
    int s = 0;
    uint32_t phase = 1, g = 0, it = 0;                       // the first pass over the ring waits for nothing
    bool ok = true;
    while (!idle && ok && walk.next(x)) {
      // the item's query rows: those of a token lie side by side, lane j copies token j of the block
      {
        if (it >= 1 && !(ok = mbar_wait_warp(q_empty, (it - 1) & 1, abort_flag, 435))) break;
        const int row0 = x.rb * C::ROWS, row1 = min(x.nq * p.G, row0 + C::ROWS);
        if (lane == 0) mbar_arrive_expect_tx(q_full, (row1 - row0) * D * 2);
        __syncwarp();
        const int i = row0 / p.G + lane;
        const int a = max(row0, i * p.G), e = min(row1, (i + 1) * p.G);
        if (a < e)
          bulk_load(smem + C::OFF_Q + (a - row0) * D * 2,
                    p.q + (static_cast<size_t>(x.first + i) * p.H + x.hkv * p.G + (a - i * p.G)) * D, (e - a) * D * 2, q_full);
        ++it;
      }
      int window = -1, tab = 0;                              // 32 table entries from block ``window`` on
      const int last_blk = (x.key_end - 1) / p.block_size;
      int key = x.key0 + (lane < pieces ? lane : 0) * p.piece;
      int blk = key / p.block_size, in = key - blk * p.block_size;
      for (int kk = x.key0; kk < x.key_end; kk += C::KEYS, ++g) {
        // the stage's pages, at most eight: all in the window that begins with the first of them
        const int blk0 = __shfl_sync(0xffffffffu, blk, 0);
        if (window < 0 || blk0 + 8 > window + 32) {
          window = blk0;
          // entries that hold the item's keys only
          tab = window + lane <= last_blk ? __ldg(p.table + static_cast<size_t>(x.b) * p.max_blocks + window + lane) : 0;
        }
        int page = __shfl_sync(0xffffffffu, tab, (blk - window) & 31);
        const bool mine = lane < pieces && key < x.key_end;
        if (mine && (page < 0 || page >= p.num_blocks)) {
          report_device_error(FA_DEV_BAD_CONFIG, 422);
          page = 0;                                          // stays in bounds; the result is reported invalid
        }
        if (g >= C::NST && !(ok = mbar_wait_warp(&empty[s], phase, abort_flag, 430))) break;
        const int live = __popc(__ballot_sync(0xffffffffu, mine));
        if (lane == 0) mbar_arrive_expect_tx(&full[s], live * p.piece * 2 * (C::CB + C::SB));
        __syncwarp();
        if (mine) {
          uint8_t* st = smem + s * C::STAGE;
          const int row = (page * p.H_kv + x.hkv) * p.block_size + in;
          const int at = lane * p.piece;
          tma_load_2d(st + at * C::CB, &p.tk, &full[s], 0, row);
          tma_load_2d(st + C::OFF_V + at * C::CB, &p.tv, &full[s], 0, row);
          bulk_load(st + C::OFF_KS + at * C::SB, p.ks + static_cast<size_t>(row) * C::SB, p.piece * C::SB, &full[s]);
          bulk_load(st + C::OFF_VS + at * C::SB, p.vs + static_cast<size_t>(row) * C::SB, p.piece * C::SB, &full[s]);
        }
        __syncwarp();
        key += C::KEYS;
        in += C::KEYS;
        while (in >= p.block_size) {
          in -= p.block_size;
          ++blk;
        }
        if (++s == C::NST) {
          s = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) {
      // drain the copies already issued (at most NST stages and an item's queries outstanding)
      if (it > 0) mbar_wait_warp(q_full, (it - 1) & 1, nullptr, 436);
      for (uint32_t y = (g > C::NST ? g - C::NST : 0); y < g; ++y) mbar_wait_warp(&full[y % C::NST], (y / C::NST) & 1, nullptr, 431);
    }
  } else {
    setmaxnreg_inc<C::REG_TEAM>();
    // ---------------------------------------------------------------- products
    const int tw = warp & 3;                                          // warp of the team
    const int r = lane >> 2, c = lane & 3;
    const int ra = tw * 32 + (r ^ (((r >> 1) ^ (r >> 2)) & 1));       // key kappa(r) of the warp's first 8
    const int e = 2 * c;
    const int v0 = tw * 32 + (e ^ (((e >> 1) ^ (e >> 2)) & 1));       // keys kappa(2c) and kappa(2c + 1)
    const int v1 = v0 ^ 1;
    // Places in a stage; 8 rows on is 8 CB bytes on, under the swizzle too.
    constexpr int SR = D == 128 ? 1 : 2;                              // lanes' rows that share a scale block (V)
    const uint8_t* const pk = smem + (D == 128 ? code_offset<D>(ra, c) : code_offset<D>(ra, c >> 1) + (c & 1) * 8);
    const uint8_t* const pks = smem + C::OFF_KS + ra * C::SB + (D == 128 ? 2 * c : c);
    const uint8_t* const pv0 = smem + C::OFF_V + (D == 128 ? code_offset<D>(v0, r >> 1) + (r & 1) * 8 : code_offset<D>(v0, r >> 2) + (r & 3) * 4);
    const uint8_t* const pv1 = smem + C::OFF_V + (D == 128 ? code_offset<D>(v1, r >> 1) + (r & 1) * 8 : code_offset<D>(v1, r >> 2) + (r & 3) * 4);
    const uint8_t* const pvs0 = smem + C::OFF_VS + v0 * C::SB + r / SR;
    const uint8_t* const pvs1 = smem + C::OFF_VS + v1 * C::SB + r / SR;
    int s = 0;
    uint32_t phase = 0, it = 0;
    bool ok = true;
    while (walk.next(x)) {
      const int rows = x.nq * p.G;
      // Queries: lane (r, c) holds row r's elements [c d/4, (c+1) d/4) as B operands; the factors and
      // key limits of rows 2c and 2c + 1, whose scores the lane gets, come from the lanes that hold them.
      uint32_t qb[NT][C::KS][2];
      float2 fac[NT];
      int vis[NT][2];
      if (!(ok = mbar_wait_warp(q_full, it & 1, abort_flag, 437))) break;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int row = x.rb * C::ROWS + 8 * n + r;
        const int i = row / p.G;
        const uint8_t* src = smem + C::OFF_Q + (8 * n + r) * D * 2 + c * (D / 2);
        uint4 w[D / 32];
        float big = 0.f;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          w[j] = make_uint4(0u, 0u, 0u, 0u);
          if (row < rows) w[j] = *(reinterpret_cast<const uint4*>(src) + j);
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
        fac[n].x = __shfl_sync(0xffffffffu, f, 8 * c);
        fac[n].y = __shfl_sync(0xffffffffu, f, 8 * c + 4);
#pragma unroll
        for (int k = 0; k < 2; ++k) vis[n][k] = min(x.key_end, __shfl_sync(0xffffffffu, seen, (2 * c + k) * 4));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(q_empty);
      // m: reference, some number below every score before the first
      float2 m[NT], l[NT];
      float o[NT][C::MT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        m[n] = make_float2(kNone, kNone);
        l[n] = make_float2(0.f, 0.f);
#pragma unroll
        for (int t = 0; t < C::MT; ++t) o[n][t][0] = o[n][t][1] = o[n][t][2] = o[n][t][3] = 0.f;
      }

      for (int kk = x.key0; kk < x.key_end; kk += C::KEYS) {
        if (!(ok = mbar_wait_warp(&full[s], phase, abort_flag, 432))) break;
        const int so = s * C::STAGE;
        // S^T: this warp's 32 keys against the rows
        float sc[2][NT][4];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int sg = so + g * 16 * C::CB, ss = so + g * 16 * C::SB;
#pragma unroll
          for (int n = 0; n < NT; ++n) sc[g][n][0] = sc[g][n][1] = sc[g][n][2] = sc[g][n][3] = 0.f;
          uint32_t wa[D / 32], wb[D / 32];                     // the two keys' codes, 8 a word
          uint32_t sa[2], sb[2];                               // scales of their blocks, doubled
          if constexpr (D == 128) {
            const uint4 a = *reinterpret_cast<const uint4*>(pk + sg);
            const uint4 b = *reinterpret_cast<const uint4*>(pk + sg + 8 * C::CB);
            wa[0] = a.x; wa[1] = a.y; wa[2] = a.z; wa[3] = a.w;
            wb[0] = b.x; wb[1] = b.y; wb[2] = b.z; wb[3] = b.w;
            const uint32_t ea = e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(pks + ss));
            const uint32_t eb = e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(pks + ss + 8 * C::SB));
            sa[0] = __byte_perm(ea, ea, 0x1010); sa[1] = __byte_perm(ea, ea, 0x3232);
            sb[0] = __byte_perm(eb, eb, 0x1010); sb[1] = __byte_perm(eb, eb, 0x3232);
          } else {
            const uint2 a = *reinterpret_cast<const uint2*>(pk + sg);
            const uint2 b = *reinterpret_cast<const uint2*>(pk + sg + 8 * C::CB);
            wa[0] = a.x; wa[1] = a.y;
            wb[0] = b.x; wb[1] = b.y;
            sa[0] = e4m3x2_to_f16(pks[ss] * 0x0101u);
            sb[0] = e4m3x2_to_f16(pks[ss + 8 * C::SB] * 0x0101u);
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
              mma_f16(sc[g][n], a[0], b[0], a[1], b[1], qb[n][2 * j][0], qb[n][2 * j][1]);
              mma_f16(sc[g][n], a[2], b[2], a[3], b[3], qb[n][2 * j + 1][0], qb[n][2 * j + 1][1]);
            }
          }
        }
        // scores of keys kk + ra + 8 i for rows 2c, 2c + 1, in the log2 domain
        uint32_t pb[2][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float2 t[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) t[i] = fmul2(make_float2(sc[i >> 1][n][2 * (i & 1)], sc[i >> 1][n][2 * (i & 1) + 1]), fac[n]);
          if (kk + C::KEYS > x.full) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (kk + ra + 8 * i >= vis[n][0]) t[i].x = -INFINITY;
              if (kk + ra + 8 * i >= vis[n][1]) t[i].y = -INFINITY;
            }
          }
          const float t0 = fmaxf(fmax3(t[0].x, t[1].x, t[2].x), t[3].x), t1 = fmaxf(fmax3(t[0].y, t[1].y, t[2].y), t[3].y);
          if (__any_sync(0xffffffffu, t0 > m[n].x + (kQ4Lift + 8.f) || t1 > m[n].y + (kQ4Lift + 8.f))) {
            // a row's largest weight grew past 2^15: move its reference to 7 below the maximum (for huge
            // scores to what that rounds to, at most 8 below)
            float2 top = make_float2(fmaxf(m[n].x, t0 - kQ4Lift), fmaxf(m[n].y, t1 - kQ4Lift));
#pragma unroll
            for (int off = 4; off <= 16; off <<= 1) {
              top.x = fmaxf(top.x, __shfl_xor_sync(0xffffffffu, top.x, off));
              top.y = fmaxf(top.y, __shfl_xor_sync(0xffffffffu, top.y, off));
            }
            const float2 alpha = make_float2(fast_exp2(m[n].x - top.x), fast_exp2(m[n].y - top.y));
            m[n] = top;
            l[n] = fmul2(l[n], alpha);
#pragma unroll
            for (int i = 0; i < C::MT; ++i) {
              o[n][i][0] *= alpha.x;
              o[n][i][1] *= alpha.y;
              o[n][i][2] *= alpha.x;
              o[n][i][3] *= alpha.y;
            }
          }
          // t - m as fma(t, 1, -m) with a 1 that the compiler does not know: t's product is not to go
          // into an fma unrounded, where huge scores would leave their maximum's rounding in the exponent
          const float2 nm = make_float2(-m[n].x, -m[n].y), one = make_float2(p.one, p.one);
          float2 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 y = ffma2(t[i], one, nm);
            w[i] = make_float2(fast_exp2(y.x), fast_exp2(y.y));
            pb[i >> 1][n][i & 1] = transpose8x8(pack_f16x2(w[i].x, w[i].y));
          }
          l[n] = fadd2(l[n], fadd2(fadd2(w[0], w[1]), fadd2(w[2], w[3])));
        }
        // O^T += V^T P^T
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int sg = so + g * 16 * C::CB, ss = so + g * 16 * C::SB;
          constexpr int W = D / 64;                            // words of a row's d/8 elements
          uint32_t lo[2][W], hi[2][W], sl[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t a[W], b[W];
            if constexpr (D == 128) {
              const uint2 x0 = *reinterpret_cast<const uint2*>(pv0 + sg + 8 * h * C::CB);
              const uint2 x1 = *reinterpret_cast<const uint2*>(pv1 + sg + 8 * h * C::CB);
              a[0] = x0.x; a[1] = x0.y; b[0] = x1.x; b[1] = x1.y;
            } else {
              a[0] = *reinterpret_cast<const uint32_t*>(pv0 + sg + 8 * h * C::CB);
              b[0] = *reinterpret_cast<const uint32_t*>(pv1 + sg + 8 * h * C::CB);
            }
            uint32_t e0 = pvs0[ss + 8 * h * C::SB], e1 = pvs1[ss + 8 * h * C::SB];
            if (kk + C::KEYS > x.key_end) {
              // rows past the end hold anything, a scale that is no number among it: 0 * NaN is NaN
              if (kk + v0 + 16 * g + 8 * h >= x.key_end) e0 = 0;
              if (kk + v1 + 16 * g + 8 * h >= x.key_end) e1 = 0;
            }
            sl[h] = e4m3x2_to_f16(__byte_perm(e0, e1, 0x0040));
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
              for (int n = 0; n < NT; ++n) mma_f16(o[n][4 * j + i], w0, w1, w2, w3, pb[g][n][0], pb[g][n][1]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
        if (++s == C::NST) {
          s = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;

      // The warps' states of this stretch.  o[n][t]: rows 2c, 2c + 1 at elements r d/8 + 2t (+1), which
      // lie in shared memory at 16 t + 2 ((r + t) % 8) (+1) of the merge row (no bank twice, neither here
      // nor below).  Each warp then adds up a quarter of the rows, in the order of the warps.
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int off = 4; off <= 16; off <<= 1) {
          l[n].x += __shfl_xor_sync(0xffffffffu, l[n].x, off);
          l[n].y += __shfl_xor_sync(0xffffffffu, l[n].y, off);
        }
      }
      if (it > 0 && !(ok = mbar_wait_warp(&mrg[1], (it - 1) & 1, abort_flag, 434))) break;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int at = tw * C::ROWS + 8 * n + 2 * c + k;
#pragma unroll
          for (int t = 0; t < C::MT; ++t)
            *reinterpret_cast<float2*>(merge + at * C::MROW + 16 * t + 2 * ((r + t) & 7)) = make_float2(o[n][t][k], o[n][t][2 + k]);
          if (r == 0) ml[at] = k ? make_float2(m[n].y, l[n].y) : make_float2(m[n].x, l[n].x);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&mrg[0]);
      if (!(ok = mbar_wait_warp(&mrg[0], it & 1, abort_flag, 433))) break;
      constexpr int QR = C::ROWS / C::WARPS;                   // a warp's rows
      constexpr int PL = D / 64;                               // element pairs of a lane: lane + 32 i
#pragma unroll
      for (int y = 0; y < QR; ++y) {
        const int rr = tw * QR + y, row = x.rb * C::ROWS + rr;
        if (row >= rows) break;
        float2 st[C::WARPS];
        float M = kNone, L = 0.f;
        float2 acc[PL];
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) {
          st[w] = ml[w * C::ROWS + rr];
          M = fmaxf(M, st[w].x);
        }
#pragma unroll
        for (int i = 0; i < PL; ++i) acc[i] = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) {
          const float wt = fast_exp2(st[w].x - M);
          L = fmaf(wt, st[w].y, L);
#pragma unroll
          for (int i = 0; i < PL; ++i) {
            const int pr = lane + 32 * i, pt = pr % C::MT;     // (d/16 pairs of each r)
            const float2 v = *reinterpret_cast<const float2*>(merge + (w * C::ROWS + rr) * C::MROW + 16 * pt + 2 * ((pr / C::MT + pt) & 7));
            acc[i] = ffma2(make_float2(wt, wt), v, acc[i]);
          }
        }
        const int i = row / p.G;
        const int tok = x.first + i, head = x.hkv * p.G + (row - i * p.G);
        const size_t th = static_cast<size_t>(tok) * p.H + head;
        const bool none = L == 0.f;                            // a row that sees no key (scores that are no number: L is none)
        if (x.out < 0) {
          const float inv = none ? 0.f : p.descale_v / L;
#pragma unroll
          for (int k = 0; k < PL; ++k)
            reinterpret_cast<uint32_t*>(p.o + th * D)[lane + 32 * k] = none ? 0u : pack_bf16x2(acc[k].x * inv, acc[k].y * inv);
          if (lane == 0)
            p.lse[p.cu_q ? static_cast<size_t>(head) * p.total_q + tok : th] = none ? -INFINITY : q4_lse(M, L);
        } else {
          const size_t at = p.n_splits ? th * p.n_splits + x.out : static_cast<size_t>(x.out) * C::ROWS + rr;
          float* dst = p.part + at * (D + 2);
#pragma unroll
          for (int k = 0; k < PL; ++k) reinterpret_cast<float2*>(dst)[lane + 32 * k] = acc[k];
          if (lane == 0) *reinterpret_cast<float2*>(dst + D) = make_float2(none ? -INFINITY : M, L);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&mrg[1]);
      ++it;
    }
  }
  __syncwarp();
  __syncthreads();
}

// The sequence of packed token t, if it is one that the kernels above computed, else -1; by a whole warp.
__device__ __forceinline__ int q4_owner(const int* __restrict__ cu, int n_seqs, int total_q, int max_q, int t) {
  auto has = [&](int b) {
    const int first = __ldg(cu + b), end = __ldg(cu + b + 1);
    return first >= 0 && first <= t && t < end && end <= total_q && end - first <= max_q;
  };
  const int found = search_owner(cu, n_seqs, t);
  if (has(found)) return found;
  // in front of the first sequence or behind the last one, or boundaries that do not ascend, among which
  // some sequence may be sound all the same
  for (int b0 = 0; b0 < n_seqs; b0 += 32) {
    const int b = b0 + (threadIdx.x & 31);
    const uint32_t sound = __ballot_sync(0xffffffffu, b < n_seqs && has(b));
    if (sound) return b0 + __ffs(sound) - 1;
  }
  return -1;
}

// Joins a row's chunks where the caller gave their count (part: [row][chunk]): WPR warps a row.  Rows that
// have no states stay as they are.
template <int D, int WPR>
__global__ void __launch_bounds__(128) attend_q4_merge_kernel(const float* __restrict__ part, uint16_t* __restrict__ o,
                                                             float* __restrict__ lse, const int* __restrict__ cu_q,
                                                             int n_seqs, int H, int total_q, int max_q, int n_splits,
                                                             float descale_v) {
  const long long th = WPR > 1 ? blockIdx.x : static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int tok = static_cast<int>(th / H), head = static_cast<int>(th - static_cast<long long>(tok) * H);
  const bool some = th < static_cast<long long>(total_q) * H && (!cu_q || q4_owner(cu_q, n_seqs, total_q, max_q, tok) >= 0);
  pdl_wait();
  q4_join<D, WPR>({part + static_cast<size_t>(th) * n_splits * (D + 2), D + 2, 0, some ? n_splits : 0},
                  WPR > 1 ? threadIdx.x >> 5 : 0, WPR, o + static_cast<size_t>(th) * D,
                  lse + (cu_q ? static_cast<size_t>(head) * total_q + tok : static_cast<size_t>(th)), descale_v);
}

// Joins the states of the rows whose row block lies in several teams' shares, WPR warps a row.
template <int D, int NT, int WPR>
__global__ void __launch_bounds__(128) attend_q4_row_join_kernel(const __grid_constant__ Q4Params p, int teams) {
  constexpr int ROWS = 8 * NT;
  const long long th = WPR > 1 ? blockIdx.x : static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const bool some = th < static_cast<long long>(p.total_q) * p.H;
  const int tok = some ? static_cast<int>(th / p.H) : 0, head = static_cast<int>(th - static_cast<long long>(tok) * p.H);
  int b = some ? tok : -1;
  if (some && p.cu_q) b = q4_owner(p.cu_q, p.n_seqs, p.total_q, p.max_q, tok);
  long long total = 0, before = 0;                             // units of all sequences, of those before b
  for (int k = threadIdx.x & 31; k < p.n_seqs; k += 32) {
    const long long v = q4_seq(p, k, ROWS, false).units(p.H_kv);
    total += v;
    if (k < b) before += v;
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, off);
    before += __shfl_xor_sync(0xffffffffu, before, off);
  }
  Q4Share sh;
  sh.set(total, teams);
  Q4States st{p.part, 2 * ROWS * (D + 2), ROWS * (D + 2), 0};
  if (b >= 0) {                                                // (else no sequence's: stays as it is)
    const Q4Seq seq = q4_seq(p, b, ROWS, false);
    const int row = (tok - seq.first) * p.G + head % p.G;
    const long long u0 = before + (static_cast<long long>(row / ROWS) * p.H_kv + head / p.G) * seq.steps;
    const int c0 = sh.owner(u0), c1 = sh.owner(u0 + seq.steps - 1);
    if (c0 != c1) {                                            // (else its team wrote the result)
      st.base += (static_cast<size_t>(2 * c0) * ROWS + row % ROWS) * (D + 2);
      st.n = c1 - c0 + 1;
    }
  }
  pdl_wait();
  q4_join<D, WPR>(st, WPR > 1 ? threadIdx.x >> 5 : 0, WPR, p.o + static_cast<size_t>(th) * D,
                  p.lse + (p.cu_q ? static_cast<size_t>(head) * p.total_q + tok : static_cast<size_t>(th)), p.descale_v);
}

// The same for many row blocks, most of which are not divided.  Those that are hold a bound between shares:
// a block takes the row block of bound i + 1 if that is the first within it, and its warps share the rows out.
constexpr int kQ4JoinWarps = 16;

template <int D, int NT>
__global__ void __launch_bounds__(32 * kQ4JoinWarps) attend_q4_join_kernel(const __grid_constant__ Q4Params p, int teams) {
  constexpr int ROWS = 8 * NT;
  __shared__ Q4Item item;                                      // b, hkv, rb, first, nq; n in ``len``, first team in ``out``
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (warp == 0) {
    const int i = blockIdx.x;
    int b;
    long long before = 0;                                      // units of the sequences before b
    const Q4Share sh = q4_share(p, ROWS, teams, false, [&](const Q4Share& y) { return i + 1 < y.n ? y.begin(i + 1) : -1LL; }, &b, &before);
    if (threadIdx.x == 0) {
      item.len = 0;
      if (b >= 0) {
        const Q4Seq seq = q4_seq(p, b, ROWS, false);
        const int pair = static_cast<int>(sh.begin(i + 1) - before) / seq.steps;   // (below 2^31 units a sequence)
        const long long u0 = before + static_cast<long long>(pair) * seq.steps;
        const int c0 = sh.owner(u0), c1 = sh.owner(u0 + seq.steps - 1);
        if (c0 != c1 && c0 == i) {                             // (c0 == i: bound i + 1 is its first)
          item.b = b;
          item.hkv = pair % p.H_kv;
          item.rb = pair / p.H_kv;
          item.first = seq.first;
          item.nq = seq.nq;
          item.len = c1 - c0 + 1;
          item.out = c0;
        }
      }
    }
  }
  __syncthreads();
  pdl_wait();
  if (item.len == 0) return;
  const int row0 = item.rb * ROWS, rows = min(ROWS, item.nq * p.G - row0);
  int wpr = warps;                                             // warps a row
  while (wpr > 1 && wpr * rows > warps) wpr >>= 1;
  const int at_once = warps / wpr;
  for (int r0 = 0; r0 < rows; r0 += at_once) {
    const int rr = r0 + warp / wpr;
    const bool some = rr < rows;
    const int row = row0 + (some ? rr : 0), i = row / p.G;
    const int tok = item.first + i, head = item.hkv * p.G + (row - i * p.G);
    const size_t th = static_cast<size_t>(tok) * p.H + head;
    const Q4States st{p.part + (static_cast<size_t>(2 * item.out) * ROWS + rr) * (D + 2), 2 * ROWS * (D + 2), ROWS * (D + 2),
                      some ? item.len : 0};
    q4_join<D, kQ4JoinWarps>(st, warp, wpr, p.o + th * D, p.lse + (p.cu_q ? static_cast<size_t>(head) * p.total_q + tok : th), p.descale_v);
  }
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
  // a stage's keys in pieces that never cross a page
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
  p.row_blocks = static_cast<int>((q4_rows(a.H, a.H_kv, a.max_seqlen_q) + C::ROWS - 1) / C::ROWS);
  const long long pairs = static_cast<long long>(a.n_seqs) * a.H_kv * p.row_blocks;
  p.n_items = static_cast<int>(pairs * a.n_splits);
  p.score = a.scale * 1.4426950408889634f * a.descale_k;
  p.descale_v = a.descale_v;
  p.one = 1.f;
  const long long most = min(q4_sm_count(), kQ4MaxShares / C::TEAMS);
  const long long steps = (static_cast<long long>(a.max_seqlen_k) + kQ4Step - 1) / kQ4Step;
  // Short row blocks, and enough of them for a quarter of the teams, are not divided: the states and the
  // join cost as much as some four steps (8 key heads, 512 tokens, 64 sequences 18.6 us, whole 14.4; 24, 14.5
  // and 13.7, though 38, 13.8 and 14.4; of 1000 tokens 38 sequences 17.2, whole 21.2).
  p.whole = steps <= 1 || (steps <= 5 && 4 * pairs >= most * C::TEAMS) ? 1 : 0;
  static int attr_done[64] = {0};
  cudaError_t e = ensure_smem_attr(attend_q4_kernel<D, NT>, C::SMEM_BYTES, attr_done, C::THREADS, C::REG_NEED);
  if (e != cudaSuccess) return e;
  // (a share is kQ4MinUnits long at least, and there are pairs * steps units at most)
  const long long want = a.n_splits ? p.n_items : pairs * max(1LL, steps) / kQ4MinUnits;
  const int grid = static_cast<int>(max(1LL, min(most, want)));
  log_launch("attend_q4_kernel<D, NT>", static_cast<unsigned long long>(grid), C::THREADS, static_cast<unsigned long long>(C::SMEM_BYTES));
  attend_q4_kernel<D, NT><<<grid, C::THREADS, C::SMEM_BYTES, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.n_splits || p.whole) return e;
  const int teams = C::TEAMS * grid;
  // By rows up to two row blocks a team, us by rows and by bounds: 16 x 4000 tokens of 16 query heads a key
  // head 16 and 20, 48 x 8192 55 and 58, 128 x 1500 of 4 43 and 44 (1024 row blocks), 256 x 1500 76 and 73.
  if (pairs <= 1024) {
    const long long out_rows = static_cast<long long>(a.total_q) * a.H;
    const int warps = q4_join_warps(out_rows);
    const unsigned blocks = static_cast<unsigned>((out_rows * warps + 3) / 4);
    log_launch("attend_q4_row_join_kernel<D, NT, WPR>", blocks, 128, 0ull);
    return launch_join(warps == 1 ? attend_q4_row_join_kernel<D, NT, 1> : attend_q4_row_join_kernel<D, NT, 4>, blocks, 128, stream, p, teams);
  }
  const unsigned threads = NT > 1 ? 32 * kQ4JoinWarps : p.G * a.max_seqlen_q > 4 ? 256 : 128;   // a warp a row
  log_launch("attend_q4_join_kernel<D, NT>", static_cast<unsigned long long>(teams - 1), threads, 0ull);
  return launch_join(attend_q4_join_kernel<D, NT>, static_cast<unsigned>(teams - 1), threads, stream, p, teams);
}

template <int D, int WPR>
static cudaError_t launch_attend_q4_merge(const PagedQ4Args& a, cudaStream_t stream) {
  const unsigned blocks = static_cast<unsigned>((static_cast<long long>(a.total_q) * a.H * WPR + 3) / 4);
  log_launch("attend_q4_merge_kernel<D, WPR>", blocks, 128, 0ull);
  return launch_join(attend_q4_merge_kernel<D, WPR>, blocks, 128, stream, static_cast<const float*>(a.part),
                     static_cast<uint16_t*>(a.o), a.lse, a.cu_q, a.n_seqs, a.H, a.total_q, a.max_seqlen_q,
                     a.n_splits, a.descale_v);
}

cudaError_t launch_attend_q4(const PagedQ4Args& a, cudaStream_t stream) {
  cudaError_t e;
  if (q4_use_tiles(a.H, a.H_kv, a.max_seqlen_q, a.d)) {
    e = launch_attend_q4_tile(a, stream);
  } else {
    // 8 rows suffice for up to 8 query heads a key head at one token; else 16 share the unpacked keys
    const bool small = q4_rows(a.H, a.H_kv, a.max_seqlen_q) <= 8;
    if (a.d == 64) e = small ? launch_attend_q4_d<64, 1>(a, stream) : launch_attend_q4_d<64, 2>(a, stream);
    else e = small ? launch_attend_q4_d<128, 1>(a, stream) : launch_attend_q4_d<128, 2>(a, stream);
  }
  if (e != cudaSuccess || a.n_splits <= 1) return e;
  if (q4_join_warps(static_cast<long long>(a.total_q) * a.H) == 1)
    return a.d == 64 ? launch_attend_q4_merge<64, 1>(a, stream) : launch_attend_q4_merge<128, 1>(a, stream);
  return a.d == 64 ? launch_attend_q4_merge<64, 4>(a, stream) : launch_attend_q4_merge<128, 4>(a, stream);
}

}  // namespace fa

FA_DEFINE_STATUS_FETCH(status_fetch_attend_q4)
