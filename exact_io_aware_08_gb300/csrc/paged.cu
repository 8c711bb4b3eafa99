// Filling a paged key/value cache and reading a 4-bit one back.
//
// Append: each packed token's query and key heads are rotated by the token's position (its place in the
// sequence, or one that is given: a drafted token's depth, places behind evicted tokens), keys and
// values go to the token's row of its page, in bf16 or rounded to the 4-bit format (q4.cuh).
// Pairs (x1, x2) become (x1 c - x2 s, x2 c + x1 s) in fp32, every product and sum rounded by itself.
// 4 bits: of 16 consecutive elements, scale = e4m3(max |x| / (6 descale)) and
// code = e2m1(x / (scale descale)), true divisions, so that a tie is a tie.
//
// Both directions only move data (a few operations a byte), so they are bound by HBM on long calls
// and by the chain of dependent loads (boundaries, length, page, then the store) on short ones.
// A head's row is spread over d/16 lanes, 16 elements each as two 16-byte vectors: the two halves of
// eight pairs where the pairs lie rotary/2 apart, so that a lane needs eight cosines and eight sines
// and keeps them for all the heads that it takes of the token.
#include "fa_kernels.h"
#include "q4.cuh"

namespace fa {

struct AppendParams {
  const uint16_t *q, *k, *v;
  uint16_t* q_out;
  uint16_t *k_cache, *v_cache;                        // bf16 cache [pages, block, H_kv, d]
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;   // 4-bit cache [pages, H_kv, block, d/2 | d/16]
  const float *cos, *sin;                             // [n_positions, rotary/2]
  const int *cu, *seqlens, *table;
  long long q_stride, k_stride, v_stride;             // elements from one token to the next
  int n_seqs, H, H_kv, total, max_blocks, block_size, num_blocks, rotary, n_positions;
  int warps_per_token;
  float descale_k, descale_v, one;
  const int* positions;                               // [total] or null
};

constexpr int kPagedThreads = 128;
constexpr float kUp = 1.f + 0x1p-20f, kDown = 1.f - 0x1p-20f;

// The 4-bit form of 16 values: the lane's vector 0 (f[0..7]) and 1 (f[8..15]).  ``split``: they
// belong to two blocks, each completed by the neighbouring lane's vector; else to one block.
__device__ __forceinline__ void quantise16(const float (&f)[16], bool split, float descale,
                                           uint32_t (&code)[2], uint32_t (&scale)[2]) {
  float a[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[0] = fmaxf(a[0], fabsf(f[i]));
    a[1] = fmaxf(a[1], fabsf(f[8 + i]));
  }
  const float o0 = __shfl_xor_sync(0xffffffffu, a[0], 1);
  const float o1 = __shfl_xor_sync(0xffffffffu, a[1], 1);
  const float both = fmaxf(a[0], a[1]);
  a[0] = split ? fmaxf(a[0], o0) : both;
  a[1] = split ? fmaxf(a[1], o1) : both;
  // A quotient decides only between neighbouring codes.  The product with the reciprocal is within
  // 2^-22 of it; where the codes of that product 2^-20 up and down agree, so does the quotient's
  // (rounding is monotone), and the division, some ten instructions, is made only where they differ.
  const float six = __fmul_rn(6.f, descale), inv6 = __frcp_rn(six);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float2 near = fmul2(make_float2(__fmul_rn(a[h], inv6), __fmul_rn(a[h], inv6)), make_float2(kUp, kDown));
    const uint32_t two = f32x2_to_e4m3(near.x, near.y);
    scale[h] = two & 0xffu;
    if (scale[h] != two >> 8) scale[h] = f32x2_to_e4m3(__fdiv_rn(a[h], six), 0.f) & 0xffu;
    const float sd = __fmul_rn(f16x2_to_f32(e4m3x2_to_f16(scale[h])).x, descale);
    const float inv = sd > 0.f ? __frcp_rn(sd) : 0.f;        // (a scale of 0: codes of 0 with x's signs)
    const float iu = __fmul_rn(inv, kUp), id = __fmul_rn(inv, kDown);
    const float2 up = make_float2(iu, iu), down = make_float2(id, id);
    float y[8], z[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 q = make_float2(f[8 * h + 2 * i], f[8 * h + 2 * i + 1]);
      const float2 u = fmul2(q, up), v = fmul2(q, down);
      y[2 * i] = u.x; y[2 * i + 1] = u.y;
      z[2 * i] = v.x; z[2 * i + 1] = v.y;
    }
    code[h] = f32x8_to_e2m1(y);
    if (code[h] != f32x8_to_e2m1(z)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = sd > 0.f ? __fdiv_rn(f[8 * h + i], sd) : copysignf(0.f, f[8 * h + i]);
      code[h] = f32x8_to_e2m1(y);
    }
  }
}

// (six passes in 4 bits: 124 registers without a limit, 200 against 194 us for 24 mixed sequences)
template <int D, bool Q4, bool INTER, int U>
__global__ void __launch_bounds__(kPagedThreads, Q4 && U == 6 ? 5 : 1) append_kernel(const AppendParams p) {
  constexpr int L = D / 16;                       // lanes a head
  constexpr int SPW = 32 / L;                     // heads a warp takes at once
  const int lane = threadIdx.x & 31;
  const int w = blockIdx.x * (kPagedThreads / 32) + (threadIdx.x >> 5);
  const int t = w / p.warps_per_token;
  if (t >= p.total) return;
  const int part = w - t * p.warps_per_token;
  const int u = lane % L;
  const int slots = p.H + 2 * p.H_kv;
  const int r16 = p.rotary / 16;
  const bool rotates = u < r16;
  const bool split = rotates && !INTER;

  // the data does not depend on the token's place: loads first
  uint4 x0[U], x1[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int slot = (part * U + j) * SPW + lane / L;
    x0[j] = x1[j] = make_uint4(0u, 0u, 0u, 0u);
    if (slot < slots) {
      const uint16_t* src = slot < p.H ? p.q + t * p.q_stride + static_cast<long long>(slot) * D
                            : slot < p.H + p.H_kv
                                ? p.k + t * p.k_stride + static_cast<long long>(slot - p.H) * D
                                : p.v + t * p.v_stride + static_cast<long long>(slot - p.H - p.H_kv) * D;
      const bool sp = split && slot < p.H + p.H_kv;
      x0[j] = *reinterpret_cast<const uint4*>(src + (sp ? u : 2 * u) * 8);
      x1[j] = *reinterpret_cast<const uint4*>(src + (sp ? u + r16 : 2 * u + 1) * 8);
    }
  }

  const int given = p.positions ? __ldg(p.positions + t) : 0;
  int first, count, page, row;
  const int b = owner_of_token(p.cu, p.n_seqs, p.total, t, &first, &count, 400);
  if (b < 0) return;
  const int len = __ldg(p.seqlens + b);
  const int pos = len - count + (t - first);
  const int turn = p.positions ? given : pos;     // where the tables are read
  if (len < count || (p.rotary > 0 && (turn < 0 || turn >= p.n_positions))) {
    if (lane == 0) report_device_error(FA_DEV_BAD_CONFIG, 401);
    return;
  }
  if (!place_of_token(p.table, p.max_blocks, p.block_size, p.num_blocks, b, len, pos, &page, &row, 402)) return;

  // The sums are fma(product, 1, product) with a 1 that the compiler does not know: of mul.f32x2 and
  // add.f32x2 it makes one fma although both carry .rn, and the product goes unrounded.
  const float2 one = make_float2(p.one, p.one);
  float2 c[4], s[4], ns[4];                        // of the lane's pairs 2 i and 2 i + 1
  if (rotates) {
    const size_t at = static_cast<size_t>(turn) * (p.rotary / 2) + 8 * u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p.cos + at) + i);
      const float4 e = __ldg(reinterpret_cast<const float4*>(p.sin + at) + i);
      c[2 * i] = make_float2(a.x, a.y); c[2 * i + 1] = make_float2(a.z, a.w);
      s[2 * i] = make_float2(e.x, e.y); s[2 * i + 1] = make_float2(e.z, e.w);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) ns[i] = make_float2(-s[i].x, -s[i].y);
  }

#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int slot = (part * U + j) * SPW + lane / L;
    const bool is_q = slot < p.H, is_v = slot >= p.H + p.H_kv;
    const bool rot = rotates && !is_v;
    const bool sp = rot && !INTER;
    const uint32_t in[8] = {x0[j].x, x0[j].y, x0[j].z, x0[j].w, x1[j].x, x1[j].y, x1[j].z, x1[j].w};
    float f[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[2 * i] = bf16_lo(in[i]);
      f[2 * i + 1] = bf16_hi(in[i]);
    }
    if (rot) {
      // two pairs at a time: their first sides A and second sides E, which lie in the lane's vectors 0
      // and 1, or side by side
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        constexpr int step = INTER ? 2 : 1;
        const int a = INTER ? 4 * i : 2 * i, e = INTER ? 4 * i + 1 : 8 + 2 * i;
        const float2 A = make_float2(f[a], f[a + step]), E = make_float2(f[e], f[e + step]);
        const float2 y1 = ffma2(fmul2(A, c[i]), one, fmul2(E, ns[i]));
        const float2 y2 = ffma2(fmul2(E, c[i]), one, fmul2(A, s[i]));
        f[a] = y1.x; f[a + step] = y1.y;
        f[e] = y2.x; f[e + step] = y2.y;
      }
    }
    const int v0 = sp ? u : 2 * u, v1 = sp ? u + r16 : 2 * u + 1;
    // (a pass of query heads only, the same for the whole warp, has nothing to quantise)
    if (Q4 && (part * U + j) * SPW + SPW > p.H) {
      uint32_t code[2], scale[2];
      quantise16(f, sp, is_v ? p.descale_v : p.descale_k, code, scale);
      if (slot < slots && !is_q) {
        const int h = slot - p.H - (is_v ? p.H_kv : 0);
        const size_t r = (static_cast<size_t>(page) * p.H_kv + h) * p.block_size + row;
        uint8_t* cd = (is_v ? p.v_codes : p.k_codes) + r * (D / 2);
        uint8_t* sc = (is_v ? p.v_scales : p.k_scales) + r * (D / 16);
        if (sp) {
          *reinterpret_cast<uint32_t*>(cd + 4 * v0) = code[0];
          *reinterpret_cast<uint32_t*>(cd + 4 * v1) = code[1];
          sc[((u & 1) ? v1 : v0) >> 1] = static_cast<uint8_t>((u & 1) ? scale[1] : scale[0]);
        } else {
          *reinterpret_cast<uint2*>(cd + 4 * v0) = make_uint2(code[0], code[1]);
          sc[u] = static_cast<uint8_t>(scale[0]);
        }
      }
    }
    if (slot < slots && (!Q4 || is_q)) {
      uint32_t out[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) out[i] = rot ? pack_bf16x2(f[2 * i], f[2 * i + 1]) : in[i];
      const int h = slot - (is_q ? 0 : is_v ? p.H + p.H_kv : p.H);
      uint16_t* dst = is_q ? p.q_out + (static_cast<size_t>(t) * p.H + h) * D
                           : (is_v ? p.v_cache : p.k_cache) +
                                 ((static_cast<size_t>(page) * p.block_size + row) * p.H_kv + h) * D;
      *reinterpret_cast<uint4*>(dst + 8 * v0) = make_uint4(out[0], out[1], out[2], out[3]);
      *reinterpret_cast<uint4*>(dst + 8 * v1) = make_uint4(out[4], out[5], out[6], out[7]);
    }
  }
}

struct GatherParams {
  const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  uint16_t *k, *v;                                // [total, H_kv, d]
  const int *cu, *seqlens, *table;
  int n_seqs, H_kv, total, max_blocks, block_size, num_blocks, warps_per_token;
  float descale_k, descale_v;
};

template <int D, int U>
__global__ void __launch_bounds__(kPagedThreads) gather_q4_kernel(const GatherParams p) {
  constexpr int L = D / 16;
  constexpr int SPW = 32 / L;
  const int lane = threadIdx.x & 31;
  const int w = blockIdx.x * (kPagedThreads / 32) + (threadIdx.x >> 5);
  const int t = w / p.warps_per_token;
  if (t >= p.total) return;
  const int part = w - t * p.warps_per_token;
  const int u = lane % L;
  int first, count, page, row;
  const int b = owner_of_token(p.cu, p.n_seqs, p.total, t, &first, &count, 410);
  if (b < 0) return;
  const int len = __ldg(p.seqlens + b);
  const int pos = len - count + (t - first);
  if (len < count) {
    if (lane == 0) report_device_error(FA_DEV_BAD_CONFIG, 411);
    return;
  }
  if (!place_of_token(p.table, p.max_blocks, p.block_size, p.num_blocks, b, len, pos, &page, &row, 412)) return;
  uint2 code[U];
  uint32_t scale[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int slot = (part * U + j) * SPW + lane / L;
    const bool is_v = slot >= p.H_kv;
    if (slot < 2 * p.H_kv) {
      const size_t r = (static_cast<size_t>(page) * p.H_kv + (is_v ? slot - p.H_kv : slot)) * p.block_size + row;
      code[j] = *(reinterpret_cast<const uint2*>((is_v ? p.v_codes : p.k_codes) + r * (D / 2)) + u);
      scale[j] = (is_v ? p.v_scales : p.k_scales)[r * (D / 16) + u];
    }
  }
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int slot = (part * U + j) * SPW + lane / L;
    if (slot >= 2 * p.H_kv) continue;
    const bool is_v = slot >= p.H_kv;
    const float descale = is_v ? p.descale_v : p.descale_k;
    const uint32_t s = e4m3x2_to_f16(scale[j] * 0x0101u);
    uint32_t h[2][4], out[8];
    e2m1x8_to_f16(code[j].x, h[0]);
    e2m1x8_to_f16(code[j].y, h[1]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = f16x2_to_f32(hmul2(h[i >> 2][i & 3], s));
      out[i] = pack_bf16x2(__fmul_rn(f.x, descale), __fmul_rn(f.y, descale));
    }
    uint16_t* dst = (is_v ? p.v : p.k) + (static_cast<size_t>(t) * p.H_kv + (is_v ? slot - p.H_kv : slot)) * D + 16 * u;
    *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
    *reinterpret_cast<uint4*>(dst + 8) = make_uint4(out[4], out[5], out[6], out[7]);
  }
}

// A warp takes U passes of a token.  One where the passes are too few to fill the GPU twice over, so
// that they spread (4 x 16 tokens of 96 heads: 3.0 us, 4.0 with eight passes a warp); else more, so that the search for
// the token's place (four dependent loads) is shared and more bytes are in flight behind it.  How
// many: 6, or 3 where that leaves fewer passes empty, the one or two that there are, or, in bf16 only, 8
// where none is empty then.  Measured on the GPU: 4 x 4096 tokens of 24 passes in bf16 with 2, 3, 6 and 8
// 142, 133, 129, 124 us; 24 mixed sequences of 12 passes in 4 bits with 2, 3, 4 and 6 239, 258, 237, 194; of
// 2 passes in 4 bits with 2, 3 and 4 44, 59, 68.
static bool few_passes(long long passes) { return passes < 152LL * 64; }

template <int D, bool Q4, bool INTER, int U>
static cudaError_t launch_append_u(AppendParams& p, long long passes, cudaStream_t stream) {
  p.warps_per_token = static_cast<int>((passes + U - 1) / U);
  const long long warps = static_cast<long long>(p.total) * p.warps_per_token;
  const long long grid = (warps + kPagedThreads / 32 - 1) / (kPagedThreads / 32);
  log_launch(Q4 ? "append_kernel<D, true, INTER, U>" : "append_kernel<D, false, INTER, U>", static_cast<unsigned long long>(grid), kPagedThreads, 0ull);
  append_kernel<D, Q4, INTER, U><<<static_cast<unsigned>(grid), kPagedThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int D, bool Q4, bool INTER>
static cudaError_t launch_append_d(const AppendArgs& a, cudaStream_t stream) {
  AppendParams p{};
  p.q = static_cast<const uint16_t*>(a.q); p.k = static_cast<const uint16_t*>(a.k);
  p.v = static_cast<const uint16_t*>(a.v); p.q_out = static_cast<uint16_t*>(a.q_out);
  if (Q4) {
    p.k_codes = static_cast<uint8_t*>(a.k_cache); p.v_codes = static_cast<uint8_t*>(a.v_cache);
    p.k_scales = a.k_scales; p.v_scales = a.v_scales;
  } else {
    p.k_cache = static_cast<uint16_t*>(a.k_cache); p.v_cache = static_cast<uint16_t*>(a.v_cache);
  }
  p.cos = a.cos; p.sin = a.sin; p.cu = a.cu; p.seqlens = a.seqlens; p.table = a.block_table;
  p.q_stride = a.q_stride; p.k_stride = a.k_stride; p.v_stride = a.v_stride;
  p.n_seqs = a.n_seqs; p.H = a.q ? a.H : 0; p.H_kv = a.H_kv; p.total = a.total;
  p.max_blocks = a.max_blocks; p.block_size = a.block_size; p.num_blocks = a.num_blocks;
  p.rotary = a.rotary; p.n_positions = a.n_positions;
  p.descale_k = a.descale_k; p.descale_v = a.descale_v; p.one = 1.f;
  p.positions = a.positions;
  const int per_pass = 32 / (D / 16);
  const int slots = p.H + 2 * p.H_kv;
  const long long passes = (slots + per_pass - 1) / per_pass;
  if (passes == 1 || few_passes(passes * p.total)) return launch_append_u<D, Q4, INTER, 1>(p, passes, stream);
  if (passes == 2) return launch_append_u<D, Q4, INTER, 2>(p, passes, stream);
  if constexpr (!Q4)
    if (passes % 8 == 0) return launch_append_u<D, Q4, INTER, 8>(p, passes, stream);
  if ((passes + 5) / 6 * 6 <= (passes + 2) / 3 * 3) return launch_append_u<D, Q4, INTER, 6>(p, passes, stream);
  return launch_append_u<D, Q4, INTER, 3>(p, passes, stream);
}

template <int D, bool Q4>
static cudaError_t launch_append_q(const AppendArgs& a, cudaStream_t stream) {
  return a.interleaved ? launch_append_d<D, Q4, true>(a, stream) : launch_append_d<D, Q4, false>(a, stream);
}

cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream) {
  if (a.k_scales) return a.d == 64 ? launch_append_q<64, true>(a, stream) : launch_append_q<128, true>(a, stream);
  return a.d == 64 ? launch_append_q<64, false>(a, stream) : launch_append_q<128, false>(a, stream);
}

template <int D, int U>
static cudaError_t launch_gather_u(GatherParams& p, long long passes, cudaStream_t stream) {
  p.warps_per_token = static_cast<int>((passes + U - 1) / U);
  const long long warps = static_cast<long long>(p.total) * p.warps_per_token;
  const long long grid = (warps + kPagedThreads / 32 - 1) / (kPagedThreads / 32);
  log_launch("gather_q4_kernel<D, U>", static_cast<unsigned long long>(grid), kPagedThreads, 0ull);
  gather_q4_kernel<D, U><<<static_cast<unsigned>(grid), kPagedThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
static cudaError_t launch_gather_d(const GatherArgs& a, cudaStream_t stream) {
  GatherParams p{};
  p.k_codes = a.k_codes; p.k_scales = a.k_scales; p.v_codes = a.v_codes; p.v_scales = a.v_scales;
  p.k = static_cast<uint16_t*>(a.k); p.v = static_cast<uint16_t*>(a.v);
  p.cu = a.cu; p.seqlens = a.seqlens; p.table = a.block_table;
  p.n_seqs = a.n_seqs; p.H_kv = a.H_kv; p.total = a.total; p.max_blocks = a.max_blocks;
  p.block_size = a.block_size; p.num_blocks = a.num_blocks;
  p.descale_k = a.descale_k; p.descale_v = a.descale_v;
  const int per_pass = 32 / (D / 16);
  const long long passes = (2LL * p.H_kv + per_pass - 1) / per_pass;
  // two passes a warp where there are (8 x 16384 tokens of 4 passes, with 1, 2 and 4: 140, 123, 167 us)
  if (passes == 1 || few_passes(passes * p.total)) return launch_gather_u<D, 1>(p, passes, stream);
  return launch_gather_u<D, 2>(p, passes, stream);
}

cudaError_t launch_gather_q4(const GatherArgs& a, cudaStream_t stream) {
  return a.d == 64 ? launch_gather_d<64>(a, stream) : launch_gather_d<128>(a, stream);
}

}  // namespace fa

FA_DEFINE_STATUS_FETCH(status_fetch_paged)
