// The 4-bit cache's number formats on the device, and the places of tokens in a paged cache.
//
// A row of d elements is d/2 code bytes (element 2i in the low four bits of byte i, 2i + 1 in the
// high four) and d/16 scale bytes.  A code is e2m1 (sign, 2 exponent bits, 1 mantissa bit: 0, 0.5,
// 1, 1.5, 2, 3, 4, 6 and their negatives), a scale e4m3.  A code has 2 significant bits and a scale
// 4, so code * scale has at most 6 and lies in [2^-10, 2688]: every product is an exact fp16 number.
#pragma once

#include "sm103_paged.cuh"

namespace fa {

// Four code bytes -> eight fp16 values, byte j's pair in out[j] (low half = low four bits).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&out)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3]) : "r"(w));
}

// Two scale bytes (in the low half of ``w``) -> two fp16 values (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

// Eight fp32 values rounded (to nearest even, saturating at +-6) to e2m1, element i in bits 4i..4i+3.
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float* y) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}

// Two fp32 values -> e4m3 (to nearest even, saturating at 448), ``lo`` in the low byte of 16 bits.
__device__ __forceinline__ uint32_t f32x2_to_e4m3(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %2, %1;\n\tcvt.u32.u16 %0, h;\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t w) {
  float2 f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "cvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}" : "=f"(f.x), "=f"(f.y) : "r"(w));
  return f;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The b with cu[b] <= t < cu[b+1] of ascending boundaries, found by the whole warp, 32 boundaries a
// step.  Whatever they hold, b stays in [0, n_seqs) and the search ends, since each step shrinks the range.
__device__ __forceinline__ int search_owner(const int* __restrict__ cu, int n_seqs, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n_seqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + step * (lane + 1);
    const bool before = at < hi && __ldg(cu + at) <= t;
    lo += __popc(__ballot_sync(0xffffffffu, before)) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// The sequence that owns packed token ``t``.  Returns -1 for a token at or behind cu[n_seqs] (a padding
// row), and for boundaries that do not enclose it (which are reported).
__device__ __forceinline__ int owner_of_token(const int* __restrict__ cu, int n_seqs, int total, int t,
                                              int* first, int* count, int where) {
  const int lane = threadIdx.x & 31;
  const int end = __ldg(cu + n_seqs);
  const int lo = search_owner(cu, n_seqs, t);
  const int a = __ldg(cu + lo), b = __ldg(cu + lo + 1);
  const bool padding = t >= end;
  if ((t == 0 && (end > total || end < 0)) || (!padding && (a > t || b <= t || a < 0 || b > total))) {
    if (lane == 0) report_device_error(FA_DEV_BAD_CONFIG, where);
    return -1;
  }
  *first = a;
  *count = b - a;
  return padding ? -1 : lo;
}

// Page and row of logical token ``pos`` of sequence b; false (reported) where the position or the
// page lies outside the cache.
__device__ __forceinline__ bool place_of_token(const int* __restrict__ table, int max_blocks,
                                               int block_size, int num_blocks, int b, int len, int pos,
                                               int* page, int* row, int where) {
  const int blk = pos / block_size;
  bool ok = pos >= 0 && pos < len && blk < max_blocks;
  *row = pos - blk * block_size;
  *page = ok ? __ldg(table + static_cast<size_t>(b) * max_blocks + blk) : -1;
  ok = ok && *page >= 0 && *page < num_blocks;
  if (!ok && (threadIdx.x & 31) == 0) report_device_error(FA_DEV_BAD_CONFIG, where);
  return ok;
}

// Weights for the product with V are fp16.  Their reference lies so far below a row's maximum (at the last
// time that it was moved: the maximum may since have grown by 8) that the largest is 2^7 to 2^15: a weight
// 2^-21 of it keeps fp16's 11 bits, and what is lost of smaller ones is 2^-32 of it at most.
constexpr float kQ4Lift = 7.f;

// The log-sum-exp of a row: reference M, sum L of its weights.  (Their lift is taken off both first: the
// logarithm of a large L has a coarse step.)
__device__ __forceinline__ float q4_lse(float M, float L) {
  return ((M + kQ4Lift) + log2f(L * 0x1p-7f)) * 0.6931471805599453f;
}

// A row's states: n of them, ``stride`` floats apart, the first one ``skip`` floats further on.  n = 0: no row.
struct Q4States {
  const float* base;
  size_t stride, skip;
  int n;
};

// Writes a row's result from its states (O~ [D], then reference and sum).  ``wpr`` warps share a row,
// every wpr-th state each, eight in flight at a time (a load takes about a microsecond here, so one warp
// that read 63 states one after the other took 30 us).  ``warp``: this warp in the block, of WARPS at most
// (1: warps that have nothing to do with one another); called by all warps of the block.
template <int D, int WARPS>
__device__ __forceinline__ void q4_join(const Q4States& x, int warp, int wpr, uint16_t* o, float* lse, float descale_v) {
  constexpr int V = D / 64;                                    // pairs of elements a lane
  constexpr int AT_ONCE = 8;
  const int lane = threadIdx.x & 31, w = WARPS == 1 ? 0 : warp % wpr;
  if (WARPS == 1) wpr = 1;
  float M = -INFINITY, L = 0.f;
  float2 acc[V];
#pragma unroll
  for (int k = 0; k < V; ++k) acc[k] = make_float2(0.f, 0.f);
  auto add = [&](float2 ml, const float2 (&v)[V]) {
    if (ml.y == 0.f) return;                                   // no keys (a sum that is no number goes on)
    const float top = fmaxf(M, ml.x);
    const float alpha = top == M ? 1.f : fast_exp2(M - top), wt = fast_exp2(ml.x - top);
    M = top;
    L = fmaf(L, alpha, wt * ml.y);
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = ffma2(make_float2(wt, wt), v[k], fmul2(acc[k], make_float2(alpha, alpha)));
  };
  for (int i0 = w; i0 < x.n; i0 += wpr * AT_ONCE) {
    float2 ml[AT_ONCE], v[AT_ONCE][V];
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
      const int i = i0 + j * wpr;
      ml[j] = make_float2(0.f, 0.f);
      if (i < x.n) {
        const float* st = x.base + i * x.stride + (i == 0 ? x.skip : 0);
        ml[j] = *reinterpret_cast<const float2*>(st + D);
#pragma unroll
        for (int k = 0; k < V; ++k) v[j][k] = *reinterpret_cast<const float2*>(st + 64 * k + 2 * lane);
      }
    }
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) add(ml[j], v[j]);
  }
  if constexpr (WARPS > 1) {
    __shared__ float2 ml_of[WARPS], acc_of[WARPS][V][32];
    __syncthreads();                                           // (the row before has been read)
    if (w > 0) {
      if (lane == 0) ml_of[warp] = make_float2(M, L);
#pragma unroll
      for (int k = 0; k < V; ++k) acc_of[warp][k][lane] = acc[k];
    }
    __syncthreads();
    if (w > 0) return;
    for (int i = 1; i < wpr; ++i) {
      float2 v[V];
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] = acc_of[warp + i][k][lane];
      add(ml_of[warp + i], v);
    }
  }
  if (x.n == 0) return;
  const bool none = L == 0.f;
  const float inv = none ? 0.f : descale_v / L;
#pragma unroll
  for (int k = 0; k < V; ++k)
    *reinterpret_cast<uint32_t*>(o + 64 * k + 2 * lane) = none ? 0u : pack_bf16x2(acc[k].x * inv, acc[k].y * inv);
  if (lane == 0) *lse = none ? -INFINITY : q4_lse(M, L);
}

// Warps a row: all four of a block while the rows are few enough to run side by side all the same
// (one sequence of 8000 tokens and 8 key heads: 14 us, one warp a row 23; 2048 rows of 4 tokens of 16
// sequences: 35 us, 33).
inline int q4_join_warps(long long rows) { return rows <= 1024 ? 4 : 1; }

// The join runs behind the chunks on the stream, but may start while their last CTAs run
// (programmatic dependent launch): it reads lengths and boundaries, then waits for the states.
template <typename... P, typename... A>
static cudaError_t launch_join(void (*kernel)(P...), dim3 blocks, unsigned threads, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = blocks;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace fa
