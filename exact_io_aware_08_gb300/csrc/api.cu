// C ABI of libfa (declared in include/fa.h): argument validation, workspace carving, dispatch
// to the kernel launchers, device-status collection.  Nothing here allocates memory or falls
// back to another implementation: an unsupported call returns an error before any launch.
#include <cmath>
#include <cstdlib>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "../../include/fa.h"
#include "fa_kernels.h"

namespace fa {
// Process-wide diagnostic counters (fa_debug_counters); read by the launchers.
unsigned long long* g_debug_counters = nullptr;
unsigned long long* debug_counters() { return g_debug_counters; }

void log_launch(const char* kernel, unsigned long long grid, unsigned threads, unsigned long long smem) {
  static const bool on = [] {
    const char* v = std::getenv("FA_LOG");
    return v != nullptr && v[0] != '\0' && std::strcmp(v, "0") != 0;
  }();
  if (on) std::fprintf(stderr, "[fa] launch %s grid=%llu block=%u smem=%llu\n", kernel, grid, threads, smem);
}
}  // namespace fa

namespace {

thread_local char g_msg[512] = "no error";

fa_status_t fail(fa_status_t st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return st;
}

fa_status_t cuda_fail(cudaError_t e, const char* what) {
  return fail(FA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Shared shape checks.  Returns FA_OK or an error (message set).
fa_status_t check_shape(int B, int H, int n_q, int n_kv, int d, float scale) {
  if (B < 1 || H < 1) return fail(FA_ERR_INVALID_ARG, "B and H must be >= 1 (got B=%d H=%d)", B, H);
  if (n_q < 0 || n_kv < 0)
    return fail(FA_ERR_INVALID_ARG, "sequence lengths must be >= 0 (got N_q=%d N_kv=%d)", n_q, n_kv);
  if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED, "head dim d=%d not supported (64 or 128)", d);
  if (!std::isfinite(scale) || !(scale > 0.f))
    return fail(FA_ERR_INVALID_ARG, "scale must be finite and > 0 (got %g)", static_cast<double>(scale));
  const long long bh = static_cast<long long>(B) * H;
  if (bh > (1LL << 30)) return fail(FA_ERR_UNSUPPORTED, "B*H=%lld too large", bh);
  const long long lim = (1LL << 31) / d;
  if (n_q >= lim || n_kv >= lim)
    return fail(FA_ERR_UNSUPPORTED, "sequence length too large for d=%d (limit %lld)", d, lim);
  // grid of (query tiles x heads) must fit in gridDim.x
  const long long tiles = (static_cast<long long>(n_q) + 127) / 128;
  if (tiles * bh >= (1LL << 31)) return fail(FA_ERR_UNSUPPORTED, "too many (tile, head) work items");
  return FA_OK;
}

// The decode kernels index their (b, h, chunk) work items with 32-bit ints.
fa_status_t check_decode_items(int B, int H, int n_splits) {
  const long long items = static_cast<long long>(B) * H * n_splits;
  if (items >= (1LL << 31))
    return fail(FA_ERR_UNSUPPORTED, "B*H*n_splits=%lld too large (limit 2^31 - 1)", items);
  return FA_OK;
}

}  // namespace

extern "C" {

const char* fa_status_string(fa_status_t s) {
  switch (s) {
    case FA_OK: return "FA_OK";
    case FA_ERR_INVALID_ARG: return "FA_ERR_INVALID_ARG";
    case FA_ERR_UNSUPPORTED: return "FA_ERR_UNSUPPORTED";
    case FA_ERR_WORKSPACE: return "FA_ERR_WORKSPACE";
    case FA_ERR_CUDA: return "FA_ERR_CUDA";
    case FA_ERR_DEVICE_TIMEOUT: return "FA_ERR_DEVICE_TIMEOUT";
  }
  return "FA_ERR_UNKNOWN";
}

const char* fa_last_error_message(void) { return g_msg; }

fa_status_t fa_fwd(const fa_bf16_t* q, const fa_bf16_t* k, const fa_bf16_t* v, fa_bf16_t* o,
                   float* lse, int B, int H, int N_q, int N_kv, int d, float scale, int causal,
                   void* stream) {
  fa_status_t st = check_shape(B, H, N_q, N_kv, d, scale);
  if (st != FA_OK) return st;
  if (causal && N_q != N_kv)
    return fail(FA_ERR_UNSUPPORTED, "causal requires N_q == N_kv (got %d, %d)", N_q, N_kv);
  if (N_q == 0) return FA_OK;
  if (!q || !o || !lse || (N_kv > 0 && (!k || !v)))
    return fail(FA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return fail(FA_ERR_INVALID_ARG, "arrays must be 16-byte aligned");
  fa::FwdArgs a{q, k ? k : q, v ? v : q, o, lse, B, H, N_q, N_kv, d, scale, causal ? 1 : 0};
  if (N_kv == 0) { a.k = q; a.v = q; }   // maps need a valid base; no key tile is read
  cudaError_t e = fa::launch_fwd(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "fa_fwd launch");
  return FA_OK;
}

fa_status_t fa_fwd_fp8(const fa_e4m3_t* q, const fa_e4m3_t* k, const fa_e4m3_t* v, fa_bf16_t* o,
                       float* lse, int B, int H, int N_q, int N_kv, int d, float scale,
                       float descale_q, float descale_k, float descale_v, int causal,
                       void* stream) {
  fa_status_t st = check_shape(B, H, N_q, N_kv, d, scale);
  if (st != FA_OK) return st;
  if (d != 128) return fail(FA_ERR_UNSUPPORTED, "the fp8 forward supports d = 128 only (got %d)", d);
  for (float ds : {descale_q, descale_k, descale_v})
    if (!std::isfinite(ds) || !(ds > 0.f))
      return fail(FA_ERR_INVALID_ARG, "descale factors must be finite and > 0 (got %g)",
                  static_cast<double>(ds));
  if (!std::isfinite(scale * descale_q * descale_k) || !(scale * descale_q * descale_k > 0.f))
    return fail(FA_ERR_INVALID_ARG, "scale * descale_q * descale_k must be a finite positive float");
  if (causal && N_q != N_kv)
    return fail(FA_ERR_UNSUPPORTED, "causal requires N_q == N_kv (got %d, %d)", N_q, N_kv);
  if (N_q == 0) return FA_OK;
  if (!q || !o || !lse || (N_kv > 0 && (!k || !v)))
    return fail(FA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return fail(FA_ERR_INVALID_ARG, "arrays must be 16-byte aligned");
  fa::FwdArgs a{q, k ? k : q, v ? v : q, o, lse, B, H, N_q, N_kv, d, scale, causal ? 1 : 0};
  if (N_kv == 0) { a.k = q; a.v = q; }
  a.descale_q = descale_q;
  a.descale_k = descale_k;
  a.descale_v = descale_v;
  cudaError_t e = fa::launch_fwd_fp8(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "fa_fwd_fp8 launch");
  return FA_OK;
}

fa_status_t fa_fwd_varlen(const fa_bf16_t* q, const fa_bf16_t* k, const fa_bf16_t* v,
                          fa_bf16_t* o, float* lse, const int* cu_seqlens_q,
                          const int* cu_seqlens_k, int n_seqs, int H, int total_q, int total_k,
                          int max_seqlen_q, int max_seqlen_k, int d, float scale, int causal,
                          void* stream) {
  if (n_seqs < 1) return fail(FA_ERR_INVALID_ARG, "n_seqs must be >= 1 (got %d)", n_seqs);
  if (total_q < 0 || total_k < 0 || max_seqlen_q < 0 || max_seqlen_k < 0)
    return fail(FA_ERR_INVALID_ARG, "totals and max sequence lengths must be >= 0");
  if (max_seqlen_q > total_q || max_seqlen_k > total_k)
    return fail(FA_ERR_INVALID_ARG, "max_seqlen exceeds the total token count");
  fa_status_t st = check_shape(1, H, max_seqlen_q, max_seqlen_k, d, scale);
  if (st != FA_OK) return st;
  const long long lim = (1LL << 31) / (static_cast<long long>(d) * H);
  if (total_q >= lim || total_k >= lim)
    return fail(FA_ERR_UNSUPPORTED, "total tokens too large for H=%d d=%d", H, d);
  const long long items = ((static_cast<long long>(max_seqlen_q) + 255) / 256) * n_seqs * H;
  if (items >= (1LL << 31)) return fail(FA_ERR_UNSUPPORTED, "too many (block, sequence, head) items");
  if (total_q == 0 || max_seqlen_q == 0) return FA_OK;
  if (!q || !o || !lse || !cu_seqlens_q || !cu_seqlens_k || (total_k > 0 && (!k || !v)))
    return fail(FA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return fail(FA_ERR_INVALID_ARG, "arrays must be 16-byte aligned");
  fa::FwdVarlenArgs a{};
  a.q = q; a.k = total_k ? k : q; a.v = total_k ? v : q; a.o = o; a.lse = lse;
  a.cu_q = cu_seqlens_q; a.cu_k = cu_seqlens_k;
  a.n_seqs = n_seqs; a.H = H; a.total_q = total_q; a.total_k = total_k;
  a.max_seqlen_q = max_seqlen_q; a.max_seqlen_k = max_seqlen_k; a.d = d; a.scale = scale;
  a.causal = causal ? 1 : 0;
  cudaError_t e = fa::launch_fwd_varlen(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "fa_fwd_varlen launch");
  return FA_OK;
}

size_t fa_bwd_workspace_size(int B, int H, int N_q, int N_kv, int d) {
  if (B < 1 || H < 1 || N_q < 0 || N_kv < 0 || (d != 64 && d != 128)) return 0;
  return fa::bwd_dq_acc_bytes(B, H, N_q, d) + fa::bwd_delta_bytes(B, H, N_q);
}

}  // extern "C"

namespace {

// Validation shared by fa_bwd and its three steps.  ``need`` selects which arrays must be
// present: bit i for argument i of {q, k, v, o, lse, dO, dq, dk, dv}.
fa_status_t check_bwd(const void* const (&ptrs)[9], unsigned need, const void* ws, size_t ws_bytes,
                      int B, int H, int N_q, int N_kv, int d, float scale, int causal,
                      fa::BwdArgs* a) {
  fa_status_t st = check_shape(B, H, N_q, N_kv, d, scale);
  if (st != FA_OK) return st;
  if (causal && N_q != N_kv)
    return fail(FA_ERR_UNSUPPORTED, "causal requires N_q == N_kv (got %d, %d)", N_q, N_kv);
  const bool rows_q[9] = {true, false, false, true, true, true, true, false, false};
  for (int i = 0; i < 9; ++i) {
    const bool nonempty = rows_q[i] ? N_q > 0 : N_kv > 0;
    if ((need >> i & 1u) && nonempty && !ptrs[i])
      return fail(FA_ERR_INVALID_ARG, "null pointer argument (#%d)", i);
    if (ptrs[i] && !aligned16(ptrs[i])) return fail(FA_ERR_INVALID_ARG, "arrays must be 16-byte aligned");
  }
  const size_t need_ws = fa_bwd_workspace_size(B, H, N_q, N_kv, d);
  if (!ws || ws_bytes < need_ws || (reinterpret_cast<uintptr_t>(ws) & 255u))
    return fail(FA_ERR_WORKSPACE, "workspace must be >= %zu bytes and 256-byte aligned (got %zu)",
                need_ws, ws_bytes);
  *a = fa::BwdArgs{};
  a->q = ptrs[0]; a->k = ptrs[1]; a->v = ptrs[2]; a->o = ptrs[3];
  a->lse = static_cast<const float*>(ptrs[4]); a->dO = ptrs[5];
  a->dq = const_cast<void*>(ptrs[6]); a->dk = const_cast<void*>(ptrs[7]);
  a->dv = const_cast<void*>(ptrs[8]);
  a->dq_acc = static_cast<float*>(const_cast<void*>(ws));
  a->delta = reinterpret_cast<float*>(static_cast<char*>(const_cast<void*>(ws)) +
                                      fa::bwd_dq_acc_bytes(B, H, N_q, d));
  a->B = B; a->H = H; a->n_q = N_q; a->n_kv = N_kv; a->d = d; a->scale = scale;
  a->causal = causal ? 1 : 0;
  return FA_OK;
}

constexpr unsigned kNeedAll = 0x1FFu;
constexpr unsigned kNeedPrep = (1u << 3) | (1u << 5);                                  // o, dO
constexpr unsigned kNeedMain = 1u | 2u | 4u | (1u << 4) | (1u << 5) | (1u << 7) | (1u << 8);
constexpr unsigned kNeedFinish = 1u << 6;                                              // dq

}  // namespace

extern "C" {

fa_status_t fa_bwd(const fa_bf16_t* q, const fa_bf16_t* k, const fa_bf16_t* v,
                   const fa_bf16_t* o, const float* lse, const fa_bf16_t* dO, fa_bf16_t* dq,
                   fa_bf16_t* dk, fa_bf16_t* dv, void* ws, size_t ws_bytes, int B, int H,
                   int N_q, int N_kv, int d, float scale, int causal, void* stream) {
  fa::BwdArgs a;
  const void* const ptrs[9] = {q, k, v, o, lse, dO, dq, dk, dv};
  fa_status_t st = check_bwd(ptrs, kNeedAll, ws, ws_bytes, B, H, N_q, N_kv, d, scale, causal, &a);
  if (st != FA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = fa::launch_bwd_prep(a, s);
  if (e == cudaSuccess) e = fa::launch_bwd_main(a, s);
  if (e == cudaSuccess) e = fa::launch_bwd_finish(a, s);
  if (e != cudaSuccess) return cuda_fail(e, "fa_bwd launch");
  return FA_OK;
}

fa_status_t fa_fwd_window(const fa_bf16_t* q, const fa_bf16_t* k, const fa_bf16_t* v,
                          fa_bf16_t* o, float* lse, int B, int H, int N, int d, float scale,
                          int window_left, int window_right, void* stream) {
  fa_status_t st = check_shape(B, H, N, N, d, scale);
  if (st != FA_OK) return st;
  if (N == 0) return FA_OK;
  if (!q || !k || !v || !o || !lse) return fail(FA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return fail(FA_ERR_INVALID_ARG, "arrays must be 16-byte aligned");
  fa::FwdArgs a{q, k, v, o, lse, B, H, N, N, d, scale, 0};
  a.windowed = true;
  a.win_left = window_left < 0 ? fa::kWinUnbounded : std::min(window_left, fa::kWinUnbounded);
  a.win_right = window_right < 0 ? fa::kWinUnbounded : std::min(window_right, fa::kWinUnbounded);
  cudaError_t e = fa::launch_fwd(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "fa_fwd_window launch");
  return FA_OK;
}

fa_status_t fa_bwd_window(const fa_bf16_t* q, const fa_bf16_t* k, const fa_bf16_t* v,
                          const fa_bf16_t* o, const float* lse, const fa_bf16_t* dO,
                          fa_bf16_t* dq, fa_bf16_t* dk, fa_bf16_t* dv, void* ws, size_t ws_bytes,
                          int B, int H, int N, int d, float scale, int window_left,
                          int window_right, void* stream) {
  fa::BwdArgs a;
  const void* const ptrs[9] = {q, k, v, o, lse, dO, dq, dk, dv};
  fa_status_t st = check_bwd(ptrs, kNeedAll, ws, ws_bytes, B, H, N, N, d, scale, 0, &a);
  if (st != FA_OK) return st;
  a.windowed = true;
  a.win_left = window_left < 0 ? fa::kWinUnbounded : std::min(window_left, fa::kWinUnbounded);
  a.win_right = window_right < 0 ? fa::kWinUnbounded : std::min(window_right, fa::kWinUnbounded);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = fa::launch_bwd_prep(a, s);
  if (e == cudaSuccess) e = fa::launch_bwd_main(a, s);
  if (e == cudaSuccess) e = fa::launch_bwd_finish(a, s);
  if (e != cudaSuccess) return cuda_fail(e, "fa_bwd_window launch");
  return FA_OK;
}

// Block-sparse calls: the mask must exist (unless a side is empty) and cover at most
// kBlockSparseMaxTiles key blocks.
static fa_status_t check_block_mask(const unsigned char* block_mask, int mask_per_head, int N_q,
                                    int N_kv) {
  if (mask_per_head != 0 && mask_per_head != 1)
    return fail(FA_ERR_INVALID_ARG, "mask_per_head must be 0 or 1 (got %d)", mask_per_head);
  if (N_q > 0 && N_kv > 0 && !block_mask) return fail(FA_ERR_INVALID_ARG, "null block_mask");
  const int kb = (N_kv + fa::kBlockSize - 1) / fa::kBlockSize;
  if (kb > fa::kBlockSparseMaxTiles)
    return fail(FA_ERR_UNSUPPORTED, "block-sparse attention covers at most %d key blocks (N_kv <= %d; got %d)",
                fa::kBlockSparseMaxTiles, fa::kBlockSparseMaxTiles * fa::kBlockSize, N_kv);
  return FA_OK;
}

fa_status_t fa_fwd_block_sparse(const fa_bf16_t* q, const fa_bf16_t* k, const fa_bf16_t* v,
                                fa_bf16_t* o, float* lse, int B, int H, int N_q, int N_kv, int d,
                                float scale, int causal, const unsigned char* block_mask,
                                int mask_per_head, void* stream) {
  fa_status_t st = check_shape(B, H, N_q, N_kv, d, scale);
  if (st != FA_OK) return st;
  if (causal && N_q != N_kv)
    return fail(FA_ERR_UNSUPPORTED, "causal requires N_q == N_kv (got %d, %d)", N_q, N_kv);
  st = check_block_mask(block_mask, mask_per_head, N_q, N_kv);
  if (st != FA_OK) return st;
  if (N_q == 0) return FA_OK;
  if (!q || !o || !lse || (N_kv > 0 && (!k || !v)))
    return fail(FA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return fail(FA_ERR_INVALID_ARG, "arrays must be 16-byte aligned");
  fa::FwdArgs a{q, k ? k : q, v ? v : q, o, lse, B, H, N_q, N_kv, d, scale, causal ? 1 : 0};
  if (N_kv == 0) {
    a.k = q;                             // no key at all: the plain kernel writes O = 0, lse = -inf
    a.v = q;
  } else {
    a.block_mask = reinterpret_cast<const uint8_t*>(block_mask);
    a.bm_per_head = mask_per_head;
  }
  cudaError_t e = fa::launch_fwd(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "fa_fwd_block_sparse launch");
  return FA_OK;
}

fa_status_t fa_bwd_block_sparse(const fa_bf16_t* q, const fa_bf16_t* k, const fa_bf16_t* v,
                                const fa_bf16_t* o, const float* lse, const fa_bf16_t* dO,
                                fa_bf16_t* dq, fa_bf16_t* dk, fa_bf16_t* dv, void* ws,
                                size_t ws_bytes, int B, int H, int N_q, int N_kv, int d,
                                float scale, int causal, const unsigned char* block_mask,
                                int mask_per_head, void* stream) {
  fa::BwdArgs a;
  const void* const ptrs[9] = {q, k, v, o, lse, dO, dq, dk, dv};
  fa_status_t st = check_bwd(ptrs, kNeedAll, ws, ws_bytes, B, H, N_q, N_kv, d, scale, causal, &a);
  if (st != FA_OK) return st;
  st = check_block_mask(block_mask, mask_per_head, N_q, N_kv);
  if (st != FA_OK) return st;
  a.block_mask = reinterpret_cast<const uint8_t*>(block_mask);
  a.bm_per_head = mask_per_head;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = fa::launch_bwd_prep(a, s);
  if (e == cudaSuccess) e = fa::launch_bwd_main(a, s);
  if (e == cudaSuccess) e = fa::launch_bwd_finish(a, s);
  if (e != cudaSuccess) return cuda_fail(e, "fa_bwd_block_sparse launch");
  return FA_OK;
}

fa_status_t fa_bwd_prep(const fa_bf16_t* o, const fa_bf16_t* dO, void* ws, size_t ws_bytes,
                        int B, int H, int N_q, int N_kv, int d, void* stream) {
  fa::BwdArgs a;
  const void* const ptrs[9] = {nullptr, nullptr, nullptr, o, nullptr, dO, nullptr, nullptr, nullptr};
  fa_status_t st = check_bwd(ptrs, kNeedPrep, ws, ws_bytes, B, H, N_q, N_kv, d, 1.f, 0, &a);
  if (st != FA_OK) return st;
  cudaError_t e = fa::launch_bwd_prep(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : cuda_fail(e, "fa_bwd_prep launch");
}

fa_status_t fa_bwd_main(const fa_bf16_t* q, const fa_bf16_t* k, const fa_bf16_t* v,
                        const float* lse, const fa_bf16_t* dO, fa_bf16_t* dk, fa_bf16_t* dv,
                        void* ws, size_t ws_bytes, int B, int H, int N_q, int N_kv, int d,
                        float scale, int causal, void* stream) {
  fa::BwdArgs a;
  const void* const ptrs[9] = {q, k, v, nullptr, lse, dO, nullptr, dk, dv};
  fa_status_t st = check_bwd(ptrs, kNeedMain, ws, ws_bytes, B, H, N_q, N_kv, d, scale, causal, &a);
  if (st != FA_OK) return st;
  cudaError_t e = fa::launch_bwd_main(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : cuda_fail(e, "fa_bwd_main launch");
}

fa_status_t fa_bwd_finish(fa_bf16_t* dq, const void* ws, size_t ws_bytes, int B, int H, int N_q,
                          int N_kv, int d, float scale, void* stream) {
  fa::BwdArgs a;
  const void* const ptrs[9] = {nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, dq, nullptr, nullptr};
  fa_status_t st = check_bwd(ptrs, kNeedFinish, ws, ws_bytes, B, H, N_q, N_kv, d, scale, 0, &a);
  if (st != FA_OK) return st;
  cudaError_t e = fa::launch_bwd_finish(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : cuda_fail(e, "fa_bwd_finish launch");
}

fa_status_t fa_bwd_varlen(const fa_bf16_t* q, const fa_bf16_t* k, const fa_bf16_t* v,
                          const fa_bf16_t* o, const float* lse, const fa_bf16_t* dO,
                          fa_bf16_t* dq, fa_bf16_t* dk, fa_bf16_t* dv, void* ws, size_t ws_bytes,
                          const int* cu_seqlens_q, const int* cu_seqlens_k, int n_seqs, int H,
                          int total_q, int total_k, int max_seqlen_q, int max_seqlen_k, int d,
                          float scale, int causal, void* stream) {
  if (n_seqs < 1) return fail(FA_ERR_INVALID_ARG, "n_seqs must be >= 1 (got %d)", n_seqs);
  if (total_q < 0 || total_k < 0 || max_seqlen_q < 0 || max_seqlen_k < 0)
    return fail(FA_ERR_INVALID_ARG, "totals and max sequence lengths must be >= 0");
  if (max_seqlen_q > total_q || max_seqlen_k > total_k)
    return fail(FA_ERR_INVALID_ARG, "max_seqlen exceeds the total token count");
  if (!cu_seqlens_q || !cu_seqlens_k) return fail(FA_ERR_INVALID_ARG, "null cu_seqlens");
  const long long lim = (1LL << 31) / (static_cast<long long>(d > 0 ? d : 1) * (H > 0 ? H : 1));
  if (total_q >= lim || total_k >= lim)
    return fail(FA_ERR_UNSUPPORTED, "total tokens too large for H=%d d=%d", H, d);
  const long long items = ((static_cast<long long>(max_seqlen_k) + 127) / 128) * n_seqs * (H > 0 ? H : 1);
  if (items >= (1LL << 31)) return fail(FA_ERR_UNSUPPORTED, "too many (key tile, sequence, head) items");
  // the packed layout is one [1, H, total, d]-sized problem for the prep and finish steps
  fa::BwdArgs a;
  const void* const ptrs[9] = {q, k, v, o, lse, dO, dq, dk, dv};
  fa_status_t st = check_bwd(ptrs, kNeedAll, ws, ws_bytes, 1, H, total_q, total_k, d, scale, 0, &a);
  if (st != FA_OK) return st;
  if (total_q == 0 && total_k == 0) return FA_OK;
  a.causal = causal ? 1 : 0;
  a.cu_q = cu_seqlens_q;
  a.cu_k = cu_seqlens_k;
  a.n_seqs = n_seqs;
  a.total_q = total_q;
  a.total_k = total_k;
  a.max_seqlen_q = max_seqlen_q;
  a.max_seqlen_k = max_seqlen_k;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = fa::launch_bwd_prep(a, s);
  if (e == cudaSuccess) e = fa::launch_bwd_main(a, s);
  if (e == cudaSuccess) e = fa::launch_bwd_finish(a, s);
  if (e != cudaSuccess) return cuda_fail(e, "fa_bwd_varlen launch");
  return FA_OK;
}

size_t fa_decode_workspace_size(int B, int H, int N_kv, int d, int n_splits) {
  if (B < 1 || H < 1 || N_kv < 0 || (d != 64 && d != 128)) return 0;
  if (n_splits <= 0) n_splits = fa::decode_auto_splits(B, H, N_kv);
  if (n_splits > fa::kDecodeMaxSplits) return 0;
  if (static_cast<long long>(B) * H * n_splits >= (1LL << 31)) return 0;
  return fa::decode_part_bytes(B, H, d, n_splits);
}

fa_status_t fa_decode_splitkv(const fa_bf16_t* q, const fa_bf16_t* k, const fa_bf16_t* v,
                              fa_bf16_t* o, float* lse, int B, int H, int N_kv, int d,
                              float scale, int n_splits, void* ws, size_t ws_bytes,
                              void* stream) {
  fa_status_t st = check_shape(B, H, 1, N_kv, d, scale);
  if (st != FA_OK) return st;
  if (n_splits > fa::kDecodeMaxSplits)
    return fail(FA_ERR_UNSUPPORTED, "n_splits=%d exceeds %d", n_splits, fa::kDecodeMaxSplits);
  if (n_splits <= 0) n_splits = fa::decode_auto_splits(B, H, N_kv);
  if ((st = check_decode_items(B, H, n_splits)) != FA_OK) return st;
  if (!q || !o || !lse || (N_kv > 0 && (!k || !v)))
    return fail(FA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return fail(FA_ERR_INVALID_ARG, "arrays must be 16-byte aligned");
  const size_t need_ws = fa::decode_part_bytes(B, H, d, n_splits);
  if (!ws || ws_bytes < need_ws || !aligned16(ws))
    return fail(FA_ERR_WORKSPACE, "workspace must be >= %zu bytes and 16-byte aligned (got %zu)",
                need_ws, ws_bytes);
  fa::DecodeArgs a{};
  a.q = q; a.k = N_kv ? k : q; a.v = N_kv ? v : q; a.o = o; a.lse = lse;
  a.part = static_cast<float*>(ws);
  a.B = B; a.H = H; a.n_kv = N_kv; a.d = d; a.scale = scale; a.n_splits = n_splits;
  a.chunk = fa::decode_chunk(N_kv, n_splits);
  cudaError_t e = fa::launch_decode(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "fa_decode_splitkv launch");
  return FA_OK;
}

fa_status_t fa_decode_splitkv_noalloc(const fa_bf16_t* q, const fa_bf16_t* k, const fa_bf16_t* v,
                                      fa_bf16_t* o, float* lse, int B, int H, int N_kv, int d,
                                      float scale, int n_splits, void* stream) {
  fa_status_t st = check_shape(B, H, 1, N_kv, d, scale);
  if (st != FA_OK) return st;
  if (n_splits > fa::kDecodeMaxSplits)
    return fail(FA_ERR_UNSUPPORTED, "n_splits=%d exceeds %d", n_splits, fa::kDecodeMaxSplits);
  if (n_splits <= 0) n_splits = fa::decode_auto_splits(B, H, N_kv);
  if ((st = check_decode_items(B, H, n_splits)) != FA_OK) return st;
  if (!q || !o || !lse || (N_kv > 0 && (!k || !v)))
    return fail(FA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return fail(FA_ERR_INVALID_ARG, "arrays must be 16-byte aligned");
  const size_t need = fa::decode_part_bytes(B, H, d, n_splits);
  if (need > fa::kDecodeNoallocScratchBytes)
    return fail(FA_ERR_UNSUPPORTED,
                "fa_decode_splitkv_noalloc: B*H*n_splits*(d+2)*4 = %zu bytes exceeds the fixed "
                "scratch of %zu bytes; use fa_decode_splitkv with a workspace or fewer splits",
                need, fa::kDecodeNoallocScratchBytes);
  float* scratch = nullptr;
  cudaError_t e = fa::decode_noalloc_scratch(&scratch);
  if (e != cudaSuccess) return cuda_fail(e, "fa_decode_splitkv_noalloc scratch lookup");
  fa::DecodeArgs a{};
  a.q = q; a.k = N_kv ? k : q; a.v = N_kv ? v : q; a.o = o; a.lse = lse;
  a.part = scratch;
  a.B = B; a.H = H; a.n_kv = N_kv; a.d = d; a.scale = scale; a.n_splits = n_splits;
  a.chunk = fa::decode_chunk(N_kv, n_splits);
  e = fa::launch_decode(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "fa_decode_splitkv_noalloc launch");
  return FA_OK;
}

fa_status_t fa_decode_paged(const fa_bf16_t* q, const fa_bf16_t* k_cache,
                            const fa_bf16_t* v_cache, fa_bf16_t* o, float* lse,
                            const int* block_table, const int* seqlens_k, int B, int H,
                            int max_blocks_per_seq, int block_size, int num_blocks,
                            int max_seqlen_k, int d, float scale, int n_splits, void* ws,
                            size_t ws_bytes, void* stream) {
  fa_status_t st = check_shape(B, H, 1, max_seqlen_k, d, scale);
  if (st != FA_OK) return st;
  if (block_size < 64 || block_size % 64 != 0)
    return fail(FA_ERR_UNSUPPORTED, "block_size must be a positive multiple of 64 (got %d)",
                block_size);
  if (num_blocks < 1 || max_blocks_per_seq < 1)
    return fail(FA_ERR_INVALID_ARG, "num_blocks and max_blocks_per_seq must be >= 1 (got %d, %d)",
                num_blocks, max_blocks_per_seq);
  if (static_cast<long long>(num_blocks) * block_size >= (1LL << 31))
    return fail(FA_ERR_UNSUPPORTED, "num_blocks * block_size must be < 2^31");
  if (static_cast<long long>(max_seqlen_k) > static_cast<long long>(max_blocks_per_seq) * block_size)
    return fail(FA_ERR_INVALID_ARG, "max_seqlen_k=%d exceeds max_blocks_per_seq * block_size",
                max_seqlen_k);
  if (n_splits > fa::kDecodeMaxSplits)
    return fail(FA_ERR_UNSUPPORTED, "n_splits=%d exceeds %d", n_splits, fa::kDecodeMaxSplits);
  if (n_splits <= 0) n_splits = fa::decode_auto_splits(B, H, max_seqlen_k);
  if ((st = check_decode_items(B, H, n_splits)) != FA_OK) return st;
  if (!q || !k_cache || !v_cache || !o || !lse || !block_table || !seqlens_k)
    return fail(FA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) ||
      !aligned16(lse))
    return fail(FA_ERR_INVALID_ARG, "arrays must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(seqlens_k)) & 3u)
    return fail(FA_ERR_INVALID_ARG, "block_table and seqlens_k must be 4-byte aligned");
  const size_t need_ws = fa::decode_part_bytes(B, H, d, n_splits);
  if (!ws || ws_bytes < need_ws || !aligned16(ws))
    return fail(FA_ERR_WORKSPACE, "workspace must be >= %zu bytes and 16-byte aligned (got %zu)",
                need_ws, ws_bytes);
  fa::DecodePagedArgs a{};
  a.q = q; a.k_cache = k_cache; a.v_cache = v_cache; a.o = o; a.lse = lse;
  a.part = static_cast<float*>(ws);
  a.block_table = block_table; a.seqlens = seqlens_k;
  a.B = B; a.H = H; a.d = d; a.num_blocks = num_blocks; a.block_size = block_size;
  a.max_blocks = max_blocks_per_seq; a.max_seqlen = max_seqlen_k;
  a.scale = scale; a.n_splits = n_splits;
  a.chunk = fa::decode_chunk(max_seqlen_k, n_splits);
  cudaError_t e = fa::launch_decode_paged(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "fa_decode_paged launch");
  return FA_OK;
}

}  // extern "C"

namespace {

// Shape and pages of the paged-cache calls.  ``granule``: the block size must be a multiple of it.
fa_status_t check_paged(int n_seqs, int H, int H_kv, int d, int max_blocks_per_seq, int block_size,
                        int num_blocks, int granule) {
  if (n_seqs < 1 || H_kv < 1 || H < 0)
    return fail(FA_ERR_INVALID_ARG, "n_seqs and H_kv must be >= 1 and H >= 0 (got %d, %d, %d)", n_seqs, H_kv, H);
  if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED, "head dim d=%d not supported (64 or 128)", d);
  if (num_blocks < 1 || max_blocks_per_seq < 1)
    return fail(FA_ERR_INVALID_ARG, "num_blocks and max_blocks_per_seq must be >= 1 (got %d, %d)",
                num_blocks, max_blocks_per_seq);
  if (block_size < granule || block_size % granule != 0)
    return fail(FA_ERR_UNSUPPORTED, "block_size must be a positive multiple of %d (got %d)", granule, block_size);
  const long long rows = static_cast<long long>(num_blocks) * block_size;
  if (rows >= (1LL << 31) || rows * H_kv >= (1LL << 31))
    return fail(FA_ERR_UNSUPPORTED, "num_blocks * block_size * H_kv must be < 2^31");
  if (static_cast<long long>(max_blocks_per_seq) * block_size >= (1LL << 31))
    return fail(FA_ERR_UNSUPPORTED, "max_blocks_per_seq * block_size must be < 2^31");
  return FA_OK;
}

fa_status_t check_descale(float descale) {
  // 6 * descale and 448 * descale are formed in fp32
  if (!std::isfinite(descale) || !(descale >= 1e-30f) || !(descale <= 1e30f))
    return fail(FA_ERR_INVALID_ARG, "descale factors must be in [1e-30, 1e30] (got %g)", static_cast<double>(descale));
  return FA_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

fa_status_t check_index_arrays(const int* a, const int* b, const int* c) {
  if (!a || !b || !c) return fail(FA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned4(a) || !aligned4(b) || !aligned4(c))
    return fail(FA_ERR_INVALID_ARG, "block_table, seqlens_k and cu_seqlens must be 4-byte aligned");
  return FA_OK;
}

fa_status_t append(const void* q, const void* k, const void* v, void* q_out, void* k_cache, void* k_scales,
                   void* v_cache, void* v_scales, bool q4, const float* cos, const float* sin, const int* cu,
                   const int* seqlens, const int* table, int n_seqs, int H, int H_kv, int total,
                   long long q_stride, long long k_stride, long long v_stride, int max_blocks, int block_size,
                   int num_blocks, int d, int rotary, int interleaved, int n_positions, float descale_k,
                   float descale_v, void* stream, const char* name) {
  fa_status_t st = check_paged(n_seqs, H, H_kv, d, max_blocks, block_size, num_blocks, q4 ? 16 : 1);
  if (st != FA_OK) return st;
  if (total < 0) return fail(FA_ERR_INVALID_ARG, "total must be >= 0 (got %d)", total);
  if (rotary < 0 || rotary > d || rotary % 32 != 0)
    return fail(FA_ERR_UNSUPPORTED, "rotary_dim must be a multiple of 32 in [0, d] (got %d)", rotary);
  if (interleaved != 0 && interleaved != 1)
    return fail(FA_ERR_INVALID_ARG, "interleaved must be 0 or 1 (got %d)", interleaved);
  if (q && H < 1) return fail(FA_ERR_INVALID_ARG, "H must be >= 1 with queries (got %d)", H);
  if (!q) H = 0;
  if (q4) {
    if ((st = check_descale(descale_k)) != FA_OK || (st = check_descale(descale_v)) != FA_OK) return st;
  }
  // one warp per 32 lanes of a token's heads: the warps are counted in an int
  const long long warps = (static_cast<long long>(H) + 2LL * H_kv + 1) * total;
  if (warps >= (1LL << 31)) return fail(FA_ERR_UNSUPPORTED, "total * (H + 2 H_kv) must be < 2^31");
  if (total == 0) return FA_OK;
  if (!k || !v || !k_cache || !v_cache || (q4 && (!k_scales || !v_scales)) || (q && !q_out) ||
      (rotary > 0 && (!cos || !sin)))
    return fail(FA_ERR_INVALID_ARG, "null pointer argument");
  if ((st = check_index_arrays(cu, seqlens, table)) != FA_OK) return st;
  if (rotary > 0 && n_positions < 1) return fail(FA_ERR_INVALID_ARG, "n_positions must be >= 1 (got %d)", n_positions);
  for (const void* x : {q, k, v, static_cast<const void*>(q_out), static_cast<const void*>(k_cache),
                        static_cast<const void*>(v_cache), static_cast<const void*>(k_scales),
                        static_cast<const void*>(v_scales), static_cast<const void*>(rotary ? cos : nullptr),
                        static_cast<const void*>(rotary ? sin : nullptr)})
    if (!aligned16(x)) return fail(FA_ERR_INVALID_ARG, "arrays must be 16-byte aligned");
  const long long need[3] = {static_cast<long long>(H) * d, static_cast<long long>(H_kv) * d, static_cast<long long>(H_kv) * d};
  const long long have[3] = {q_stride, k_stride, v_stride};
  for (int i = q ? 0 : 1; i < 3; ++i)
    if ((total > 1 && have[i] < need[i]) || have[i] < 0 || have[i] % 8 != 0 || have[i] >= (1LL << 40))
      return fail(FA_ERR_INVALID_ARG, "token strides must be multiples of 8 elements of at least a token's heads (got %lld)", have[i]);
  fa::AppendArgs a{};
  a.q = q; a.k = k; a.v = v; a.q_out = q_out; a.k_cache = k_cache; a.v_cache = v_cache;
  a.k_scales = static_cast<uint8_t*>(k_scales); a.v_scales = static_cast<uint8_t*>(v_scales);
  a.cos = cos; a.sin = sin; a.cu = cu; a.seqlens = seqlens; a.block_table = table;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.n_seqs = n_seqs; a.H = H; a.H_kv = H_kv; a.total = total; a.max_blocks = max_blocks;
  a.block_size = block_size; a.num_blocks = num_blocks; a.d = d; a.rotary = rotary;
  a.interleaved = interleaved; a.n_positions = n_positions; a.descale_k = descale_k; a.descale_v = descale_v;
  cudaError_t e = fa::launch_append(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : cuda_fail(e, name);
}

// Split count of a 4-bit attention call (0: the library shares the work out itself), or an error.
fa_status_t q4_splits(int n_seqs, int H, int H_kv, int max_seqlen_q, int d, int* n_splits) {
  const long long items = fa::q4_items(n_seqs, H, H_kv, max_seqlen_q, d);
  if (*n_splits > fa::kDecodeMaxSplits)
    return fail(FA_ERR_UNSUPPORTED, "n_splits=%d exceeds %d", *n_splits, fa::kDecodeMaxSplits);
  if (*n_splits < 0) *n_splits = 0;
  if (items >= (1LL << 30) || items * 2 * *n_splits >= (1LL << 31))
    return fail(FA_ERR_UNSUPPORTED, "too many (sequence, key head, row block, split) items");
  return FA_OK;
}

size_t q4_part_bytes(int total_q, int H, int H_kv, int max_seqlen_q, int d, int n_splits) {
  return n_splits == 0 ? fa::q4_auto_bytes(H, H_kv, max_seqlen_q, d) : n_splits == 1 ? 16 : fa::decode_part_bytes(total_q, H, d, n_splits);
}

size_t q4_workspace(int n_seqs, int H, int H_kv, int total_q, int max_seqlen_q, int max_seqlen_k, int d, int n_splits) {
  if (n_seqs < 1 || H < 1 || H_kv < 1 || H % H_kv != 0 || total_q < 0 || max_seqlen_q < 0 || max_seqlen_k < 0 ||
      (d != 64 && d != 128) || static_cast<long long>(total_q) * H >= (1LL << 31))
    return 0;
  if (q4_splits(n_seqs, H, H_kv, max_seqlen_q, d, &n_splits) != FA_OK) return 0;
  return q4_part_bytes(total_q, H, H_kv, max_seqlen_q, d, n_splits);
}

fa_status_t attend_q4(const void* q, const void* k_codes, const void* k_scales, const void* v_codes,
                      const void* v_scales, void* o, float* lse, const int* cu_q, const int* seqlens,
                      const int* table, int n_seqs, int H, int H_kv, int total_q, int max_seqlen_q,
                      int max_blocks, int block_size, int num_blocks, int max_seqlen_k, int d, float scale,
                      float descale_k, float descale_v, int causal, int n_splits, void* ws, size_t ws_bytes,
                      void* stream, const char* name) {
  fa_status_t st = check_paged(n_seqs, H, H_kv, d, max_blocks, block_size, num_blocks, 16);
  if (st != FA_OK) return st;
  if (H < 1 || H % H_kv != 0) return fail(FA_ERR_INVALID_ARG, "H must be a positive multiple of H_kv (got %d, %d)", H, H_kv);
  if (total_q < 0 || max_seqlen_q < 0 || max_seqlen_k < 0)
    return fail(FA_ERR_INVALID_ARG, "totals and max sequence lengths must be >= 0");
  if (max_seqlen_q > total_q) return fail(FA_ERR_INVALID_ARG, "max_seqlen exceeds the total token count");
  if (static_cast<long long>(max_seqlen_k) > static_cast<long long>(max_blocks) * block_size)
    return fail(FA_ERR_INVALID_ARG, "max_seqlen_k=%d exceeds max_blocks_per_seq * block_size", max_seqlen_k);
  if (max_seqlen_k >= (1LL << 31) / d) return fail(FA_ERR_UNSUPPORTED, "max_seqlen_k too large for d=%d", d);
  if (static_cast<long long>(total_q) * H >= (1LL << 31)) return fail(FA_ERR_UNSUPPORTED, "total_q * H must be < 2^31");
  if (!std::isfinite(scale) || !(scale > 0.f))
    return fail(FA_ERR_INVALID_ARG, "scale must be finite and > 0 (got %g)", static_cast<double>(scale));
  if ((st = check_descale(descale_k)) != FA_OK || (st = check_descale(descale_v)) != FA_OK) return st;
  const float score = scale * 1.4426950408889634f * descale_k;
  if (!(score >= 1e-34f) || !(score <= 1e34f))
    return fail(FA_ERR_INVALID_ARG, "scale * descale_k must be in about [1e-34, 1e34] (got %g)", static_cast<double>(score));
  if ((st = q4_splits(n_seqs, H, H_kv, max_seqlen_q, d, &n_splits)) != FA_OK) return st;
  // key steps of a sequence are counted in an int, those of all of them over the shares too
  if (fa::q4_items(1, H, H_kv, max_seqlen_q, d) * (max_seqlen_k / fa::kQ4Step + 1) >= (1LL << 31) ||
      fa::q4_items(n_seqs, H, H_kv, max_seqlen_q, d) * (max_seqlen_k / fa::kQ4Step + 1) >= (1LL << 38))
    return fail(FA_ERR_UNSUPPORTED, "too many (key head, row block, key step) units");
  if (total_q == 0 || max_seqlen_q == 0) return FA_OK;
  if (!q || !k_codes || !k_scales || !v_codes || !v_scales || !o || !lse)
    return fail(FA_ERR_INVALID_ARG, "null pointer argument");
  for (const void* x : {q, k_codes, k_scales, v_codes, v_scales, static_cast<const void*>(o), static_cast<const void*>(lse)})
    if (!aligned16(x)) return fail(FA_ERR_INVALID_ARG, "arrays must be 16-byte aligned");
  if ((st = check_index_arrays(cu_q ? cu_q : seqlens, seqlens, table)) != FA_OK) return st;
  if (n_splits != 1) {
    const size_t need = q4_part_bytes(total_q, H, H_kv, max_seqlen_q, d, n_splits);
    if (!ws || ws_bytes < need || !aligned16(ws))
      return fail(FA_ERR_WORKSPACE, "workspace must be >= %zu bytes and 16-byte aligned (got %zu)", need, ws_bytes);
  }
  fa::PagedQ4Args a{};
  a.q = q; a.o = o; a.lse = lse; a.part = static_cast<float*>(ws);
  a.k_codes = static_cast<const uint8_t*>(k_codes); a.k_scales = static_cast<const uint8_t*>(k_scales);
  a.v_codes = static_cast<const uint8_t*>(v_codes); a.v_scales = static_cast<const uint8_t*>(v_scales);
  a.cu_q = cu_q; a.seqlens = seqlens; a.block_table = table;
  a.n_seqs = n_seqs; a.H = H; a.H_kv = H_kv; a.total_q = total_q; a.max_seqlen_q = max_seqlen_q; a.d = d;
  a.num_blocks = num_blocks; a.block_size = block_size; a.max_blocks = max_blocks; a.max_seqlen_k = max_seqlen_k;
  a.causal = causal ? 1 : 0; a.scale = scale; a.descale_k = descale_k; a.descale_v = descale_v;
  a.n_splits = n_splits;
  a.chunk = n_splits ? fa::q4_chunk(max_seqlen_k, n_splits) : 0;
  cudaError_t e = fa::launch_attend_q4(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : cuda_fail(e, name);
}

}  // namespace

extern "C" {

fa_status_t fa_append_paged(const fa_bf16_t* q, const fa_bf16_t* k, const fa_bf16_t* v, fa_bf16_t* q_out,
                            fa_bf16_t* k_cache, fa_bf16_t* v_cache, const float* cos, const float* sin,
                            const int* cu_seqlens, const int* seqlens_k, const int* block_table, int n_seqs,
                            int H, int H_kv, int total, long long q_stride, long long k_stride,
                            long long v_stride, int max_blocks_per_seq, int block_size, int num_blocks, int d,
                            int rotary_dim, int interleaved, int n_positions, void* stream) {
  return append(q, k, v, q_out, k_cache, nullptr, v_cache, nullptr, false, cos, sin, cu_seqlens, seqlens_k,
                block_table, n_seqs, H, H_kv, total, q_stride, k_stride, v_stride, max_blocks_per_seq,
                block_size, num_blocks, d, rotary_dim, interleaved, n_positions, 1.f, 1.f, stream,
                "fa_append_paged launch");
}

fa_status_t fa_append_paged_q4(const fa_bf16_t* q, const fa_bf16_t* k, const fa_bf16_t* v, fa_bf16_t* q_out,
                               fa_e2m1x2_t* k_codes, fa_e4m3_t* k_scales, fa_e2m1x2_t* v_codes,
                               fa_e4m3_t* v_scales, const float* cos, const float* sin, const int* cu_seqlens,
                               const int* seqlens_k, const int* block_table, int n_seqs, int H, int H_kv,
                               int total, long long q_stride, long long k_stride, long long v_stride,
                               int max_blocks_per_seq, int block_size, int num_blocks, int d, int rotary_dim,
                               int interleaved, int n_positions, float descale_k, float descale_v, void* stream) {
  return append(q, k, v, q_out, k_codes, k_scales, v_codes, v_scales, true, cos, sin, cu_seqlens, seqlens_k,
                block_table, n_seqs, H, H_kv, total, q_stride, k_stride, v_stride, max_blocks_per_seq,
                block_size, num_blocks, d, rotary_dim, interleaved, n_positions, descale_k, descale_v, stream,
                "fa_append_paged_q4 launch");
}

fa_status_t fa_gather_paged_q4(const fa_e2m1x2_t* k_codes, const fa_e4m3_t* k_scales, const fa_e2m1x2_t* v_codes,
                               const fa_e4m3_t* v_scales, fa_bf16_t* k, fa_bf16_t* v, const int* cu_seqlens,
                               const int* seqlens_k, const int* block_table, int n_seqs, int H_kv, int total,
                               int max_blocks_per_seq, int block_size, int num_blocks, int d, float descale_k,
                               float descale_v, void* stream) {
  fa_status_t st = check_paged(n_seqs, 0, H_kv, d, max_blocks_per_seq, block_size, num_blocks, 16);
  if (st != FA_OK) return st;
  if (total < 0) return fail(FA_ERR_INVALID_ARG, "total must be >= 0 (got %d)", total);
  if ((st = check_descale(descale_k)) != FA_OK || (st = check_descale(descale_v)) != FA_OK) return st;
  if ((2LL * H_kv + 1) * total >= (1LL << 31)) return fail(FA_ERR_UNSUPPORTED, "total * H_kv too large");
  if (total == 0) return FA_OK;
  if (!k_codes || !k_scales || !v_codes || !v_scales || !k || !v) return fail(FA_ERR_INVALID_ARG, "null pointer argument");
  if ((st = check_index_arrays(cu_seqlens, seqlens_k, block_table)) != FA_OK) return st;
  for (const void* x : {static_cast<const void*>(k_codes), static_cast<const void*>(k_scales),
                        static_cast<const void*>(v_codes), static_cast<const void*>(v_scales),
                        static_cast<const void*>(k), static_cast<const void*>(v)})
    if (!aligned16(x)) return fail(FA_ERR_INVALID_ARG, "arrays must be 16-byte aligned");
  fa::GatherArgs a{k_codes, k_scales, v_codes, v_scales, k, v, cu_seqlens, seqlens_k, block_table,
                   n_seqs, H_kv, total, max_blocks_per_seq, block_size, num_blocks, d, descale_k, descale_v};
  cudaError_t e = fa::launch_gather_q4(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : cuda_fail(e, "fa_gather_paged_q4 launch");
}

size_t fa_decode_paged_q4_workspace_size(int B, int H, int H_kv, int max_seqlen_k, int d, int n_splits) {
  return q4_workspace(B, H, H_kv, B, 1, max_seqlen_k, d, n_splits);
}

fa_status_t fa_decode_paged_q4(const fa_bf16_t* q, const fa_e2m1x2_t* k_codes, const fa_e4m3_t* k_scales,
                               const fa_e2m1x2_t* v_codes, const fa_e4m3_t* v_scales, fa_bf16_t* o, float* lse,
                               const int* block_table, const int* seqlens_k, int B, int H, int H_kv,
                               int max_blocks_per_seq, int block_size, int num_blocks, int max_seqlen_k, int d,
                               float scale, float descale_k, float descale_v, int n_splits, void* ws,
                               size_t ws_bytes, void* stream) {
  return attend_q4(q, k_codes, k_scales, v_codes, v_scales, o, lse, nullptr, seqlens_k, block_table, B, H, H_kv,
                   B, 1, max_blocks_per_seq, block_size, num_blocks, max_seqlen_k, d, scale, descale_k, descale_v,
                   0, n_splits, ws, ws_bytes, stream, "fa_decode_paged_q4 launch");
}

size_t fa_fwd_paged_q4_workspace_size(int n_seqs, int H, int H_kv, int total_q, int max_seqlen_q,
                                      int max_seqlen_k, int d, int n_splits) {
  return q4_workspace(n_seqs, H, H_kv, total_q, max_seqlen_q, max_seqlen_k, d, n_splits);
}

fa_status_t fa_fwd_paged_q4(const fa_bf16_t* q, const fa_e2m1x2_t* k_codes, const fa_e4m3_t* k_scales,
                            const fa_e2m1x2_t* v_codes, const fa_e4m3_t* v_scales, fa_bf16_t* o, float* lse,
                            const int* cu_seqlens_q, const int* seqlens_k, const int* block_table, int n_seqs,
                            int H, int H_kv, int total_q, int max_seqlen_q, int max_blocks_per_seq,
                            int block_size, int num_blocks, int max_seqlen_k, int d, float scale,
                            float descale_k, float descale_v, int causal, int n_splits, void* ws,
                            size_t ws_bytes, void* stream) {
  if (!cu_seqlens_q) return fail(FA_ERR_INVALID_ARG, "null cu_seqlens_q");
  return attend_q4(q, k_codes, k_scales, v_codes, v_scales, o, lse, cu_seqlens_q, seqlens_k, block_table, n_seqs,
                   H, H_kv, total_q, max_seqlen_q, max_blocks_per_seq, block_size, num_blocks, max_seqlen_k, d,
                   scale, descale_k, descale_v, causal, n_splits, ws, ws_bytes, stream, "fa_fwd_paged_q4 launch");
}

fa_status_t fa_debug_counters(unsigned long long* device_counters) {
  fa::g_debug_counters = device_counters;
  return FA_OK;
}

fa_status_t fa_selftest_wait_timeout(unsigned int limit_us, void* stream) {
  if (limit_us == 0 || limit_us > 10u * 1000u * 1000u)
    return fail(FA_ERR_INVALID_ARG, "limit_us must be in [1, 10000000] (got %u)", limit_us);
  cudaError_t e = fa::launch_selftest_wait(static_cast<unsigned long long>(limit_us) * 1000ull,
                                           static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "fa_selftest_wait_timeout launch");
  return FA_OK;
}

fa_status_t fa_sync_status(void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned int code = 0, c = 0;
  int where = 0, w = 0;
  cudaError_t (*fetch[])(cudaStream_t, unsigned int*, int*) = {
      fa::status_fetch_fwd, fa::status_fetch_bwd, fa::status_fetch_decode,
      fa::status_fetch_selftest, fa::status_fetch_paged, fa::status_fetch_attend_q4,
      fa::status_fetch_attend_q4_tile};
  for (auto f : fetch) {
    cudaError_t e = f(s, &c, &w);
    if (e != cudaSuccess) return cuda_fail(e, "fa_sync_status");
    if (c) { code |= c; where = w; }
  }
  if (code & fa::FA_DEV_TIMEOUT)
    return fail(FA_ERR_DEVICE_TIMEOUT, "a kernel's bounded wait ran out (site %d)", where);
  if (code & fa::FA_DEV_BAD_CONFIG)
    return fail(FA_ERR_INVALID_ARG,
                "a kernel found invalid sequence boundaries (cu_seqlens / max_seqlen), lengths or cache "
                "blocks (site %d)",
                where);
  if (code) return fail(FA_ERR_CUDA, "device reported error code %u (site %d)", code, where);
  return FA_OK;
}

}  // extern "C"
