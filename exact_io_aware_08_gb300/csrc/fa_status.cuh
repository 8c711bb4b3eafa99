// Device-side error reporting.  Kernels never trap: a wait that runs out of time, or a launch
// that finds an impossible configuration, records a code here and returns.  The host reads
// and clears the word in fa_sync_status().
//
// The library is built without relocatable device code, so every translation unit that
// launches kernels owns its own status word; FA_DEFINE_STATUS_FETCH gives each one host
// accessors: where the word is, so that fa_sync_status() looks at all of them in one go, and
// what it holds, for the units in turn once one of them has something to say.
#pragma once

#include <cuda_runtime.h>

#include "fa_kernels.h"

namespace fa {

static __device__ unsigned int g_dev_status = 0;
static __device__ int g_dev_where = 0;

__device__ __forceinline__ void report_device_error(unsigned int code, int where) {
  atomicOr(&g_dev_status, code);
  atomicExch(&g_dev_where, where);
}

}  // namespace fa

// Host accessor: copy this TU's status word out (after synchronising ``stream``) and clear it.  Each copy is
// a round trip to the device (some 9 us), so that a clean word, the usual one, is all that is read.
// NAME_word: the word's address.
#define FA_DEFINE_STATUS_FETCH(NAME)                                                         \
  namespace fa {                                                                             \
  cudaError_t NAME(cudaStream_t stream, unsigned int* code, int* where) {                    \
    cudaError_t e = cudaStreamSynchronize(stream);                                           \
    if (e != cudaSuccess) return e;                                                          \
    e = cudaMemcpyFromSymbol(code, g_dev_status, sizeof(unsigned int));                      \
    if (e != cudaSuccess || !*code) return e;                                                \
    e = cudaMemcpyFromSymbol(where, g_dev_where, sizeof(int));                               \
    if (e != cudaSuccess) return e;                                                          \
    const unsigned int zero = 0;                                                             \
    return cudaMemcpyToSymbol(g_dev_status, &zero, sizeof(unsigned int));                    \
  }                                                                                          \
  cudaError_t NAME##_word(const unsigned int** at) {                                         \
    void* p = nullptr;                                                                       \
    const cudaError_t e = cudaGetSymbolAddress(&p, g_dev_status);                            \
    *at = static_cast<const unsigned int*>(p);                                               \
    return e;                                                                                \
  }                                                                                          \
  }
