// Pieces shared by the kernels over a batch of chunks (append, read back, chunk
// attention): the device status, conversions, and the split of attention work
// over CTAs (mk_walk.cuh).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math_constants.h>

#include "mk_internal.h"
#include "mk_walk.cuh"

namespace mkc {

// first device error of the state; later calls exit at once until mk_reset
__device__ __forceinline__ void raise(Ctrl *c, int code, int where) {
    if (atomicCAS(&c->status, 0, code) == 0) atomicExch(&c->where, where);
    atomicExch(&c->abort, 1);
}
__device__ __forceinline__ bool aborted(const Ctrl *c) { return *(volatile const int *)&c->abort != 0; }

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__nv_fp8_e4m3 v) { return __half2float(__half(__nv_cvt_fp8_to_halfraw(v.__x, __NV_E4M3))); }

// N consecutive elements (16-byte aligned, or N*sizeof(T) aligned where that is less)
template <class T, int N>
struct alignas((sizeof(T) * N) < 16 ? (sizeof(T) * N) : 16) Vec {
    T v[N];
};

}  // namespace mkc
