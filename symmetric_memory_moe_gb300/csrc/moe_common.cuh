// moe_common.cuh -- what the MoE block operators share: element types,
// reductions, and argument checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <string>

#include "symm_internal.h"

namespace moe {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the block's warps, the same in every thread; `red` holds one float
// per warp.  Ends with a barrier, so `red` may be used again at once.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  const int warps = (int)(blockDim.x >> 5);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < warps; ++w) s += red[w];
  __syncthreads();
  return s;
}

// The same with one barrier: `red` may be written again only after another
// barrier of the block.
__device__ __forceinline__ float block_sum_once(float v, float* red) {
  v = warp_sum(v);
  const int lane = threadIdx.x & 31, warps = (int)(blockDim.x >> 5);
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < warps ? red[lane] : 0.f);
}

// Programmatic dependent launch: a kernel launched by launch() may start while
// the one before it on the stream ends; wait_for_earlier() holds it (before its
// first access to memory) until that one's writes are visible.
// let_next_start() is for a kernel whose own second launch follows.
__device__ __forceinline__ void wait_for_earlier() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... P, typename... A>
int launch(const char* what, void (*kernel)(P...), unsigned grid, unsigned block, size_t smem,
           cudaStream_t s, A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return symm_host::cuda_check(cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...), what);
}

inline size_t dtype_bytes(int dtype) { return dtype == SYMM_DTYPE_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) {
  return dtype == SYMM_DTYPE_F16 || dtype == SYMM_DTYPE_BF16 || dtype == SYMM_DTYPE_F32;
}
inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Runs the body of a C entry point: no C++ exception leaves it.
template <typename F>
int entry(const char* what, F&& body) {
  try {
    return body();
  } catch (...) {
    try {
      return symm_host::fail(SYMM_ECUDA, std::string(what) + ": out of host memory");
    } catch (...) {
      return SYMM_ECUDA;
    }
  }
}

}  // namespace moe
