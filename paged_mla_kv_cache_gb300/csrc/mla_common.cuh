// Helpers shared by the latent-attention kernels (mla_*.cu): element types,
// launches, block scans, and the host checks of the C entry points.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cstdlib>
#include <mutex>

#include "pmg_mla.h"

namespace pmg_mla {

using bf16 = __nv_bfloat16;
using f16 = __half;
using e4m3 = __nv_fp8_e4m3;

// ---- element types --------------------------------------------------------

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(f16 x) { return __half2float(x); }
__device__ __forceinline__ float to_f(e4m3 x) { return static_cast<float>(x); }

template <class T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ bf16 from_f<bf16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ f16 from_f<f16>(float x) { return __float2half_rn(x); }
// round to nearest even, saturating at +-448; NaN stays NaN
template <>
__device__ __forceinline__ e4m3 from_f<e4m3>(float x) {
  e4m3 y;
  y.__x = __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
  return y;
}

// ---- flags, dependent launch ----------------------------------------------

__device__ __forceinline__ void set_flag(int32_t* err, int bits) {
  if (bits != 0 && err != nullptr) atomicOr(err, bits);
}

// Every kernel here is launched with programmatic dependent launch: the next
// kernel may begin its launch now, and nothing is read or written before the
// previous one has finished.
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_entry() {
  pdl_launch();
  pdl_wait();
}

// ---- block-wide sums ------------------------------------------------------

// Exclusive prefix sum over the threads of a block (blockDim a multiple of 32,
// at most 1024) and the total; `scratch` holds 33 values of T.
template <class T>
__device__ __forceinline__ T block_scan(T x, T* scratch, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  T inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    T w = lane < warps ? scratch[lane] : T(0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    scratch[lane] = w;
  }
  __syncthreads();
  const T before = warp > 0 ? scratch[warp - 1] : T(0);
  total = scratch[warps - 1];
  __syncthreads();
  return before + inc - x;
}

// ---- host side ------------------------------------------------------------

inline bool aligned(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

inline int elem_bytes(int dtype) {
  switch (dtype) {
    case PMG_BF16: case PMG_FP16: return 2;
    case PMG_FP32: return 4;
    case PMG_FP8_E4M3: return 1;
    default: return 0;
  }
}

// Strides whose byte offsets, times any index of 31 bits, could pass 63 bits are refused.
inline bool stride_ok(int64_t s) { return s >= 0 && s <= (int64_t{1} << 40); }

inline bool use_pdl() {
  static const bool on = [] {
    const char* e = std::getenv("PMG_PDL");
    return e == nullptr || e[0] != '0';
  }();
  return on;
}

inline int sm_count(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PMG_ERR_CUDA;
  if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return PMG_ERR_CUDA;
  return PMG_OK;
}

// Raises a kernel's dynamic shared memory limit, once a device and kernel.
inline int allow_smem(const void* kernel, int bytes) {
  static std::mutex mu;
  static struct { const void* kernel; int dev; } done[256];
  static int count = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PMG_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < count; ++i)
    if (done[i].kernel == kernel && done[i].dev == dev) return PMG_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return PMG_ERR_CUDA;
  if (count < 256) done[count++] = {kernel, dev};
  return PMG_OK;
}

template <class... Formal, class... Actual>
inline int launch(void (*kernel)(Formal...), dim3 grid, int threads, size_t smem, void* stream, Actual&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = use_pdl() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Formal>(args)...) == cudaSuccess ? PMG_OK : PMG_ERR_CUDA;
}

}  // namespace pmg_mla
