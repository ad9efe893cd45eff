// Pieces shared by the kernels of the layer around the SSD forward pass
// (convolution, selective scan, single-token step, 4-bit products, beam
// search): typed loads and stores, the activations, and host-side checks.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"
#include "ssd_internal.cuh"

namespace ssd {

// ------------------------------------------------------------------ values
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// v / (1 + exp(-v)).  Below about -88 exp(-v) is infinite and the quotient -0, the limit.
__device__ __forceinline__ float silu(float v) { return __fdividef(v, 1.f + __expf(-v)); }

// log(1 + exp(v)); above 20 it equals v in 32 bits.
__device__ __forceinline__ float softplus(float v) { return v > 20.f ? v : log1pf(__expf(v)); }

// ------------------------------------------------------------------ host side
inline bool aligned_to(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
inline size_t elem_size(int dtype) { return dtype == SSD_BF16 ? 2 : 4; }
inline bool known_dtype(int dtype) { return dtype == SSD_F32 || dtype == SSD_BF16; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline ssd_status launched(cudaError_t e) { return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA; }

// Multiprocessors of the current device; 152 (a GB300's) where it cannot be asked.
int layer_sm_count();

}  // namespace ssd
