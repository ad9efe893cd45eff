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

// 2^v and 1/v by the special-function unit, to about 2^-22 of the value; results below the normal
// numbers are 0, which spares the instructions that would keep them.
__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// v / (1 + exp(-v)).  Where exp(-v) is infinite (v below -88) the quotient is -0, the limit.
__device__ __forceinline__ float silu(float v) { return v * rcp_fast(1.f + exp2_fast(-kLog2e * v)); }

// log(1 + exp(v)) = max(v, 0) + log(1 + e), e = exp(-|v|), and with s = e / (2 + e) <= 1/3
// log(1 + e) = 2 atanh(s) = 2 (s + s^3 (1/3 + s^2/5 + s^4/7 + ...)): no digits are lost for small
// e, as they are in log(1 + e) itself.  The bracket as a polynomial in s^2 <= 1/9, through its
// values at five Chebyshev points: 1e-9 of log(1 + e) at most.  (The series' first five terms are
// 1.1e-7 low for all v near 0, twice what rounding does to any one, and steps add up over a prompt.)
constexpr float kAtanh0 = 0x1.555556p-2f, kAtanh1 = 0x1.9998d4p-3f, kAtanh2 = 0x1.24c926p-3f, kAtanh3 = 0x1.bc8cf8p-4f,
                kAtanh4 = 0x1.dba26p-4f;
__device__ __forceinline__ float softplus(float v) {
  const float e = expf(-fabsf(v));
  const float s = e * rcp_fast(2.f + e);
  const float q = s * s;
  float r = fmaf(q, kAtanh4, kAtanh3);
  r = fmaf(q, r, kAtanh2);
  r = fmaf(q, r, kAtanh1);
  r = fmaf(q, r, kAtanh0);
  r = fmaf(q * s, r, s);
  return fmaf(2.f, r, fmaxf(v, 0.f));
}

// Two 32-bit numbers in one 64-bit register, for the packed multiply-adds.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Loads past the L1, or of what is read once, that stay behind the waits in front of them (griddepcontrol.wait, the
// acquire of a flag): volatile, with a clobber, where a plain hint is an expression that the compiler may move.
__device__ __forceinline__ float4 load_once(const float* p) {
  float4 v;
  asm volatile("ld.global.cs.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(__cvta_generic_to_global(p))
               : "memory");
  return v;
}
__device__ __forceinline__ uint64_t load_l2(const uint64_t* p) {
  uint64_t v;
  asm volatile("ld.global.cg.b64 %0, [%1];" : "=l"(v) : "l"(__cvta_generic_to_global(p)) : "memory");
  return v;
}

// ------------------------------------------------------------------ order of launches
// These kernels are launched as programmatic dependents of the work before them in the stream and begin
// with this: a wait until that work has completed and its results are visible (nothing is read or
// written before), and the signal that lets the next such kernel be set up meanwhile.  A decoding loop's
// launches are a few us long, and this takes the set-up of each out of the chain.  What differs:
//  - whole-sequence scans of more than one block a multiprocessor start when the work before has ended
//    (launch_lanes), and clear_kernel, in front of scan_slots_kernel, never signals, for the same reason;
//  - scan_kernel's states' launch signals at its end, w4_kernel before its wait.  A signal only allows the
//    next kernel to be set up; that kernel's own wait is for this one's completion all the same;
//  - w4_kernel behind columns_kernel reads its codes before it waits: columns_kernel signals after its own
//    wait, so by then nobody writes them;
//  - delta_prepare_kernel, behind a pair of launches of the same call that uses the other buffer, reads nothing that the
//    call's kernels write and writes a buffer whose last reader ended earlier: it begins beside the walk in front, and only its last block
//    waits, at its end, so that the walk behind it does not begin before that walk has ended.
// What the kernel in front may write is read by ordinary or volatile loads, never through the read-only
// path, which wants data that stay unchanged for as long as the kernel is resident.
__device__ __forceinline__ void begin_kernel() {
  grid_dep_wait();
  grid_dep_launch();
}

// ------------------------------------------------------------------ host side
inline bool aligned_to(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
inline size_t elem_size(int dtype) { return dtype == SSD_BF16 ? 2 : 4; }
inline bool known_dtype(int dtype) { return dtype == SSD_F32 || dtype == SSD_BF16; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline ssd_status launched(cudaError_t e) { return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA; }

// Multiprocessors of the current device; 152 (a GB300's) where it cannot be asked.
int layer_sm_count();

}  // namespace ssd
