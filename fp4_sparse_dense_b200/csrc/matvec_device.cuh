// Device code shared by the few-row products: asynchronous copies, the widening of FP4 codes to
// 16-bit operands, and the typed store of an output.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "experts_internal.h"
#include "sm100_ptx.cuh"

namespace sharq {

constexpr int kStepK = 128;  // K of a step

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Eight codes of a word -> four f16x2, codes (2 j, 2 j + 1) in word j.
__device__ __forceinline__ void widen(uint32_t w, uint32_t* h) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Two E4M3 bytes -> f16x2.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(uint16_t(two)));
  return d;
}

// The same codes as bf16 values times 2^-126 (the code's exponent and mantissa bits in
// bf16's, E2M1's subnormal 0.5 as bf16's): codes (i, i + 4) in word i. A masked nibble times
// (2^6 + 2^12) has its value bits at 8..6 and its sign at 15.
__device__ __forceinline__ void widen_bf16(uint32_t w, uint32_t* h) {
  const uint32_t v = w >> 8;
  h[0] = ((w & 0x000F000Fu) * 0x1040u) & 0x81C081C0u;
  h[1] = ((w & 0x00F000F0u) * 0x0104u) & 0x81C081C0u;
  h[2] = ((v & 0x000F000Fu) * 0x1040u) & 0x81C081C0u;
  h[3] = ((v & 0x00F000F0u) * 0x0104u) & 0x81C081C0u;
}

template <int Y>
struct YType;
template <>
struct YType<SHARQ_F32> {
  typedef float T;
  static __device__ __forceinline__ T of(float v) { return v; }
};
template <>
struct YType<SHARQ_BF16> {
  typedef __nv_bfloat16 T;
  static __device__ __forceinline__ T of(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct YType<SHARQ_F16> {
  typedef __half T;
  static __device__ __forceinline__ T of(float v) { return __float2half_rn(v); }
};

__device__ __forceinline__ void store_y(const MatvecParams& p, size_t at, float v) {
  if (p.y_dtype == SHARQ_F32)
    static_cast<float*>(p.Y)[at] = v;
  else if (p.y_dtype == SHARQ_BF16)
    static_cast<__nv_bfloat16*>(p.Y)[at] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(p.Y)[at] = __float2half_rn(v);
}

template <int VIEW>
constexpr int kScaleStep = VIEW == kE4M3x16 ? 1024 : 512;  // scale bytes of 128 outputs x 128 K

}  // namespace sharq
