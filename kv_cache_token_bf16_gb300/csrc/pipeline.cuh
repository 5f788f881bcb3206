// Helpers shared by the TMA / tensor-core pipelines: bounded waits, packed fp32
// arithmetic and the host lookup of the tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "tcgen05.cuh"

namespace evict {

constexpr uint64_t kWaitLimitNs = 2000000000ull;   // bound of every pipeline wait (2 s, far above a tile's time)
constexpr uint32_t kWaitSleepNs = 20000;             // longest hardware sleep per poll
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Packed fp32 pairs: one instruction for two lanes of arithmetic, each lane rounded to nearest
// exactly as the scalar operation would be.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  return (uint64_t)__float_as_uint(lo) | ((uint64_t)__float_as_uint(hi) << 32);
}
__device__ __forceinline__ void split_f32x2(uint64_t x, float& lo, float& hi) {
  lo = __uint_as_float((uint32_t)x);
  hi = __uint_as_float((uint32_t)(x >> 32));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t sub_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// ex2 of both lanes (the special-function unit takes one value at a time)
__device__ __forceinline__ uint64_t ex2_f32x2(uint64_t x) {
  float lo, hi;
  split_f32x2(x, lo, hi);
  return pack_f32x2(ex2(lo), ex2(hi));
}

// Bounded wait on an mbarrier phase. The waiting thread sleeps in hardware
// between polls (no issue slots spent while it waits); it gives up early once
// the CTA's failure flag is set, and after kWaitLimitNs it sets the flag and
// the error word.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* fail, int* err) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = tc::global_ns();
  for (;;) {
    if (tc::mbar_try_wait_sleep(bar, parity, kWaitSleepNs)) return true;
    if (*fail) return false;
    if (tc::global_ns() - t0 > kWaitLimitNs) break;
  }
  *fail = 1;
  raise_device_error(err, kDevWaitTimeout);
  return false;
}
// The same wait ignoring the failure flag: used to let copies and MMAs already
// issued finish before the CTA releases its shared and tensor memory.
__device__ __forceinline__ void drain_phase(uint64_t* bar, uint32_t parity, int* err) {
  if (tc::mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = tc::global_ns();
  for (;;) {
    if (tc::mbar_try_wait_sleep(bar, parity, kWaitSleepNs)) return;
    if (tc::global_ns() - t0 > kWaitLimitNs) break;
  }
  raise_device_error(err, kDevWaitTimeout);
}

__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// cuTensorMapEncodeTiled from the driver, looked up once through the runtime.
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return (EncodeTiledFn) nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

}  // namespace evict
