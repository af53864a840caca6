// Device helpers of the paged 8-bit cache: e4m3 conversions, page lookups.
#pragma once

#include "device_common.cuh"

namespace lowram {

// Two e4m3 codes (byte 0 first) to fp16, exactly (every e4m3 value is an fp16 value).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
// Four e4m3 codes (byte 0 first) to floats.
__device__ __forceinline__ void e4m3x4_to_float(uint32_t w, float* o) {
  const uint32_t a = e4m3x2_to_f16x2((uint16_t)(w & 0xffffu));
  const uint32_t b = e4m3x2_to_f16x2((uint16_t)(w >> 16));
  const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&b));
  o[0] = fa.x; o[1] = fa.y; o[2] = fb.x; o[3] = fb.y;
}
// Two floats to e4m3 (round to nearest even; |x| <= 448 or NaN): lo in byte 0.
__device__ __forceinline__ uint32_t float2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t float4_to_e4m3x4(const float* x) {
  return float2_to_e4m3x2(x[0], x[1]) | (float2_to_e4m3x2(x[2], x[3]) << 16);
}

// The paged kernels are launched as programmatic dependents of whatever precedes them in the
// stream: a kernel's blocks may be set up while the one before still runs, and touch memory only
// behind grid_dependency_wait(), which returns when the kernels before have ended and their writes
// are visible. A kernel lets the next be set up only behind its own wait, in every path, so whatever
// the next one does early (the merge reads the lengths) sees everything older than its predecessor.
// (Back to back calls of an append and an attend: about 2 us less than plain launches.)
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem,
                             cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t lc{};
  lc.gridDim = grid;
  lc.blockDim = dim3(threads);
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &at;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, P(args)...);
}

// Length of sequence b, cut to what its page list can hold (reported when it was not in range).
__device__ __forceinline__ int paged_len(const lowram_pages& pg, int b, int* status) {
  const int n = pg.lens[b], top = pg.max_pages * pg.page_tokens;
  if (n >= 0 && n <= top) return n;
  raise_status(status, kStatusDeviceCheck);
  return n < 0 ? 0 : top;
}

// Page index of entry i of sequence b's list, or -1 (reported) if it is out of range.
__device__ __forceinline__ int paged_page(const lowram_pages& pg, int b, int i, int* status) {
  const int p = pg.table[(size_t)b * pg.max_pages + i];
  if (p >= 0 && p < pg.n_pages) return p;
  raise_status(status, kStatusDeviceCheck);
  return -1;
}

}  // namespace lowram
