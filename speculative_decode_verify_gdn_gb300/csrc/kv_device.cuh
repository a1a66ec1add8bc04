// Device and launch helpers that the kernels of the attention layers share.
#pragma once

#include <cuda_fp16.h>

#include "gdn_common.cuh"
#include "kv_kernels.h"

namespace gdn {

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return F16 ? __half22float2(*reinterpret_cast<const __half2*>(&w)) : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}

// Two f32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// A slot's length, 0 (and a status bit) when it is negative or beyond the table's columns.
__device__ __forceinline__ int checked_slot_len(int len, const gdn_kv_dims& d, uint32_t* err) {
  if (len < 0 || (long long)len > (long long)d.max_pages * d.page_size) {
    atomicOr(err, GDN_DEVERR_KV_LEN);
    return 0;
  }
  return len;
}

// The slot of a sequence's prefix, -1 without one (or, with a status bit, out of range).
__device__ __forceinline__ int checked_prefix(const int32_t* prefix_of, int b, const gdn_kv_dims& d, uint32_t* err) {
  if (!prefix_of) return -1;
  const int s = prefix_of[b];
  if (s < -1 || s >= d.n_slots) atomicOr(err, GDN_DEVERR_KV_SLOT);
  return s < 0 || s >= d.n_slots ? -1 : s;
}

// The last sequence b < B with cu[b] <= token, by a converged warp: 32 bounds at a time, a trip to L2
// for each factor of 32 in B.  (Whatever cu holds, the answer is in 0..B-1.)
__device__ __forceinline__ int find_sequence(const int32_t* cu, int B, int token, int lane) {
  int lo = 0, n = B;
  while (n > 1) {
    const int step = (n + 31) / 32, i = lane * step;
    const uint32_t at_or_before = __ballot_sync(0xffffffffu, i < n && cu[lo + i] <= token);
    const int j = at_or_before ? 31 - __clz(int(at_or_before)) : 0;
    lo += j * step;
    n = n - j * step < step ? n - j * step : step;
  }
  return lo;
}

template <typename... Args>
cudaError_t launch_dependent(void (*kernel)(Args...), unsigned grid, int threads, int smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(unsigned(threads), 1, 1);
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace gdn
