// Loads in stream order, and eight consecutive values of a row (fp32 or bf16, 16-byte aligned).
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace dfssm {

// What an earlier kernel of the stream may have written is read after pdl_wait(), with these or with plain loads.  Not
// with a read-only load (__ldg, or one through a __restrict__ parameter): the compiler may move that above the
// wait, as nothing in the kernel itself writes the memory.  The wait clobbers memory, which plain loads do not cross;
// volatile assembly keeps its place as well, and its batches stay together.
__device__ __forceinline__ uint32_t ld_u32(const void* p) {
  uint32_t r;
  asm volatile("ld.global.u32 %0, [%1];" : "=r"(r) : "l"(p));
  return r;
}
__device__ __forceinline__ int ld_s32(const int32_t* p) { return (int)ld_u32(p); }
__device__ __forceinline__ float ld_f32(const float* p) { return __uint_as_float(ld_u32(p)); }
__device__ __forceinline__ uint4 ld_u32x4(const void* p) {
  uint4 r;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}
__device__ __forceinline__ float4 ld_f32x4(const void* p) {
  const uint4 r = ld_u32x4(p);
  return make_float4(__uint_as_float(r.x), __uint_as_float(r.y), __uint_as_float(r.z), __uint_as_float(r.w));
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  const uint4 a = ld_u32x4(p), b = ld_u32x4(p + 4);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = ld_u32x4(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&v)[8]) {
  st_f4(p, make_float4(v[0], v[1], v[2], v[3]));
  st_f4(p + 4, make_float4(v[4], v[5], v[6], v[7]));
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight codes as bytes.
__device__ __forceinline__ uint2 pack_codes(const int (&cd)[8]) {
  uint32_t lo = 0u, hi = 0u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    lo |= ((uint32_t)cd[k] & 0xFFu) << (8 * k);
    hi |= ((uint32_t)cd[k + 4] & 0xFFu) << (8 * k);
  }
  return make_uint2(lo, hi);
}

}  // namespace dfssm
