// ssm_vec.cuh -- groups of eight consecutive elements moved with 16-byte accesses.
#pragma once

#include "ssm_common.cuh"

namespace ssm {

// Eight elements as loaded: 16 bytes of bf16 or 32 bytes of fp32.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
  uint4 a;
};
template <> struct Raw8<float> {
  float4 a, b;
};

// p: 16-byte aligned. Streamed data that is read once: no L1 allocation.
__device__ __forceinline__ void ld8(const __nv_bfloat16 *p, Raw8<__nv_bfloat16> &r) {
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.a.x), "=r"(r.a.y), "=r"(r.a.z), "=r"(r.a.w) : "l"(p));
}
// fp32: the two halves of a lane's 32 bytes come from the same lines, so these do go through L1.
__device__ __forceinline__ void ld8(const float *p, Raw8<float> &r) {
  r.a = reinterpret_cast<const float4 *>(p)[0];
  r.b = reinterpret_cast<const float4 *>(p)[1];
}
__device__ __forceinline__ void zero8(Raw8<__nv_bfloat16> &r) { r.a = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void zero8(Raw8<float> &r) { r.a = r.b = make_float4(0, 0, 0, 0); }

__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16> &r, float *v) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {  // a bf16 is the top half of a float
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack8(const Raw8<float> &r, float *v) {
  v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
  v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
}
// One element into slot e of a raw group.
__device__ __forceinline__ void put8(Raw8<__nv_bfloat16> &r, int e, __nv_bfloat16 v) {
  uint32_t *w = reinterpret_cast<uint32_t *>(&r.a);
  const uint32_t b = (uint32_t)__bfloat16_as_ushort(v);
  w[e >> 1] |= (e & 1) ? b << 16 : b;
}
__device__ __forceinline__ void put8(Raw8<float> &r, int e, float v) {
  if (e < 4) reinterpret_cast<float *>(&r.a)[e] = v;
  else reinterpret_cast<float *>(&r.b)[e - 4] = v;
}

__device__ __forceinline__ void st8(__nv_bfloat16 *p, const float *v) {
  uint4 r;
  uint32_t *w = reinterpret_cast<uint32_t *>(&r);
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  *reinterpret_cast<uint4 *>(p) = r;
}
__device__ __forceinline__ void st8(float *p, const float *v) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

}  // namespace ssm
