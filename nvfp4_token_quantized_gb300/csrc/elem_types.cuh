// elem_types.cuh - the three element types of the operators around the layer
// as FP32 values, one at a time or eight at a time.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace moe {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Two packed 16-bit values.
__device__ __forceinline__ float2 unpack2(uint32_t w, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight values as four pairs for the two-lane FP32 instructions.
struct Pairs {
  float2 p[4];
};

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)),
        "l"(*reinterpret_cast<uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Eight values held raw, 16 bytes for the 16-bit types and 32 for FP32.
template <typename T>
struct Raw8 {
  uint4 q[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Pairs unpack(const Raw8<T>& r) {
  Pairs o;
  const uint32_t w[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) o.p[i] = unpack2(w[i], T());
  return o;
}
template <>
__device__ __forceinline__ Pairs unpack<float>(const Raw8<float>& r) {
  Pairs o;
  o.p[0] = make_float2(__uint_as_float(r.q[0].x), __uint_as_float(r.q[0].y));
  o.p[1] = make_float2(__uint_as_float(r.q[0].z), __uint_as_float(r.q[0].w));
  o.p[2] = make_float2(__uint_as_float(r.q[1].x), __uint_as_float(r.q[1].y));
  o.p[3] = make_float2(__uint_as_float(r.q[1].z), __uint_as_float(r.q[1].w));
  return o;
}
// 16-byte aligned accesses (plain ones: an operand may be overwritten in place
// by the same thread later).
template <typename T>
__device__ __forceinline__ Raw8<T> load_raw(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int u = 0; u < (int)sizeof(T) / 2; ++u) r.q[u] = reinterpret_cast<const uint4*>(p)[u];
  return r;
}
template <typename T>
__device__ __forceinline__ void store_pairs(T* p, const Pairs& v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2(v.p[0].x, v.p[0].y, T()), pack2(v.p[1].x, v.p[1].y, T()),
                                            pack2(v.p[2].x, v.p[2].y, T()), pack2(v.p[3].x, v.p[3].y, T()));
}
template <>
__device__ __forceinline__ void store_pairs<float>(float* p, const Pairs& v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v.p[0].x, v.p[0].y, v.p[1].x, v.p[1].y);
  reinterpret_cast<float4*>(p)[1] = make_float4(v.p[2].x, v.p[2].y, v.p[3].x, v.p[3].y);
}

}  // namespace moe
