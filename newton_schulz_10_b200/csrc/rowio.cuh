// Row accesses by a run-time element type (muon_dtype), shared by the stack
// update's kernels.
#pragma once

#include "common.cuh"

namespace muon {

__device__ __forceinline__ float4 unpack4(const __nv_bfloat16*, uint2 u) {
  const float2 a = Elem<__nv_bfloat16>::unpack2(u.x), b = Elem<__nv_bfloat16>::unpack2(u.y);
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float4 unpack4(const __half*, uint2 u) {
  const float2 a = Elem<__half>::unpack2(u.x), b = Elem<__half>::unpack2(u.y);
  return make_float4(a.x, a.y, b.x, b.y);
}
template <typename T>
__device__ __forceinline__ uint2 pack4(float4 v) {
  return make_uint2(Elem<T>::pack2(v.x, v.y), Elem<T>::pack2(v.z, v.w));
}

// Four or one elements of a row of the given type (muon_dtype).
__device__ __forceinline__ float4 load4(const void* row, int type, int64_t c) {
  if (type == MUON_F32) return *reinterpret_cast<const float4*>(static_cast<const float*>(row) + c);
  const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(row) + c);
  return type == MUON_BF16 ? unpack4((const __nv_bfloat16*)nullptr, u) : unpack4((const __half*)nullptr, u);
}
__device__ __forceinline__ float load1(const void* row, int type, int64_t c) {
  if (type == MUON_F32) return static_cast<const float*>(row)[c];
  return type == MUON_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(row)[c])
                           : __half2float(static_cast<const __half*>(row)[c]);
}
__device__ __forceinline__ void store4(void* row, int type, int64_t c, float4 v) {
  if (type == MUON_F32) *reinterpret_cast<float4*>(static_cast<float*>(row) + c) = v;
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(row) + c) = type == MUON_BF16 ? pack4<__nv_bfloat16>(v) : pack4<__half>(v);
}
__device__ __forceinline__ void store1(void* row, int type, int64_t c, float v) {
  if (type == MUON_F32) static_cast<float*>(row)[c] = v;
  else if (type == MUON_BF16) static_cast<__nv_bfloat16*>(row)[c] = __float2bfloat16_rn(v);
  else static_cast<__half*>(row)[c] = __float2half_rn(v);
}
__device__ __forceinline__ const void* row_at(const void* base, int type, int64_t off) {
  return static_cast<const char*>(base) + off * (type == MUON_F32 ? 4 : 2);
}
__device__ __forceinline__ void* row_at(void* base, int type, int64_t off) {
  return static_cast<char*>(base) + off * (type == MUON_F32 ? 4 : 2);
}

template <typename T> struct TypeOf;
template <> struct TypeOf<float> { static constexpr int value = MUON_F32; };
template <> struct TypeOf<__nv_bfloat16> { static constexpr int value = MUON_BF16; };
template <> struct TypeOf<__half> { static constexpr int value = MUON_F16; };

// The update's target from the updated momentum y and the gradient g.
__device__ __forceinline__ float target(float y, float g, float mu, int nesterov) { return nesterov ? fmaf(mu, y, g) : y; }

}  // namespace muon
