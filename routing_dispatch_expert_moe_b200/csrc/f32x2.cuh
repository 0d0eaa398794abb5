// Packed pairs of fp32 (sm_100 executes add, mul and fma on two neighbouring registers with one
// instruction): the row kernels that are bound by instruction issue work on pairs.  Each half
// rounds as the scalar operation does.
#pragma once

#include "common.cuh"

namespace moe {

using f32x2 = unsigned long long;

__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ f32x2 both(float a) { return pack2(a, a); }
__device__ __forceinline__ float2 unpack2(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float sum2(f32x2 v) {
  const float2 f = unpack2(v);
  return f.x + f.y;
}

// Eight neighbouring elements as four pairs: from the storage type, and back.
struct Oct {
  f32x2 p[4];
};
__device__ __forceinline__ Oct oct_const(float v) {
  Oct o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.p[i] = both(v);
  return o;
}
__device__ __forceinline__ Oct oct_bf16(const uint4& a) {
  Oct o;
  o.p[0] = pack2(bf16_lo(a.x), bf16_hi(a.x));
  o.p[1] = pack2(bf16_lo(a.y), bf16_hi(a.y));
  o.p[2] = pack2(bf16_lo(a.z), bf16_hi(a.z));
  o.p[3] = pack2(bf16_lo(a.w), bf16_hi(a.w));
  return o;
}
__device__ __forceinline__ Oct oct_f32(const uint4& a, const uint4& b) {
  Oct o;
  o.p[0] = pack2(__uint_as_float(a.x), __uint_as_float(a.y));
  o.p[1] = pack2(__uint_as_float(a.z), __uint_as_float(a.w));
  o.p[2] = pack2(__uint_as_float(b.x), __uint_as_float(b.y));
  o.p[3] = pack2(__uint_as_float(b.z), __uint_as_float(b.w));
  return o;
}
template <typename T>
__device__ __forceinline__ void store_oct(void* base, long long e, const Oct& o);
template <>
__device__ __forceinline__ void store_oct<__nv_bfloat16>(void* base, long long e, const Oct& o) {
  const float2 a = unpack2(o.p[0]), b = unpack2(o.p[1]), c = unpack2(o.p[2]), d = unpack2(o.p[3]);
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + e) =
      make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(b.x, b.y), pack_bf16x2(c.x, c.y), pack_bf16x2(d.x, d.y));
}
template <>
__device__ __forceinline__ void store_oct<float>(void* base, long long e, const Oct& o) {
  const float2 a = unpack2(o.p[0]), b = unpack2(o.p[1]), c = unpack2(o.p[2]), d = unpack2(o.p[3]);
  float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + e);
  p[0] = make_float4(a.x, a.y, b.x, b.y);
  p[1] = make_float4(c.x, c.y, d.x, d.y);
}

// log(1 + e) / e on [0, 1]: a degree-7 polynomial fitted here for the least largest relative error
// (2.4e-7).  Times e it keeps the relative precision of a small e.
__device__ __forceinline__ f32x2 log1p_over(f32x2 e) {
  f32x2 s = fma2(both(-0.00853919890f), e, both(0.0440895967f));
  s = fma2(s, e, both(-0.107681662f));
  s = fma2(s, e, both(0.177452385f));
  s = fma2(s, e, both(-0.244954616f));
  s = fma2(s, e, both(0.332754791f));
  s = fma2(s, e, both(-0.499974042f));
  return fma2(s, e, both(0.999999821f));
}
__device__ __forceinline__ f32x2 log1p_unit(f32x2 e) { return mul2(log1p_over(e), e); }

}  // namespace moe
