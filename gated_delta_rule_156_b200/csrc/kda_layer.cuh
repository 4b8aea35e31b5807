// Shared by the layer operators (short convolution, selective scan, block
// norm): launch arguments, vector loads, activations, sequence lookup.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_common.cuh"
#include "kda_layer_internal.h"

namespace kda {

// VEC consecutive elements as fp32, in one access of VEC * sizeof(IO) bytes
// (the address must be aligned to that).
template <typename IO, int VEC>
struct Raw;  // storage of VEC elements
template <>
struct Raw<__nv_bfloat16, 1> { uint16_t r; };
template <>
struct Raw<__nv_bfloat16, 2> { uint32_t r; };
template <>
struct Raw<__nv_bfloat16, 4> { uint2 r; };
template <>
struct Raw<__nv_bfloat16, 8> { uint4 r; };
template <>
struct Raw<float, 1> { float r; };
template <>
struct Raw<float, 2> { float2 r; };
template <>
struct Raw<float, 4> { float4 r; };
template <>
struct Raw<float, 8> { float4 r[2]; };

template <typename IO, int VEC>
__device__ __forceinline__ Raw<IO, VEC> load_raw(const IO* p) {
  return *reinterpret_cast<const Raw<IO, VEC>*>(p);
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, 1>& a, float (&v)[1]) {
  v[0] = __uint_as_float((uint32_t)a.r << 16);
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, 2>& a, float (&v)[2]) {
  v[0] = bf_lo(a.r); v[1] = bf_hi(a.r);
}
__device__ __forceinline__ void unpack(const Raw<float, 2>& a, float (&v)[2]) {
  v[0] = a.r.x; v[1] = a.r.y;
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, 4>& a, float (&v)[4]) {
  v[0] = bf_lo(a.r.x); v[1] = bf_hi(a.r.x); v[2] = bf_lo(a.r.y); v[3] = bf_hi(a.r.y);
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, 8>& a, float (&v)[8]) {
  v[0] = bf_lo(a.r.x); v[1] = bf_hi(a.r.x); v[2] = bf_lo(a.r.y); v[3] = bf_hi(a.r.y);
  v[4] = bf_lo(a.r.z); v[5] = bf_hi(a.r.z); v[6] = bf_lo(a.r.w); v[7] = bf_hi(a.r.w);
}
__device__ __forceinline__ void unpack(const Raw<float, 1>& a, float (&v)[1]) { v[0] = a.r; }
__device__ __forceinline__ void unpack(const Raw<float, 4>& a, float (&v)[4]) {
  v[0] = a.r.x; v[1] = a.r.y; v[2] = a.r.z; v[3] = a.r.w;
}
__device__ __forceinline__ void unpack(const Raw<float, 8>& a, float (&v)[8]) {
  v[0] = a.r[0].x; v[1] = a.r[0].y; v[2] = a.r[0].z; v[3] = a.r[0].w;
  v[4] = a.r[1].x; v[5] = a.r[1].y; v[6] = a.r[1].z; v[7] = a.r[1].w;
}

__device__ __forceinline__ uint32_t bf_pair(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ void pack(const float (&v)[1], Raw<__nv_bfloat16, 1>& a) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v[0]);
  a.r = *reinterpret_cast<const uint16_t*>(&b);
}
__device__ __forceinline__ void pack(const float (&v)[2], Raw<__nv_bfloat16, 2>& a) {
  a.r = bf_pair(v[0], v[1]);
}
__device__ __forceinline__ void pack(const float (&v)[2], Raw<float, 2>& a) {
  a.r = make_float2(v[0], v[1]);
}
__device__ __forceinline__ void pack(const float (&v)[4], Raw<__nv_bfloat16, 4>& a) {
  a.r = make_uint2(bf_pair(v[0], v[1]), bf_pair(v[2], v[3]));
}
__device__ __forceinline__ void pack(const float (&v)[8], Raw<__nv_bfloat16, 8>& a) {
  a.r = make_uint4(bf_pair(v[0], v[1]), bf_pair(v[2], v[3]), bf_pair(v[4], v[5]),
                   bf_pair(v[6], v[7]));
}
__device__ __forceinline__ void pack(const float (&v)[1], Raw<float, 1>& a) { a.r = v[0]; }
__device__ __forceinline__ void pack(const float (&v)[4], Raw<float, 4>& a) {
  a.r = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void pack(const float (&v)[8], Raw<float, 8>& a) {
  a.r[0] = make_float4(v[0], v[1], v[2], v[3]);
  a.r[1] = make_float4(v[4], v[5], v[6], v[7]);
}

template <typename IO, int VEC>
__device__ __forceinline__ void load_vec(const IO* p, float (&v)[VEC]) {
  unpack(load_raw<IO, VEC>(p), v);
}
template <typename IO, int VEC>
__device__ __forceinline__ void store_vec(IO* p, const float (&v)[VEC]) {
  Raw<IO, VEC> a;
  pack(v, a);
  *reinterpret_cast<Raw<IO, VEC>*>(p) = a;
}

// 2^x and 1 / x, to 2 and 1 units of 2^-23; results below 2^-126 are 0.
__device__ __forceinline__ float ex2_f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_f(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eLow = 1.4426950408889634 - (double)kLog2e;
constexpr float kLn2 = 0.6931471805599453f;
__device__ __forceinline__ float sigmoid_f(float x) {
  return rcp_f(1.f + ex2_f(-kLog2e * x));
}
// d silu(x) / dx from x and s = sigmoid(x)
__device__ __forceinline__ float silu_grad(float x, float s) {
  return s * fmaf(x, 1.f - s, 1.f);
}
// softplus(x) = max(x, 0) + log(1 + e), e = exp(-|x|).  With s = e / (2 + e),
// log(1 + e) = 2 atanh(s) = 2 s (1 + s^2/3 + s^4/5 + ...): s <= 1/3, so seven
// terms leave 2e-8 of the value, for the smallest steps too (a logarithm of
// 1 + e would lose them).  There e is all of the value, and rounding its base-2
// argument p costs e up to 2^-25 |p|.  For an fp32 x what p lacks is put into
// e; a bf16 x is itself rounded by 2^-9 of its value, which costs e 2^15 times
// as much, and keeps the shorter form (a prompt of 2 x 8192 x 4096 in bf16 500
// us, 517 with the longer one; 2 x 4096 x 2048 in fp32 207 and 214 us).
template <typename IO>
__device__ __forceinline__ float softplus_f(float x) {
  float e, top = fmaxf(x, 0.f);
  if constexpr (sizeof(IO) == 4) {
    // beyond 126 e is 0, and an infinity would make the remainder NaN
    const float t = fabsf(x) < 126.f ? -fabsf(x) : -126.f, p = kLog2e * t;
    const float r = fmaf(t, kLog2eLow, fmaf(t, kLog2e, -p));
    e = ex2_f(p);
    e = fmaf(e * kLn2, r, e);
    top = x < 0.f ? 0.f : x;  // NaN stays NaN (otherwise e brings it)
  } else {
    e = ex2_f(-kLog2e * fabsf(x));
  }
  const float s = e * rcp_f(2.f + e), q = s * s;
  float p = 1.f / 13.f;
  p = fmaf(p, q, 1.f / 11.f);
  p = fmaf(p, q, 1.f / 9.f);
  p = fmaf(p, q, 1.f / 7.f);
  p = fmaf(p, q, 1.f / 5.f);
  p = fmaf(p, q, 1.f / 3.f);
  p = fmaf(p, q, 1.f);
  return fmaf(2.f * s, p, top);
}

// Two fp32 values in one 64-bit register pair, and the packed arithmetic on
// them (one instruction for two results, same rounding as two).
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 both(float x) { return pack2(x, x); }
__device__ __forceinline__ float sum2(f32x2 v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return lo + hi;
}
__device__ __forceinline__ f32x2 sigmoid2(f32x2 x) {
  float a, b;
  unpack2(mul2(x, both(-kLog2e)), a, b);
  unpack2(add2(pack2(ex2_f(a), ex2_f(b)), both(1.f)), a, b);
  return pack2(rcp_f(a), rcp_f(b));
}

// VEC elements as pairs; a single one is a pair with 0.
template <int VEC>
constexpr int kPairs = (VEC + 1) / 2;
template <typename IO, int VEC>
__device__ __forceinline__ void unpack_pairs(const Raw<IO, VEC>& a, f32x2 (&p)[kPairs<VEC>]) {
  float v[VEC];
  unpack(a, v);
#pragma unroll
  for (int i = 0; i < kPairs<VEC>; ++i) p[i] = pack2(v[2 * i], 2 * i + 1 < VEC ? v[(2 * i + 1) % VEC] : 0.f);
}
template <typename IO, int VEC>
__device__ __forceinline__ void load_pairs(const IO* q, f32x2 (&p)[kPairs<VEC>]) {
  unpack_pairs<IO, VEC>(load_raw<IO, VEC>(q), p);
}
template <typename IO, int VEC>
__device__ __forceinline__ void store_pairs(IO* q, const f32x2 (&p)[kPairs<VEC>]) {
  float v[VEC];
#pragma unroll
  for (int i = 0; i < kPairs<VEC>; ++i) {
    float lo, hi;
    unpack2(p[i], lo, hi);
    v[2 * i] = lo;
    if (2 * i + 1 < VEC) v[(2 * i + 1) % VEC] = hi;
  }
  store_vec<IO, VEC>(q, v);
}

// The sequence that owns a token of the flat token axis.
struct SeqCursor {
  int s, start, end;  // token range [start, end) of sequence s
};
// First sequence whose end lies behind token t (its start may lie behind t as
// well: a gap).  Returns false when there is none.
__device__ __forceinline__ bool find_seq(const int32_t* cu, int n_seqs, int T,
                                         int t, SeqCursor* c) {
  if (cu == nullptr) {
    c->s = t / T;
    c->start = c->s * T;
    c->end = c->start + T;
    return c->s < n_seqs;
  }
  int lo = 0, hi = n_seqs;  // the answer lies in [lo, hi]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (clampi(cu[mid + 1], 0, T) > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  if (lo >= n_seqs) return false;
  c->s = lo;
  seq_range(cu, lo, T, &c->start, &c->end);
  return c->end > t;
}

}  // namespace kda
