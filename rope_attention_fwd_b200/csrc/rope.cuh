// rope.cuh -- the rotation of one channel pair at one position, shared by the stand-alone
// rotation and the cache append (both produce the same bits for the same row).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace ra {

// amplitude * (cos, sin) of phi = pos * theta, formed in fp64 and rounded once to fp32.
// Cody-Waite reduction to |r| <= pi/4 by multiples of pi/2 held in two fp64 words (the angle
// of a position of 2^31 keeps more than 20 bits below fp32's), then the Taylor series of sin
// and cos to r^15 and r^14: the truncation is below 1e-15, far below fp32's half step, so the
// result is the correctly rounded one but for ties closer than that.  About 25 fp64
// instructions; the library's sincos spends twice as many and keeps a slow path for large
// arguments on the stack.
__device__ __forceinline__ float2 cos_sin(double pos, double theta, double amplitude) {
  const double phi = pos * theta;
  const double k = rint(phi * 0.63661977236758134308);  // 2 / pi
  double r = fma(-k, 1.5707963267948965580, phi);       // pi / 2, high word
  r = fma(-k, 6.1232339957367660359e-17, r);            // pi / 2, low word
  const double z = r * r;
  double s = fma(z, -1.0 / 1307674368000.0, 1.0 / 6227020800.0);
  s = fma(z, s, -1.0 / 39916800.0);
  s = fma(z, s, 1.0 / 362880.0);
  s = fma(z, s, -1.0 / 5040.0);
  s = fma(z, s, 1.0 / 120.0);
  s = fma(z, s, -1.0 / 6.0);
  s = fma(r * z, s, r);
  double c = fma(z, -1.0 / 87178291200.0, 1.0 / 479001600.0);
  c = fma(z, c, -1.0 / 3628800.0);
  c = fma(z, c, 1.0 / 40320.0);
  c = fma(z, c, -1.0 / 720.0);
  c = fma(z, c, 1.0 / 24.0);
  c = fma(z, c, -0.5);
  c = fma(z, c, 1.0);
  const int quadrant = (int)((long long)k & 3);
  double co = (quadrant & 1) ? s : c, si = (quadrant & 1) ? c : s;
  if (quadrant == 1 || quadrant == 2) co = -co;
  if (quadrant >= 2) si = -si;
  return make_float2((float)(amplitude * co), (float)(amplitude * si));
}

// (x0, x1) turned by the angle of cs; every operation rounded on its own, so that the codes
// of a quantised row do not depend on how the compiler contracts products and sums.
__device__ __forceinline__ float2 turn(float2 cs, float x0, float x1) {
  return make_float2(__fsub_rn(__fmul_rn(cs.x, x0), __fmul_rn(cs.y, x1)),
                     __fadd_rn(__fmul_rn(cs.y, x0), __fmul_rn(cs.x, x1)));
}
// The inverse turn (times the squared amplitude): the gradient's way back.
__device__ __forceinline__ float2 turn_back(float2 cs, float y0, float y1) {
  return make_float2(__fadd_rn(__fmul_rn(cs.x, y0), __fmul_rn(cs.y, y1)),
                     __fsub_rn(__fmul_rn(cs.x, y1), __fmul_rn(cs.y, y0)));
}

// V elements of T at p as fp32 and back: one 16-byte access when V fills it, else one element.
template <typename T, int V>
struct Vec;
template <>
struct Vec<__nv_bfloat16, 8> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    w = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const {
    *reinterpret_cast<uint4*>(p) = w;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    w = make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Vec<float, 4> {
  float4 w;
  __device__ __forceinline__ void load(const float* p) { w = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = w; }
  __device__ __forceinline__ void get(float (&f)[4]) const {
    f[0] = w.x, f[1] = w.y, f[2] = w.z, f[3] = w.w;
  }
  __device__ __forceinline__ void set(const float (&f)[4]) {
    w = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <>
struct Vec<__nv_bfloat16, 1> {
  __nv_bfloat16 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *p; }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *p = w; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = __bfloat162float(w); }
  __device__ __forceinline__ void set(const float (&f)[1]) { w = __float2bfloat16_rn(f[0]); }
};
template <>
struct Vec<float, 1> {
  float w;
  __device__ __forceinline__ void load(const float* p) { w = *p; }
  __device__ __forceinline__ void store(float* p) const { *p = w; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = w; }
  __device__ __forceinline__ void set(const float (&f)[1]) { w = f[0]; }
};

}  // namespace ra
