// Pairs of fp32 values and the instructions that work on both at once.
#pragma once

#include <stdint.h>
#include <string.h>

namespace lrmoe {

struct F2 {
  uint64_t b;
  F2() = default;
  __device__ __forceinline__ F2(float x, float y) { asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(x), "f"(y)); }
  __device__ __forceinline__ explicit F2(float x) : F2(x, x) {}
  static F2 twice(float x) {
    uint32_t u;
    memcpy(&u, &x, 4);
    F2 r;
    r.b = u | ((uint64_t)u << 32);
    return r;
  }
  __device__ __forceinline__ float x() const { return __uint_as_float((uint32_t)b); }
  __device__ __forceinline__ float y() const { return __uint_as_float((uint32_t)(b >> 32)); }
};
__device__ __forceinline__ F2 operator*(F2 a, F2 c) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(a.b), "l"(c.b));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 c) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(a.b), "l"(c.b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 c, F2 d) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.b) : "l"(a.b), "l"(c.b), "l"(d.b));
  return r;
}

}  // namespace lrmoe
