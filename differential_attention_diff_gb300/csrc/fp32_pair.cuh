// fp32_pair.cuh — two fp32 numbers in a register pair, and one instruction for
// both: half the issue slots where those are what a kernel lacks.
#pragma once
#include <cuda_runtime.h>

namespace da {

struct F2 {
  unsigned long long v;
  __device__ __forceinline__ F2(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
  __device__ __forceinline__ explicit F2(unsigned long long x) : v(x) {}
  __device__ __forceinline__ uint2 bits() const {
    uint2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(r.x), "=r"(r.y) : "l"(v));
    return r;
  }
};
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a.v), "l"(b.v));
  return F2(r);
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a.v), "l"(b.v));
  return F2(r);
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a.v), "l"(b.v), "l"(c.v));
  return F2(r);
}

// The same as a value type: {lo, hi} with operators.
struct F2Pair {
  unsigned long long v;
  __device__ __forceinline__ F2Pair() {}
  __device__ __forceinline__ F2Pair(float lo, float hi) : v(F2(lo, hi).v) {}
  __device__ __forceinline__ explicit F2Pair(F2 x) : v(x.v) {}
  __device__ __forceinline__ float lo() const { return __uint_as_float(F2(v).bits().x); }
  __device__ __forceinline__ float hi() const { return __uint_as_float(F2(v).bits().y); }
  __device__ __forceinline__ F2Pair operator-() const { return F2Pair(-lo(), -hi()); }
};
__device__ __forceinline__ F2Pair operator*(F2Pair a, F2Pair b) { return F2Pair(mul2(F2(a.v), F2(b.v))); }
__device__ __forceinline__ F2Pair fma2(F2Pair a, F2Pair b, F2Pair c) { return F2Pair(fma2(F2(a.v), F2(b.v), F2(c.v))); }

}  // namespace da
