// pair.cuh — numbers of 46 bits as pairs of floats, for the few values that fp32 leaves in doubt: an instruction in 64
// bits takes a warp some 60 cycles here.
#pragma once

#include <cuda_runtime.h>

namespace dqmoe {

// A number as the sum h + l, |l| at most half a unit in the last place of h (Dekker's and Knuth's exact sums and
// products, with FMA).
struct Pair {
  float h, l;
};
__device__ __forceinline__ Pair quick_sum(float a, float b) {          // |a| >= |b|, or a = 0
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Pair sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const Pair s = sum(a.h, b.h), t = sum(a.l, b.l);
  const Pair u = quick_sum(s.h, __fadd_rn(s.l, t.h));
  return quick_sum(u.h, __fadd_rn(u.l, t.l));
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
  const float p = __fmul_rn(a.h, b.h);
  const float e = __fmaf_rn(a.h, b.l, __fmaf_rn(a.l, b.h, __fmaf_rn(a.h, b.h, -p)));
  return quick_sum(p, e);
}
__device__ __forceinline__ Pair divide(Pair a, Pair b) {
  const float q = __fdiv_rn(a.h, b.h);
  // the rest of a - q b, over b
  const float p = __fmul_rn(q, b.h), e = __fmaf_rn(q, b.h, -p);
  const float r = __fadd_rn(__fsub_rn(__fsub_rn(a.h, p), e), __fmaf_rn(-q, b.l, a.l));
  return quick_sum(q, __fdiv_rn(r, b.h));
}

}  // namespace dqmoe
