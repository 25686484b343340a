// kv_rows.cuh — rows of K and V as Q4_0 blocks: loads and stores of eight values,
// a group's scale, a word of codes (dq_kv_append, dq_kv_append_rope, dq_kv_read).
#pragma once

#include "kv.cuh"

namespace dqmoe {

// eight consecutive values as fp32
template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&x)[8]) {
  if (DT == DQ_F32) {
    const float4 a = __ldg((const float4*)((const float*)p + i)), b = __ldg((const float4*)((const float*)p + i) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const uint4 v = __ldg((const uint4*)((const unsigned short*)p + i));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (DT == DQ_BF16) {
        x[2 * k] = __uint_as_float(w[k] << 16);
        x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(u32_as_h2(w[k]));
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
      }
    }
  }
}

template <int DT>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&x)[8]) {
  if (DT == DQ_F32) {
    float4* q = (float4*)((float*)p + i);
    q[0] = make_float4(x[0], x[1], x[2], x[3]);
    q[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (DT == DQ_BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
        w[k] = *(const uint32_t*)&v;
      } else {
        w[k] = h2_as_u32(__floats2half2_rn(x[2 * k], x[2 * k + 1]));
      }
    }
    *(uint4*)((unsigned short*)p + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__device__ __forceinline__ float max_of3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float min_of3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max_of8(const float (&x)[8]) {
  return max_of3(max_of3(x[0], x[1], x[2]), max_of3(x[3], x[4], x[5]), fmaxf(x[6], x[7]));
}
__device__ __forceinline__ float min_of8(const float (&x)[8]) {
  return min_of3(min_of3(x[0], x[1], x[2]), min_of3(x[3], x[4], x[5]), fminf(x[6], x[7]));
}

// The value of the largest magnitude of the 32 that 4 consecutive lanes hold eight of each, the first of
// equal ones; values beyond +-65504 count as that.  The largest and the smallest value tell it, unless they
// are equal in magnitude (or beyond): then, for the whole warp, the values are gone through in order.
__device__ __forceinline__ float first_largest(const float (&x)[8], int lane) {
  float hi = max_of8(x), lo = min_of8(x);
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
  }
  float m = hi > -lo ? hi : lo;
  if (__any_sync(0xffffffffu, hi == -lo || fmaxf(hi, -lo) > 65504.f)) {
    m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = fminf(fmaxf(x[i], -65504.f), 65504.f);
      if (fabsf(v) > fabsf(m)) m = v;
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      const float p = __shfl_xor_sync(0xffffffffu, m, o);
      const bool mine = fabsf(m) > fabsf(p) || (fabsf(m) == fabsf(p) && (lane & o) == 0);
      m = mine ? m : p;
    }
  }
  return m;
}

// The Q4_0 word of eight values with scale d, value e in nibble NIB(e): floor(x / d + 8.5), in [0, 15].
//
// For 16-bit x this is exact without a division.  x and d have at most 11 bits, so a quotient that is not
// half-way between two codes is at least 2^-14 from it (for x = X 2^a, d = D 2^b the distance is
// |2 X 2^(a-b) - (2k+1) D| / 2D, and 2^(a-b) >= D / 4X wherever the quotient is not below 1/4).  With 1 / d
// within 2^-22 of itself the sum below is off by less than 2^-17, so adding 2^-16 decides every half-way
// case upwards and no other case differently.  The sum is taken in units of 15.5, where the saturating FMA
// clamps it, and brought back by one that rounds towards zero at 2^23: the code is its lowest bits, and eight
// of them are packed by multiplications whose surplus is subtracted once.  fp32 x has no such margin: one
// correctly rounded quotient each.
template <int DT, bool V>
__device__ __forceinline__ uint32_t q4_word(const float (&x)[8], __half d) {
  const float df = __half2float(d);
  float inv;
  asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(df));
  inv = df == 0.f ? 0.f : inv * (1.f / 15.5f);
  uint32_t word = 0, surplus = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t unit = 1u << (V ? 4 * e : 4 * (e >> 1) + 16 * (e & 1));
    float t;
    if (DT == DQ_F32) {
      const float q = df == 0.f ? 8.5f : __fadd_rn(__fdiv_rn(fminf(fmaxf(x[e], -65504.f), 65504.f), df), 8.5f);
      t = __fadd_rz(fminf(fmaxf(q, 0.f), 15.5f), 8388608.f);
    } else {
      t = __fmaf_rz(__saturatef(fmaf(x[e], inv, (8.5f + 0x1p-16f) / 15.5f)), 15.5f, 8388608.f);
    }
    word += __float_as_uint(t) * unit;
    surplus += 0x4B000000u * unit;
  }
  return word - surplus;
}

template <typename F>
int by_dim(int dim, F f) {
  switch (dim) {
    case 64: return f(std::integral_constant<int, 64>());
    case 128: return f(std::integral_constant<int, 128>());
    default: return f(std::integral_constant<int, 256>());
  }
}

inline int launched(cudaError_t e) {
  if (e != cudaSuccess) return DQ_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? DQ_OK : DQ_ERR_CUDA;
}

}  // namespace dqmoe
