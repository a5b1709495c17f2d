// Rows of 16-byte words as fp32 registers, for the kernels that stream heads'
// rows (rotary positions, the paged cache, single-token attention).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace ulysses {
namespace rows {

// How a cache holds its rows: as they are, in 8 bits or in 4.
enum Held { kAsIs, kE4m3, kE2m1 };

// Streaming accesses: each word is used once, so L1 keeps none of them.
__device__ __forceinline__ uint4 ld16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld8(const void* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld4(const void* p) {
  uint32_t v;
  asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ void st16(void* p, uint4 v) { *reinterpret_cast<uint4*>(p) = v; }
__device__ __forceinline__ void st8(void* p, uint2 v) { *reinterpret_cast<uint2*>(p) = v; }

__device__ __forceinline__ void bf16x2_to_f32(uint32_t w, float* f) {
  f[0] = __uint_as_float(w << 16);
  f[1] = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ uint32_t f32_to_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 codes (low half of w) as two f16: exact, every code is an f16 value.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(w));
  return r;
}
__device__ __forceinline__ uint16_t f32_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t h = e4m3x2_to_f16x2((uint16_t)(w >> (16 * i)));
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}
// Eight e2m1 codes (the lowest four bits first) as f16 pairs: exact.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&h)[4]) {
  asm("{ .reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3; }"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}
// Eight fp32 values as e2m1 codes: nearest, half way to the even code, at most 6.
__device__ __forceinline__ uint32_t f32_to_e2m1x8(const float* f) {
  uint32_t r;
  asm("{ .reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3}; }"
      : "=r"(r) : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// Where the parts of a row of a 4-bit cache are: a page of a head holds its rows'
// codes ([page][D / 2] bytes) and behind them their block scales ([page][D / 16]).
// `row` counts rows ([num_pages][H_kv][page]), `slot` is the row's in its page.
__device__ __forceinline__ int64_t e2m1_codes(int64_t row, int slot, int D) {
  return (row - slot) * (D / 16 * 9) + slot * (D / 2);
}
__device__ __forceinline__ int64_t e2m1_blocks(int64_t row, int slot, int page, int D) {
  return (row - slot) * (D / 16 * 9) + (int64_t)page * (D / 2) + slot * (D / 16);
}

__device__ __forceinline__ float max_nan(float x, float y) {   // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
// Eight fp32 values times `by` as e4m3 codes.
__device__ __forceinline__ uint2 to_codes(const float* f, float by) {
  uint2 c;
  c.x = f32_to_e4m3x2(f[0] * by, f[1] * by) | (uint32_t)f32_to_e4m3x2(f[2] * by, f[3] * by) << 16;
  c.y = f32_to_e4m3x2(f[4] * by, f[5] * by) | (uint32_t)f32_to_e4m3x2(f[6] * by, f[7] * by) << 16;
  return c;
}

// Eight elements of type T: 16 bytes of bf16, two 16-byte words of fp32.
template <typename T> struct Row8;
template <> struct Row8<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = ld16(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { st16(p, w); }
  __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
  // largest magnitude, NaN if any is (two elements an instruction)
  __device__ __forceinline__ float amax() const {
    const uint32_t s = 0x7fff7fffu;
    const uint32_t m = max_nan_bf16x2(max_nan_bf16x2(w.x & s, w.y & s), max_nan_bf16x2(w.z & s, w.w & s));
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
  __device__ __forceinline__ uint2 codes(float by) const {
    float f[8];
    get(f);
    return to_codes(f, by);
  }
  __device__ __forceinline__ void get(float* f) const {
    bf16x2_to_f32(w.x, f); bf16x2_to_f32(w.y, f + 2); bf16x2_to_f32(w.z, f + 4); bf16x2_to_f32(w.w, f + 6);
  }
  __device__ __forceinline__ void set(const float* f) {
    w = make_uint4(f32_to_bf16x2(f[0], f[1]), f32_to_bf16x2(f[2], f[3]), f32_to_bf16x2(f[4], f[5]),
                   f32_to_bf16x2(f[6], f[7]));
  }
};
template <> struct Row8<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const float* p) { a = ld16(p); b = ld16(p + 4); }
  __device__ __forceinline__ void store(float* p) const { st16(p, a); st16(p + 4, b); }
  __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ float amax() const {
    float f[8];
    get(f);
    float m = fabsf(f[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(f[i]));
    return m;
  }
  __device__ __forceinline__ uint2 codes(float by) const {
    float f[8];
    get(f);
    return to_codes(f, by);
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y); f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
    f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y); f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
  }
  __device__ __forceinline__ void set(const float* f) {
    a = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    b = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
  }
};

// Rows r, r + step, r + 2 step, ... of a block of `no` x `ni` rows, as (outer,
// inner) indexes: one division at the start, none per row.
struct RowWalk {
  int o, i, ni, step_o, step_i;
  __device__ __forceinline__ RowWalk(int r, int step, int ni_) : ni(ni_) {
    o = r / ni;
    i = r - o * ni;
    step_o = step / ni;
    step_i = step - step_o * ni;
  }
  __device__ __forceinline__ void next() {
    i += step_i;
    o += step_o;
    if (i >= ni) { i -= ni; ++o; }
  }
};

}  // namespace rows
}  // namespace ulysses
