// The paged key-value cache: writing new tokens' rows, as they are, in 8 bits or
// in 4, and gathering them back (include/ulysses.h, ulysses_cache_write /
// ulysses_cache_read).
//
//   amax = max(max_d |x_d|, 2^-100), scale = amax / 448, code_d = e4m3(x_d * (448 / amax))
//
// or, in 4 bits, with r the least power of two with amax <= 2688 r,
//
//   b = e4m3(max_{d in its 16} |x_d / r| / 6), code_d = e2m1(x_d / r / b), scale = r
//
// (a power of two: x / r is exact, and so are code * b * r on the way back.)
// 448 is e4m3's largest value, so no code saturates; the floor keeps the
// reciprocal finite for rows of zeros and of the smallest subnormals.  One
// scale per row (token, head) is 3% of a 128-byte row and lets a row be
// written without reading any other.
//
// Bound by HBM: rows are read and written once.  A CTA takes a block of tokens
// with all their heads, K and V: it resolves each token's place once (sequence
// by bisection in cu, page from the table) and streams the rows; D / 16 lanes
// hold a row, 16 elements each, so the row's largest magnitude is a 2- or
// 3-step shuffle.  Instruction issue is next to HBM here: 8 elements a lane
// with a division for each row took 186 us where this takes 130 (131072 tokens
// of 8 heads of 128, bf16 to e4m3, K and V: 814 MB, 94% of the measured copy
// rate), so bf16 maxima are taken two at a time and one pair of divisions
// serves four rows.  Reading 65536 such tokens back: 65 us (407 MB, 93%).  (GPU
// times; a call among others takes 132 and 67 us.)
#include "internal.h"
#include "rows.cuh"

namespace ulysses {

ULYSSES_ERROR_READER(read_error_kv_cache)

namespace {

using namespace rows;

constexpr int kThreads = 256;
constexpr int kMaxTokens = kThreads;   // of a CTA: a thread resolves a token's place

// Row of the caches ([num_pages][H][page] rows, before the head's offset) of
// token t, or -1: nothing to do (past the last sequence, an empty place of the
// batch) or outside the table (reported).  write: a.lens are the lengths with
// the new tokens; read: the first positions (may be NULL).
// slot: the row's in its page.
__device__ __forceinline__ int64_t place_of(const CacheArgs& a, int64_t t, bool write, int& slot) {
  int b = (int)t;
  int64_t pos;
  if (a.cu) {
    b = doc_of(a.cu, a.B, t);
    const int64_t lo = __ldg(a.cu + b), hi = __ldg(a.cu + b + 1);
    if (t < lo || t >= hi || lo < 0 || hi > a.T) return -1;   // the last two reported by check_cu
    pos = write ? (int64_t)__ldg(a.lens + b) - (hi - t) : (a.lens ? (int64_t)__ldg(a.lens + b) : 0) + t - lo;
  } else {
    const int len = __ldg(a.lens + b);
    if (len == 0) return -1;
    pos = (int64_t)len - 1;
  }
  if (pos < 0 || pos >= (int64_t)a.cols * a.page) {
    raise_error(kErrPages);
    return -1;
  }
  const int col = (int)(pos / a.page);
  const int pg = __ldg(a.table + (int64_t)b * a.cols + col);
  if (pg < 0 || pg >= a.num_pages) {
    raise_error(kErrPages);
    return -1;
  }
  slot = (int)(pos - (int64_t)col * a.page);
  return (int64_t)pg * a.H * a.page + slot;
}

// cu[0] == 0, non-decreasing, cu[B] <= T; checked by the first CTA.  A range that
// does not lie in [0, T] shows in one of these.
__device__ __forceinline__ void check_cu(const CacheArgs& a) {
  if (blockIdx.x != 0 || !a.cu) return;
  for (int i = threadIdx.x; i <= a.B; i += kThreads) {
    const int c = __ldg(a.cu + i);
    if ((i == 0 && c != 0) || (i > 0 && c < __ldg(a.cu + i - 1)) || (i == a.B && c > a.T)) raise_error(kErrSeqlens);
  }
}

// The rows of a CTA's tokens x heads, K's and then V's, in an order in which
// rows that lie together in the tokens' tensor are neighbours: heads of one
// token where those are closer, else tokens of one head.
// Rows that a lane has in work at once: 64 bytes of loads or more in flight.
// A lane holds 16 elements of a row, the 8-element words lane and lane + D / 16.
template <typename T, Held kHeld, bool kWrite>
constexpr int rows_in_work() { return kWrite ? (sizeof(T) == 2 ? 4 : 2) : (kHeld != kAsIs ? 4 : (sizeof(T) == 2 ? 2 : 1)); }

template <typename T, Held kHeld, bool kWeights>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const __grid_constant__ CacheArgs a, int tb) {
  __shared__ int64_t place[kMaxTokens];
  const int64_t t0 = (int64_t)blockIdx.x * tb;
  const int tokens = (int)(a.T - t0 < tb ? a.T - t0 : tb);
  check_cu(a);
  int slot;
  if ((int)threadIdx.x < tokens) place[threadIdx.x] = place_of(a, t0 + threadIdx.x, true, slot);
  __syncthreads();
  constexpr int kRows = rows_in_work<T, kHeld, true>();
  const int lanes = a.D / 16, lane = threadIdx.x % lanes, e0 = lane * 8, e1 = (lane + lanes) * 8;
  const bool heads_fast = a.k_h <= a.k_s;
  const int ni = heads_fast ? a.H : tokens, no = heads_fast ? tokens : a.H;
  RowWalk walk(threadIdx.x / lanes, kThreads / lanes, ni);
  // every lane of a warp runs the same number of rounds: the row maximum is a shuffle
  for (int left = 2 * no * ni; left > 0; left -= kRows * (kThreads / lanes)) {
    Row8<T> w[kRows][2];
    int64_t row[kRows];
    bool second[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      row[u] = -1;
      w[u][0].zero();
      w[u][1].zero();
      second[u] = walk.o >= no;
      if (walk.o < 2 * no) {
        const int o = second[u] ? walk.o - no : walk.o;
        const int t = heads_fast ? o : walk.i, h = heads_fast ? walk.i : o;
        const int64_t at = place[t];
        if (at >= 0 && in_bounds(at + (int64_t)h * a.page, a.num_pages * a.H * a.page)) {
          row[u] = at + (int64_t)h * a.page;
          if (kWeights && lane == 0 && !second[u]) a.w[row[u]] = 0.f;
          const int64_t off = second[u] ? (t0 + t) * a.v_s + h * a.v_h : (t0 + t) * a.k_s + h * a.k_h;
          const T* src = reinterpret_cast<const T*>(second[u] ? a.v : a.k) + off;
          w[u][0].load(src + e0);
          w[u][1].load(src + e1);
        }
      }
      walk.next();
    }
    if (kHeld == kAsIs) {
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        if (row[u] < 0) continue;
        T* dst = reinterpret_cast<T*>(second[u] ? a.vc : a.kc) + row[u] * a.D;
        w[u][0].store(dst + e0);
        w[u][1].store(dst + e1);
      }
      continue;
    }
    // the rows' largest magnitudes; lane u of a row's lanes keeps row u's
    float mine = 0.f;
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      float amax = max_nan(w[u][0].amax(), w[u][1].amax());
      for (int o = lanes / 2; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      mine = lane % kRows == u ? amax : mine;
    }
    // so one pair of divisions serves kRows rows
    mine = max_nan(mine, 7.888609052210118e-31f);   // 2^-100
    const float inv = 448.0f / mine;
    const float scale = mine <= 3.4028234663852886e38f ? mine / 448.0f : __int_as_float(0x7fc00000);
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const float by = __shfl_sync(0xffffffffu, inv, u, lanes);
      const uint2 c0 = w[u][0].codes(by), c1 = w[u][1].codes(by);
      if (row[u] < 0) continue;
      uint8_t* dst = reinterpret_cast<uint8_t*>(second[u] ? a.vc : a.kc) + row[u] * a.D;
      st8(dst + e0, c0);
      st8(dst + e1, c1);
      if (lane == u) (second[u] ? a.vs : a.ks)[row[u]] = scale;
    }
  }
}

// ------------------------------------------------------------------ 4-bit rows

// Two floats at once.
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
  float2 r;
  asm("{ .reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 c, a, b;\n\tmov.b64 {%0, %1}, c; }"
      : "=f"(r.x), "=f"(r.y) : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 r;
  asm("{ .reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 c, a, b;\n\tmov.b64 {%0, %1}, c; }"
      : "=f"(r.x), "=f"(r.y) : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  float2 r;
  asm("{ .reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\t"
      "mov.b64 {%0, %1}, d; }"
      : "=f"(r.x), "=f"(r.y) : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
  return r;
}
// the larger magnitudes, NaN if either is (signs mean nothing)
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// A block of a row, 16 elements: a lane's part.  Loads that L1 may keep: each of a
// lane's 16-byte words is half of what a sector has.
//
// A quotient next to a border between two codes has to fall on its side in 64 bits
// too, and one on it exactly on it: ties go to the even code.
template <typename T> struct Block;
template <> struct Block<__nv_bfloat16> {
  uint4 w[2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    w[0] = *reinterpret_cast<const uint4*>(p);
    w[1] = *reinterpret_cast<const uint4*>(p + 8);
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ float amax() const {
    uint32_t m = max_abs_bf16x2(max_abs_bf16x2(w[0].x, w[0].y), max_abs_bf16x2(w[0].z, w[0].w));
    m = max_abs_bf16x2(m, max_abs_bf16x2(max_abs_bf16x2(w[1].x, w[1].y), max_abs_bf16x2(w[1].z, w[1].w)));
    return max_nan(fabsf(__uint_as_float(m << 16)), fabsf(__uint_as_float(m & 0xffff0000u)));
  }
  // Elements over b * the row's scale, whose inverse to nearest is r.  A border m
  // times b has 7 bits and an element 8, so a quotient that is not m is 2^-8 of it
  // away, 2^-10 at least; rounded to multiples of 2^-12 (what a sum with 2560 does,
  // the product being exact in it), those on a border are back on it.
  __device__ __forceinline__ void over(float, float r, float (&f)[16]) const {
    const uint32_t x[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 q = add2(fma2(make_float2(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xffff0000u)),
                                 make_float2(r, r), make_float2(2560.f, 2560.f)), make_float2(-2560.f, -2560.f));
      f[2 * i] = q.x;
      f[2 * i + 1] = q.y;
    }
  }
};
template <> struct Block<float> {
  float4 w[4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(p + 4 * i);
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ float amax() const {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max_nan(max_nan(max_nan(m, fabsf(w[i].x)), max_nan(fabsf(w[i].y), fabsf(w[i].z))), fabsf(w[i].w));
    return m;
  }
  // Rounded to nearest: a quotient's residual is exact in an FMA, and one step with
  // it rounds correctly (Markstein 1990).
  __device__ __forceinline__ void over(float minus_b, float r, float (&f)[16]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 v = w[i / 2];
      const float2 x = i % 2 ? make_float2(v.z, v.w) : make_float2(v.x, v.y), q = mul2(x, make_float2(r, r));
      const float2 y = fma2(fma2(q, make_float2(minus_b, minus_b), x), make_float2(r, r), q);
      f[2 * i] = y.x;
      f[2 * i + 1] = y.y;
    }
  }
};
// The same for one quotient, given -y and 1 / y to nearest.
__device__ __forceinline__ float divided(float x, float minus_y, float inv_y) {
  const float q = x * inv_y;
  return fmaf(fmaf(q, minus_y, x), inv_y, q);
}

// Where a CTA's tokens are in a 4-bit cache, for the first head: row (-1: nothing to
// do), and offsets of the codes and of the block scales.  Every head is
// page * 9 D / 16 bytes, and `page` rows, further.
struct Places4 {
  int64_t row[kMaxTokens], codes[kMaxTokens], blocks[kMaxTokens];
  __device__ __forceinline__ void find(const CacheArgs& a, int64_t t0, int tokens, bool write) {
    if ((int)threadIdx.x < tokens) {
      int slot = 0;
      const int64_t at = place_of(a, t0 + threadIdx.x, write, slot);
      row[threadIdx.x] = at;
      codes[threadIdx.x] = e2m1_codes(at, slot, a.D);
      blocks[threadIdx.x] = e2m1_blocks(at, slot, a.page, a.D);
    }
  }
};

// Rows to 4 bits.  A lane has a block of a row (D / 16 lanes a row), so its scale
// is the lane's own, and the row's a 2- or 3-step shuffle away.  Instruction issue
// is next to HBM again: quotients are formed two at a time, the inverse of a block
// scale comes from a table of the 127 there are, the row's scale by its bits, and
// places from offsets found once a token.  A code of magnitude 0 may have either sign.
// (131072 tokens of 8 heads of 128, bf16, K and V: 125 us for 697 MB, 82% of the
// copy rate; 113 million warp instructions keep the issue slots 73% busy.  With
// quotients by residual as for fp32 rows and places formed row by row: 161; with
// the layout of the e4m3 kernel, half a block a lane: 200.)
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) cache_write_4bit_kernel(const __grid_constant__ CacheArgs a, int tb) {
  __shared__ Places4 place;
  __shared__ float inverse[128];                           // of e4m3 values; of 0: 0
  const int64_t t0 = (int64_t)blockIdx.x * tb;
  const int tokens = (int)(a.T - t0 < tb ? a.T - t0 : tb);
  check_cu(a);
  place.find(a, t0, tokens, true);
  if (threadIdx.x < 128) {
    const uint32_t h = e4m3x2_to_f16x2((uint16_t)threadIdx.x);
    const float b = __half2float(__ushort_as_half((unsigned short)h));
    inverse[threadIdx.x] = b > 0.f ? 1.0f / b : 0.f;
  }
  __syncthreads();
  constexpr int kRows = sizeof(T) == 2 ? 4 : 2;
  const int lanes = a.D / 16, lane = threadIdx.x % lanes;
  const bool heads_fast = a.k_h <= a.k_s;
  const int ni = heads_fast ? a.H : tokens, no = heads_fast ? tokens : a.H;
  const int head_rows = a.page, head_bytes = a.page * (a.D / 16) * 9;
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {                   // K's rows, then V's
    const int64_t step_t = side ? a.v_s : a.k_s, step_h = side ? a.v_h : a.k_h;
    const T* const from = reinterpret_cast<const T*>(side ? a.v : a.k) + t0 * step_t + lane * 16;
    uint8_t* const to = reinterpret_cast<uint8_t*>(side ? a.vc : a.kc);
    float* const scales = side ? a.vs : a.ks;
    RowWalk walk(threadIdx.x / lanes, kThreads / lanes, ni);
    // every lane of a warp runs the same number of rounds: the row maximum is a shuffle
    for (int left = no * ni; left > 0; left -= kRows * (kThreads / lanes)) {
      Block<T> w[kRows];
      int t[kRows], h[kRows];                              // t -1: no row
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        t[u] = -1;
        h[u] = 0;
        if (walk.o < no) {
          h[u] = heads_fast ? walk.i : walk.o;
          const int token = heads_fast ? walk.o : walk.i;
          const int64_t at = place.row[token];
          if (at >= 0 && in_bounds(at + (int64_t)h[u] * head_rows, a.num_pages * a.H * a.page)) {
            t[u] = token;
            w[u].load(from + token * step_t + h[u] * step_h);
          }
        }
        if (t[u] < 0) w[u].zero();
        walk.next();
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const float block = w[u].amax();
        float amax = block;
        for (int o = lanes / 2; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (t[u] < 0) continue;
        // 2688 is 1.3125 * 2^11: the exponent e that takes the maximum to (1344, 2688] times 2^e
        amax = max_nan(amax, 7.888609052210118e-31f);      // 2^-100
        const uint32_t e = (__float_as_uint(amax) + 0x57ffffu >> 23) - 11;
        const float down = __uint_as_float((254 - e) << 23);
        const uint16_t code = f32_to_e4m3x2(divided(block * down, -6.0f, 1.0f / 6.0f), 0.f);
        const uint32_t bh = e4m3x2_to_f16x2(code);
        // (b = 0: all of the block is below half of the smallest scale)
        const float b = -__half2float(__ushort_as_half((unsigned short)bh)), up = __uint_as_float(e << 23);
        float f[16];
        w[u].over(b * up, inverse[code & 127] * down, f);
        const int64_t head = (int64_t)h[u] * head_bytes;
        st8(to + place.codes[t[u]] + head + lane * 8, b < 0.f ? make_uint2(f32_to_e2m1x8(f), f32_to_e2m1x8(f + 8)) : make_uint2(0, 0));
        to[place.blocks[t[u]] + head + lane] = (uint8_t)code;
        if (lane == 0) {
          const int64_t row = place.row[t[u]] + (int64_t)h[u] * head_rows;
          scales[row] = amax <= 3.4028234663852886e38f ? up : __int_as_float(0x7fc00000);
          if (a.w && side == 0) a.w[row] = 0.f;
        }
      }
    }
  }
}

// Rows from 4 bits: code * block scale exactly in f16, and the row's in fp32.  (65536
// tokens of 8 heads of 128 to bf16: 59 us for 348 MB, 87% of the copy rate; 131072
// 108 us, 95%.)
template <typename T>
__global__ void __launch_bounds__(kThreads) cache_read_4bit_kernel(const __grid_constant__ CacheArgs a, int tb) {
  __shared__ Places4 place;
  const int64_t t0 = (int64_t)blockIdx.x * tb;
  const int tokens = (int)(a.T - t0 < tb ? a.T - t0 : tb);
  check_cu(a);
  place.find(a, t0, tokens, false);
  __syncthreads();
  constexpr int kRows = 4;
  const int lanes = a.D / 16, lane = threadIdx.x % lanes;  // a lane has words lane and lane + D / 16, of 8 elements
  const bool heads_fast = a.k_h <= a.k_s;
  const int ni = heads_fast ? a.H : tokens, no = heads_fast ? tokens : a.H;
  const int head_rows = a.page, head_bytes = a.page * (a.D / 16) * 9;
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const int64_t step_t = side ? a.v_s : a.k_s, step_h = side ? a.v_h : a.k_h;
    T* const to = reinterpret_cast<T*>(side ? a.v : a.k) + t0 * step_t + lane * 8;
    const uint8_t* const from = reinterpret_cast<const uint8_t*>(side ? a.vc : a.kc);
    const float* const scales = side ? a.vs : a.ks;
    RowWalk walk(threadIdx.x / lanes, kThreads / lanes, ni);
    while (walk.o < no) {
      uint32_t codes[kRows][2], blocks[kRows][2];
      float scale[kRows];
      T* dst[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        dst[u] = nullptr;
        if (walk.o < no) {
          const int h = heads_fast ? walk.i : walk.o, t = heads_fast ? walk.o : walk.i;
          const int64_t at = place.row[t], row = at + (int64_t)h * head_rows;
          if (at >= 0 && in_bounds(row, a.num_pages * a.H * a.page)) {
            const int64_t head = (int64_t)h * head_bytes;
            dst[u] = to + t * step_t + h * step_h;
            const uint32_t* src = reinterpret_cast<const uint32_t*>(from + place.codes[t] + head) + lane;
            const uint8_t* bs = from + place.blocks[t] + head + lane / 2;
            codes[u][0] = ld4(src);
            codes[u][1] = ld4(src + lanes);
            blocks[u][0] = __ldg(bs);
            blocks[u][1] = __ldg(bs + lanes / 2);
            scale[u] = __ldg(scales + row);
          }
          walk.next();
        }
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        if (dst[u] == nullptr) continue;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t h[4];
          e2m1x8_to_f16x2(codes[u][x], h);
          const uint32_t b = e4m3x2_to_f16x2((uint16_t)(blocks[u][x] * 0x101u));
          float f[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t p = hmul2(h[i], b);             // 2 + 4 significant bits, in f16's range
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&p));
            f[2 * i] = v.x * scale[u];
            f[2 * i + 1] = v.y * scale[u];
          }
          Row8<T> y;
          y.set(f);
          y.store(dst[u] + x * lanes * 8);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ reading

template <typename T, Held kHeld>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ CacheArgs a, int tb) {
  __shared__ int64_t place[kMaxTokens];
  const int64_t t0 = (int64_t)blockIdx.x * tb;
  const int tokens = (int)(a.T - t0 < tb ? a.T - t0 : tb);
  check_cu(a);
  int slot;
  if ((int)threadIdx.x < tokens) place[threadIdx.x] = place_of(a, t0 + threadIdx.x, false, slot);
  __syncthreads();
  constexpr int kRows = rows_in_work<T, kHeld, false>();
  const int lanes = a.D / 16, lane = threadIdx.x % lanes, e0 = lane * 8, e1 = (lane + lanes) * 8;
  const bool heads_fast = a.k_h <= a.k_s;
  const int ni = heads_fast ? a.H : tokens, no = heads_fast ? tokens : a.H;
  RowWalk walk(threadIdx.x / lanes, kThreads / lanes, ni);
  while (walk.o < 2 * no) {
    Row8<T> w[kRows][2];
    uint2 codes[kRows][2];
    float scale[kRows];
    T* dst[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      dst[u] = nullptr;
      if (walk.o < 2 * no) {
        const bool second = walk.o >= no;
        const int o = second ? walk.o - no : walk.o;
        const int t = heads_fast ? o : walk.i, h = heads_fast ? walk.i : o;
        const int64_t at = place[t], row = at + (int64_t)h * a.page;
        if (at >= 0 && in_bounds(row, a.num_pages * a.H * a.page)) {
          const int64_t off = second ? (t0 + t) * a.v_s + h * a.v_h : (t0 + t) * a.k_s + h * a.k_h;
          dst[u] = reinterpret_cast<T*>(second ? a.v : a.k) + off;
          if (kHeld == kE4m3) {
            const uint8_t* src = reinterpret_cast<const uint8_t*>(second ? a.vc : a.kc) + row * a.D;
            codes[u][0] = ld8(src + e0);
            codes[u][1] = ld8(src + e1);
            scale[u] = __ldg((second ? a.vs : a.ks) + row);
          } else {
            const T* src = reinterpret_cast<const T*>(second ? a.vc : a.kc) + row * a.D;
            w[u][0].load(src + e0);
            w[u][1].load(src + e1);
          }
        }
        walk.next();
      }
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      if (dst[u] == nullptr) continue;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (kHeld == kE4m3) {
          float f[8];
          e4m3x4_to_f32(codes[u][x].x, f);
          e4m3x4_to_f32(codes[u][x].y, f + 4);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= scale[u];
          w[u][x].set(f);
        }
        w[u][x].store(dst[u] + (x ? e1 : e0));
      }
    }
  }
}

// Tokens of one CTA: eight rows a lane group (two rounds of four), so that
// resolving the places is small beside them, unless that leaves SMs idle.
// (e4m3, 4 heads of 64: 45808 tokens 15.4 us; 16 tokens a CTA, which half fill
// a round, 22.3.  17021 tokens 7.8 us; four CTAs an SM instead of one 10.0.)
// Rows to 4 bits: twice as many, for what a CTA sets up costs more (131072 tokens
// of 8 heads of 128: 125 us, with 8 rows 138; 8191 tokens 12.5).
int tokens_per_cta(const CacheArgs& a, int rows = 8) {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  int tb = 1;
  while (tb < kMaxTokens && 2 * tb * a.H * (a.D / 16) < rows * kThreads) tb *= 2;
  while (tb > 1 && (a.T + tb - 1) / tb < sms) tb /= 2;
  return tb;
}

}  // namespace

namespace {

template <typename T, bool kWeights>
void write_rows(const CacheArgs& a, unsigned grid, int tb, cudaStream_t st) {
  if (a.cache_dtype == ULYSSES_E2M1) cache_write_4bit_kernel<T><<<grid, kThreads, 0, st>>>(a, tb);
  else if (a.cache_dtype == ULYSSES_E4M3) cache_write_kernel<T, kE4m3, kWeights><<<grid, kThreads, 0, st>>>(a, tb);
  else cache_write_kernel<T, kAsIs, kWeights><<<grid, kThreads, 0, st>>>(a, tb);
}
template <typename T>
void read_rows(const CacheArgs& a, unsigned grid, int tb, cudaStream_t st) {
  if (a.cache_dtype == ULYSSES_E2M1) cache_read_4bit_kernel<T><<<grid, kThreads, 0, st>>>(a, tb);
  else if (a.cache_dtype == ULYSSES_E4M3) cache_read_kernel<T, kE4m3><<<grid, kThreads, 0, st>>>(a, tb);
  else cache_read_kernel<T, kAsIs><<<grid, kThreads, 0, st>>>(a, tb);
}

}  // namespace

int launch_cache_write(const CacheArgs& a, cudaStream_t st) {
  const int tb = tokens_per_cta(a, a.cache_dtype == ULYSSES_E2M1 ? 16 : 8);
  const unsigned grid = (unsigned)((a.T + tb - 1) / tb);
  if (a.dtype == ULYSSES_BF16) a.w ? write_rows<__nv_bfloat16, true>(a, grid, tb, st) : write_rows<__nv_bfloat16, false>(a, grid, tb, st);
  else a.w ? write_rows<float, true>(a, grid, tb, st) : write_rows<float, false>(a, grid, tb, st);
  count_launch();
  return check_launch("cache_write");
}

int launch_cache_read(const CacheArgs& a, cudaStream_t st) {
  const int tb = tokens_per_cta(a);
  const unsigned grid = (unsigned)((a.T + tb - 1) / tb);
  if (a.dtype == ULYSSES_BF16) read_rows<__nv_bfloat16>(a, grid, tb, st);
  else read_rows<float>(a, grid, tb, st);
  count_launch();
  return check_launch("cache_read");
}

}  // namespace ulysses
