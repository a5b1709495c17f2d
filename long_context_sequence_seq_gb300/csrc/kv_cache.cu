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

// x / y to nearest, given 1 / y to nearest (a quotient's residual is exact in an
// FMA, and one step with it rounds correctly: Markstein 1990).  Codes next to a
// border are then those of the definition, in 64 bits too.
__device__ __forceinline__ float divided(float x, float y, float inv_y) {
  const float q = x * inv_y;
  return fmaf(fmaf(-q, y, x), inv_y, q);
}

// The codes of a word of a 4-bit row, whose block scale is b (0: all of it is
// below half of the smallest scale).  up: the inverse of the row's scale, a power
// of two.
template <typename T>
__device__ __forceinline__ uint32_t to_e2m1(const Row8<T>& w, float up, float b) {
  const float r = 1.0f / b;
  float f[8];
  w.get(f);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = b > 0.f ? divided(f[i] * up, b, r) : 0.f;
  return f32_to_e2m1x8(f);
}

// The rows of a CTA's tokens x heads, K's and then V's, in an order in which
// rows that lie together in the tokens' tensor are neighbours: heads of one
// token where those are closer, else tokens of one head.
// Rows that a lane has in work at once: 64 bytes of loads or more in flight.
// A lane holds 16 elements of a row, the 8-element words lane and lane + D / 16.
template <typename T, Held kHeld, bool kWrite>
constexpr int rows_in_work() { return kWrite ? (sizeof(T) == 2 ? 4 : 2) : (kHeld != kAsIs ? 4 : (sizeof(T) == 2 ? 2 : 1)); }

template <typename T, Held kHeld>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const __grid_constant__ CacheArgs a, int tb) {
  __shared__ int64_t place[kMaxTokens];
  __shared__ int slots[kMaxTokens];
  const int64_t t0 = (int64_t)blockIdx.x * tb;
  const int tokens = (int)(a.T - t0 < tb ? a.T - t0 : tb);
  check_cu(a);
  if ((int)threadIdx.x < tokens) {
    int slot = 0;
    place[threadIdx.x] = place_of(a, t0 + threadIdx.x, true, slot);
    slots[threadIdx.x] = slot;
  }
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
    int slot[kRows];
    bool second[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      row[u] = -1;
      slot[u] = 0;
      w[u][0].zero();
      w[u][1].zero();
      second[u] = walk.o >= no;
      if (walk.o < 2 * no) {
        const int o = second[u] ? walk.o - no : walk.o;
        const int t = heads_fast ? o : walk.i, h = heads_fast ? walk.i : o;
        const int64_t at = place[t];
        if (at >= 0 && in_bounds(at + (int64_t)h * a.page, a.num_pages * a.H * a.page)) {
          row[u] = at + (int64_t)h * a.page;
          if (kHeld == kE2m1) slot[u] = slots[t];
          if (a.w && lane == 0 && !second[u]) a.w[row[u]] = 0.f;
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
    float block[kRows][2];                       // 4 bits: largest magnitudes of the words' blocks
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      float a0 = w[u][0].amax(), a1 = w[u][1].amax();
      if (kHeld == kE2m1) {                      // a block is the words of a pair of lanes
        block[u][0] = a0 = max_nan(a0, __shfl_xor_sync(0xffffffffu, a0, 1));
        block[u][1] = a1 = max_nan(a1, __shfl_xor_sync(0xffffffffu, a1, 1));
      }
      float amax = max_nan(a0, a1);
      for (int o = lanes / 2; o > (kHeld == kE2m1 ? 1 : 0); o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      mine = lane % kRows == u ? amax : mine;
    }
    // so one pair of divisions serves kRows rows
    mine = max_nan(mine, 7.888609052210118e-31f);   // 2^-100
    float inv = 448.0f / mine, scale = mine / 448.0f;
    if (kHeld == kE2m1) {
      // 2688 is 1.3125 * 2^11: the exponent that takes mine to (1344, 2688]
      const uint32_t e = (__float_as_uint(mine) + 0x57ffffu >> 23) - 11;
      scale = __uint_as_float(e << 23);
      inv = __uint_as_float((254 - e) << 23);
    }
    if (!(mine <= 3.4028234663852886e38f)) scale = __int_as_float(0x7fc00000);
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const float by = __shfl_sync(0xffffffffu, inv, u, lanes);
      if (kHeld == kE2m1) {
        const uint16_t b2 = f32_to_e4m3x2(divided(block[u][0] * by, 6.0f, 1.0f / 6.0f), divided(block[u][1] * by, 6.0f, 1.0f / 6.0f));
        const uint32_t bh = e4m3x2_to_f16x2(b2);
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&bh));
        const uint32_t c0 = to_e2m1(w[u][0], by, b.x), c1 = to_e2m1(w[u][1], by, b.y);
        if (row[u] < 0) continue;
        uint8_t* base = reinterpret_cast<uint8_t*>(second[u] ? a.vc : a.kc);
        uint32_t* dst = reinterpret_cast<uint32_t*>(base + e2m1_codes(row[u], slot[u], a.D));
        dst[lane] = c0;
        dst[lane + lanes] = c1;
        if ((lane & 1) == 0) {
          uint8_t* bs = base + e2m1_blocks(row[u], slot[u], a.page, a.D) + lane / 2;
          bs[0] = (uint8_t)b2;
          bs[lanes / 2] = (uint8_t)(b2 >> 8);
        }
        if (lane == u) (second[u] ? a.vs : a.ks)[row[u]] = scale;
        continue;
      }
      const uint2 c0 = w[u][0].codes(by), c1 = w[u][1].codes(by);
      if (row[u] < 0) continue;
      uint8_t* dst = reinterpret_cast<uint8_t*>(second[u] ? a.vc : a.kc) + row[u] * a.D;
      st8(dst + e0, c0);
      st8(dst + e1, c1);
      if (lane == u) (second[u] ? a.vs : a.ks)[row[u]] = scale;
    }
  }
}

template <typename T, Held kHeld>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ CacheArgs a, int tb) {
  __shared__ int64_t place[kMaxTokens];
  __shared__ int slots[kMaxTokens];
  const int64_t t0 = (int64_t)blockIdx.x * tb;
  const int tokens = (int)(a.T - t0 < tb ? a.T - t0 : tb);
  check_cu(a);
  if ((int)threadIdx.x < tokens) {
    int slot = 0;
    place[threadIdx.x] = place_of(a, t0 + threadIdx.x, false, slot);
    slots[threadIdx.x] = slot;
  }
  __syncthreads();
  constexpr int kRows = rows_in_work<T, kHeld, false>();
  const int lanes = a.D / 16, lane = threadIdx.x % lanes, e0 = lane * 8, e1 = (lane + lanes) * 8;
  const bool heads_fast = a.k_h <= a.k_s;
  const int ni = heads_fast ? a.H : tokens, no = heads_fast ? tokens : a.H;
  RowWalk walk(threadIdx.x / lanes, kThreads / lanes, ni);
  while (walk.o < 2 * no) {
    Row8<T> w[kRows][2];
    uint2 codes[kRows][2];                       // 4 bits: a word's codes and its block's scale
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
          if (kHeld == kE2m1) {
            const uint8_t* base = reinterpret_cast<const uint8_t*>(second ? a.vc : a.kc);
            const uint32_t* src = reinterpret_cast<const uint32_t*>(base + e2m1_codes(row, slots[t], a.D));
            const uint8_t* bs = base + e2m1_blocks(row, slots[t], a.page, a.D) + lane / 2;
            codes[u][0] = make_uint2(__ldg(src + lane), __ldg(bs));
            codes[u][1] = make_uint2(__ldg(src + lane + lanes), __ldg(bs + lanes / 2));
            scale[u] = __ldg((second ? a.vs : a.ks) + row);
          } else if (kHeld == kE4m3) {
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
        if (kHeld != kAsIs) {
          float f[8];
          if (kHeld == kE2m1) {
            uint32_t h[4];
            e2m1x8_to_f16x2(codes[u][x].x, h);
            const uint32_t b = e4m3x2_to_f16x2((uint16_t)(codes[u][x].y * 0x101u));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t p = hmul2(h[i], b);           // exact: 2 + 4 significant bits, in f16's range
              const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&p));
              f[2 * i] = v.x;
              f[2 * i + 1] = v.y;
            }
          } else {
            e4m3x4_to_f32(codes[u][x].x, f);
            e4m3x4_to_f32(codes[u][x].y, f + 4);
          }
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
int tokens_per_cta(const CacheArgs& a) {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  int tb = 1;
  while (tb < kMaxTokens && 2 * tb * a.H * (a.D / 16) < 8 * kThreads) tb *= 2;
  while (tb > 1 && (a.T + tb - 1) / tb < sms) tb /= 2;
  return tb;
}

}  // namespace

namespace {

template <typename T>
void write_rows(const CacheArgs& a, unsigned grid, int tb, cudaStream_t st) {
  if (a.cache_dtype == ULYSSES_E2M1) cache_write_kernel<T, kE2m1><<<grid, kThreads, 0, st>>>(a, tb);
  else if (a.cache_dtype == ULYSSES_E4M3) cache_write_kernel<T, kE4m3><<<grid, kThreads, 0, st>>>(a, tb);
  else cache_write_kernel<T, kAsIs><<<grid, kThreads, 0, st>>>(a, tb);
}
template <typename T>
void read_rows(const CacheArgs& a, unsigned grid, int tb, cudaStream_t st) {
  if (a.cache_dtype == ULYSSES_E2M1) cache_read_kernel<T, kE2m1><<<grid, kThreads, 0, st>>>(a, tb);
  else if (a.cache_dtype == ULYSSES_E4M3) cache_read_kernel<T, kE4m3><<<grid, kThreads, 0, st>>>(a, tb);
  else cache_read_kernel<T, kAsIs><<<grid, kThreads, 0, st>>>(a, tb);
}

}  // namespace

int launch_cache_write(const CacheArgs& a, cudaStream_t st) {
  const int tb = tokens_per_cta(a);
  const unsigned grid = (unsigned)((a.T + tb - 1) / tb);
  if (a.dtype == ULYSSES_BF16) write_rows<__nv_bfloat16>(a, grid, tb, st);
  else write_rows<float>(a, grid, tb, st);
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
