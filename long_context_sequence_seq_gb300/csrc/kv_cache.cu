// The paged key-value cache: writing new tokens' rows, as they are or in
// 8 bits, and gathering them back (include/ulysses.h, ulysses_cache_write /
// ulysses_cache_read).
//
//   amax = max(max_d |x_d|, 2^-100), scale = amax / 448, code_d = e4m3(x_d * (448 / amax))
//
// 448 is e4m3's largest value, so no code saturates; the floor keeps the
// reciprocal finite for rows of zeros and of the smallest subnormals.  One
// scale per row (token, head) is 3% of a 128-byte row and lets a row be
// written without reading any other.
//
// Bound by HBM: rows are read and written once.  A CTA takes a block of tokens
// with all their heads, K and V: it resolves each token's place once (sequence
// by bisection in cu, page from the table) and streams the rows; D / 8 lanes
// hold a row, 8 elements each, so the row's largest magnitude is a 3- or
// 4-step shuffle.
#include "internal.h"
#include "rows.cuh"

namespace ulysses {

ULYSSES_ERROR_READER(read_error_kv_cache)

namespace {

using namespace rows;

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;

// Row of the caches ([num_pages][H][page] rows, before the head's offset) of
// token t, or -1: nothing to do (past the last sequence, an empty place of the
// batch) or outside the table (reported).  write: a.lens are the lengths with
// the new tokens; read: the first positions (may be NULL).
__device__ __forceinline__ int64_t place_of(const CacheArgs& a, int64_t t, bool write) {
  int b = (int)t;
  int64_t pos;
  if (a.cu) {
    b = doc_of(a.cu, a.B, t);
    const int64_t lo = __ldg(a.cu + b), hi = __ldg(a.cu + b + 1);
    if (t < lo || t >= hi) return -1;
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
  return (int64_t)pg * a.H * a.page + (pos - (int64_t)col * a.page);
}

// cu[0] == 0, non-decreasing, cu[B] <= T; checked by the first CTA.
__device__ __forceinline__ void check_cu(const CacheArgs& a) {
  if (blockIdx.x != 0 || !a.cu) return;
  for (int i = threadIdx.x; i <= a.B; i += kThreads) {
    const int c = __ldg(a.cu + i);
    if ((i == 0 && c != 0) || (i > 0 && c < __ldg(a.cu + i - 1)) || (i == a.B && c > a.T)) raise_error(kErrSeqlens);
  }
}

__device__ __forceinline__ float max_nan(float x, float y) {   // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

// Row r of the CTA's tokens x heads x {K, V}: which token, head and tensor.
// Rows that lie together in memory are neighbours: heads of one token when the
// tokens' tensor has them closer, else tokens of one head.
struct RowIndex { int t, h, v; };
__device__ __forceinline__ RowIndex row_index(int r, int tokens, int heads, bool heads_fast) {
  const int per = tokens * heads;
  RowIndex x;
  x.v = r >= per;
  r -= x.v ? per : 0;
  if (heads_fast) { x.t = r / heads; x.h = r - x.t * heads; } else { x.h = r / tokens; x.t = r - x.h * tokens; }
  return x;
}

template <typename T, bool kQuant>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const __grid_constant__ CacheArgs a, int tb) {
  __shared__ int64_t place[kMaxTokens];
  const int64_t t0 = (int64_t)blockIdx.x * tb;
  const int tokens = (int)(a.T - t0 < tb ? a.T - t0 : tb);
  check_cu(a);
  if ((int)threadIdx.x < tokens) place[threadIdx.x] = place_of(a, t0 + threadIdx.x, true);
  __syncthreads();
  const int lanes = a.D / 8, lane = threadIdx.x % lanes;
  const bool heads_fast = a.k_h <= a.k_s;
  const int rows = 2 * tokens * a.H, step = kThreads / lanes;
  // every lane of a warp runs the same number of rounds: the row maximum is a shuffle
  for (int r0 = 0; r0 < rows; r0 += step) {
    const int r = r0 + threadIdx.x / lanes;
    const RowIndex x = row_index(r < rows ? r : 0, tokens, a.H, heads_fast);
    const int64_t at = place[x.t];
    const bool live = r < rows && at >= 0;
    const int64_t row = at + (int64_t)x.h * a.page;
    Row8<T> w;
    w.set((const float[8]){0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f});
    if (live)
      w.load(reinterpret_cast<const T*>(x.v ? a.v : a.k) + (t0 + x.t) * (x.v ? a.v_s : a.k_s) +
             x.h * (x.v ? a.v_h : a.k_h) + lane * 8);
    const bool ok = live && in_bounds(row, a.num_pages * a.H * a.page);
    if (!kQuant) {
      if (ok) w.store(reinterpret_cast<T*>(x.v ? a.vc : a.kc) + row * a.D + lane * 8);
    } else {
      float f[8];
      w.get(f);
      float amax = fabsf(f[0]);
#pragma unroll
      for (int i = 1; i < 8; ++i) amax = max_nan(amax, fabsf(f[i]));
      for (int o = lanes / 2; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      amax = max_nan(amax, 7.888609052210118e-31f);   // 2^-100
      const float inv = 448.0f / amax;
      const float scale = amax <= 3.4028234663852886e38f ? amax / 448.0f : __int_as_float(0x7fc00000);
      uint2 codes;
      codes.x = f32_to_e4m3x2(f[0] * inv, f[1] * inv) | (uint32_t)f32_to_e4m3x2(f[2] * inv, f[3] * inv) << 16;
      codes.y = f32_to_e4m3x2(f[4] * inv, f[5] * inv) | (uint32_t)f32_to_e4m3x2(f[6] * inv, f[7] * inv) << 16;
      if (ok) {
        st8(reinterpret_cast<uint8_t*>(x.v ? a.vc : a.kc) + row * a.D + lane * 8, codes);
        if (lane == 0) (x.v ? a.vs : a.ks)[row] = scale;
      }
    }
  }
}

template <typename T, bool kQuant>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ CacheArgs a, int tb) {
  __shared__ int64_t place[kMaxTokens];
  const int64_t t0 = (int64_t)blockIdx.x * tb;
  const int tokens = (int)(a.T - t0 < tb ? a.T - t0 : tb);
  check_cu(a);
  if ((int)threadIdx.x < tokens) place[threadIdx.x] = place_of(a, t0 + threadIdx.x, false);
  __syncthreads();
  const int lanes = a.D / 8, lane = threadIdx.x % lanes;
  const bool heads_fast = a.k_h <= a.k_s;
  for (int r = threadIdx.x / lanes; r < 2 * tokens * a.H; r += kThreads / lanes) {
    const RowIndex x = row_index(r, tokens, a.H, heads_fast);
    const int64_t at = place[x.t];
    if (at < 0) continue;
    const int64_t row = at + (int64_t)x.h * a.page;
    if (!in_bounds(row, a.num_pages * a.H * a.page)) continue;
    T* dst = reinterpret_cast<T*>(x.v ? a.v : a.k) + (t0 + x.t) * (x.v ? a.v_s : a.k_s) + x.h * (x.v ? a.v_h : a.k_h) + lane * 8;
    Row8<T> w;
    if (!kQuant) {
      w.load(reinterpret_cast<const T*>(x.v ? a.vc : a.kc) + row * a.D + lane * 8);
    } else {
      const uint2 codes = ld8(reinterpret_cast<const uint8_t*>(x.v ? a.vc : a.kc) + row * a.D + lane * 8);
      const float scale = (x.v ? a.vs : a.ks)[row];
      float f[8];
      e4m3x4_to_f32(codes.x, f);
      e4m3x4_to_f32(codes.y, f + 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= scale;
      w.set(f);
    }
    w.store(dst);
  }
}

// Tokens of one CTA: as many as leave every SM a few CTAs.
int tokens_per_cta(int64_t T) {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  int tb = kMaxTokens;
  while (tb > 1 && (T + tb - 1) / tb < 4 * sms) tb /= 2;
  return tb;
}

}  // namespace

int launch_cache_write(const CacheArgs& a, cudaStream_t st) {
  const int tb = tokens_per_cta(a.T);
  const unsigned grid = (unsigned)((a.T + tb - 1) / tb);
  const bool quant = a.cache_dtype == ULYSSES_E4M3;
  if (a.dtype == ULYSSES_BF16) {
    if (quant) cache_write_kernel<__nv_bfloat16, true><<<grid, kThreads, 0, st>>>(a, tb);
    else cache_write_kernel<__nv_bfloat16, false><<<grid, kThreads, 0, st>>>(a, tb);
  } else {
    if (quant) cache_write_kernel<float, true><<<grid, kThreads, 0, st>>>(a, tb);
    else cache_write_kernel<float, false><<<grid, kThreads, 0, st>>>(a, tb);
  }
  count_launch();
  return check_launch("cache_write");
}

int launch_cache_read(const CacheArgs& a, cudaStream_t st) {
  const int tb = tokens_per_cta(a.T);
  const unsigned grid = (unsigned)((a.T + tb - 1) / tb);
  const bool quant = a.cache_dtype == ULYSSES_E4M3;
  if (a.dtype == ULYSSES_BF16) {
    if (quant) cache_read_kernel<__nv_bfloat16, true><<<grid, kThreads, 0, st>>>(a, tb);
    else cache_read_kernel<__nv_bfloat16, false><<<grid, kThreads, 0, st>>>(a, tb);
  } else {
    if (quant) cache_read_kernel<float, true><<<grid, kThreads, 0, st>>>(a, tb);
    else cache_read_kernel<float, false><<<grid, kThreads, 0, st>>>(a, tb);
  }
  count_launch();
  return check_launch("cache_read");
}

}  // namespace ulysses
