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
__device__ __forceinline__ int64_t place_of(const CacheArgs& a, int64_t t, bool write) {
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
  return (int64_t)pg * a.H * a.page + (pos - (int64_t)col * a.page);
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
template <typename T, bool kQuant, bool kWrite>
constexpr int rows_in_work() { return kWrite ? (sizeof(T) == 2 ? 4 : 2) : (kQuant ? 4 : (sizeof(T) == 2 ? 2 : 1)); }

template <typename T, bool kQuant>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const __grid_constant__ CacheArgs a, int tb) {
  __shared__ int64_t place[kMaxTokens];
  const int64_t t0 = (int64_t)blockIdx.x * tb;
  const int tokens = (int)(a.T - t0 < tb ? a.T - t0 : tb);
  check_cu(a);
  if ((int)threadIdx.x < tokens) place[threadIdx.x] = place_of(a, t0 + threadIdx.x, true);
  __syncthreads();
  constexpr int kRows = rows_in_work<T, kQuant, true>();
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
          const int64_t off = second[u] ? (t0 + t) * a.v_s + h * a.v_h : (t0 + t) * a.k_s + h * a.k_h;
          const T* src = reinterpret_cast<const T*>(second[u] ? a.v : a.k) + off;
          w[u][0].load(src + e0);
          w[u][1].load(src + e1);
        }
      }
      walk.next();
    }
    if (!kQuant) {
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

template <typename T, bool kQuant>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ CacheArgs a, int tb) {
  __shared__ int64_t place[kMaxTokens];
  const int64_t t0 = (int64_t)blockIdx.x * tb;
  const int tokens = (int)(a.T - t0 < tb ? a.T - t0 : tb);
  check_cu(a);
  if ((int)threadIdx.x < tokens) place[threadIdx.x] = place_of(a, t0 + threadIdx.x, false);
  __syncthreads();
  constexpr int kRows = rows_in_work<T, kQuant, false>();
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
          if (kQuant) {
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
        if (kQuant) {
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

int launch_cache_write(const CacheArgs& a, cudaStream_t st) {
  const int tb = tokens_per_cta(a);
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
  const int tb = tokens_per_cta(a);
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
