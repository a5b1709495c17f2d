// Attention of one new token per sequence over the paged cache
// (include/ulysses.h, ulysses_attn_decode).
//
//   s_j = scale * q . k_j,  o = sum_j softmax(s)_j v_j,  lse = log sum_j e^{s_j}
//
// in one pass with a running maximum m (base-2 exponents): a key with
// s > m + 8 moves m and rescales the sums, otherwise m stays, which is exact
// because o = acc / l and lse = m + log l hold for any m.
//
// SIMT kernel: one CTA per (sequence, kv head, up to HG of its query heads).
// A warp walks tiles of 16 keys (always inside one page); 8 lanes hold a key's
// row, so 4 keys are in work at a time, each group of 8 lanes with a running
// softmax of its own; groups and warps are joined at the end.
#include "internal.h"
#include "rows.cuh"

namespace ulysses {

ULYSSES_ERROR_READER(read_error_attn_decode)

namespace {

using namespace rows;

constexpr int kTile = 16;                       // keys of a tile
constexpr float kNoMax = -3.4028234663852886e38f;
constexpr float kLazy = 8.f;                    // a maximum moves when exceeded by 2^8
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWarps = 4;

// Keys of sequence b: its length, cut to what the table can hold.
__device__ __forceinline__ int length_of(const DecodeArgs& a, int b) {
  int64_t n = __ldg(a.lens + b);
  const int64_t most = (int64_t)a.cols * a.page;
  if (n < 0 || n > most) {
    raise_error(kErrPages);
    n = n < 0 ? 0 : most;
  }
  return (int)n;
}

// Row index ([num_pages][H_kv][page] rows) of key `key` of sequence b, kv head
// h; -1 (reported) for a page id out of range.  key is a multiple of kTile.
__device__ __forceinline__ int64_t tile_row(const DecodeArgs& a, int b, int h, int key) {
  const int col = key / a.page;
  const int pg = __ldg(a.table + (int64_t)b * a.cols + col);
  if (pg < 0 || pg >= a.num_pages) {
    raise_error(kErrPages);
    return -1;
  }
  return ((int64_t)pg * a.H_kv + h) * a.page + (key - col * a.page);
}

// ------------------------------------------------------------------ SIMT tiles

// One lane's part of a row: 8 lanes hold D values, lane i the 16-byte words
// i, i + 8, ...  (for 8-bit rows of 64 values: 8-byte words).
template <typename TC, int D> struct LaneRow;
template <int D> struct LaneRow<float, D> {
  static constexpr int kWords = D / 32;
  uint4 w[kWords];
  __device__ __forceinline__ void load(const float* p, int i) {
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = ld16(p + (k * 8 + i) * 4);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      f[4 * k] = __uint_as_float(w[k].x); f[4 * k + 1] = __uint_as_float(w[k].y);
      f[4 * k + 2] = __uint_as_float(w[k].z); f[4 * k + 3] = __uint_as_float(w[k].w);
    }
  }
  // first of the lane's element e (in the order of get)
  __device__ static __forceinline__ int element(int e, int i) { return ((e / 4) * 8 + i) * 4 + e % 4; }
};
template <int D> struct LaneRow<__nv_bfloat16, D> {
  static constexpr int kWords = D / 64;
  uint4 w[kWords];
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int i) {
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = ld16(p + (k * 8 + i) * 8);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      bf16x2_to_f32(w[k].x, f + 8 * k); bf16x2_to_f32(w[k].y, f + 8 * k + 2);
      bf16x2_to_f32(w[k].z, f + 8 * k + 4); bf16x2_to_f32(w[k].w, f + 8 * k + 6);
    }
  }
  __device__ static __forceinline__ int element(int e, int i) { return ((e / 8) * 8 + i) * 8 + e % 8; }
};
template <int D> struct LaneRow<uint8_t, D> {
  uint32_t w[D / 32];
  __device__ __forceinline__ void load(const uint8_t* p, int i) {
    if (D == 128) {
      const uint4 v = ld16(p + i * 16);
      w[0] = v.x; w[1] = v.y; w[D / 32 - 2] = v.z; w[D / 32 - 1] = v.w;
    } else {
      const uint2 v = ld8(p + i * 8);
      w[0] = v.x; w[1] = v.y;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < D / 32; ++k) w[k] = 0;
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int k = 0; k < D / 32; ++k) e4m3x4_to_f32(w[k], f + 4 * k);
  }
  __device__ static __forceinline__ int element(int e, int i) { return i * (D / 8) + e; }
};

template <typename TQ, typename TC, int D, int HG>
__global__ void __launch_bounds__(kWarps * 32) decode_simt_kernel(const __grid_constant__ DecodeArgs a) {
  constexpr bool kQuant = sizeof(TC) == 1;
  constexpr int E = D / 8;                      // elements of a row per lane
  const int groups = (a.G + HG - 1) / HG;
  const int gi = blockIdx.x % groups, h = (blockIdx.x / groups) % a.H_kv, b = blockIdx.x / groups / a.H_kv;
  const int g0 = gi * HG, gn = a.G - g0 < HG ? a.G - g0 : HG;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i = lane & 7, grp = lane >> 3;
  const int len = length_of(a, b);
  const int64_t total = a.num_pages * a.H_kv * a.page;

  float q[HG][E], acc[HG][E], m[HG], l[HG];
#pragma unroll
  for (int g = 0; g < HG; ++g) {
    m[g] = kNoMax;
    l[g] = 0.f;
    const int hq = h * a.G + g0 + (g < gn ? g : 0);
    const TQ* qp = reinterpret_cast<const TQ*>(a.q) + (int64_t)b * a.q_b + (int64_t)hq * a.q_h;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      q[g][e] = to_f32<TQ>(qp[LaneRow<TC, D>::element(e, i)]) * a.scale_log2;
      acc[g][e] = 0.f;
    }
  }
  for (int key0 = warp * kTile; key0 < len; key0 += kWarps * kTile) {
    const int64_t row0 = tile_row(a, b, h, key0);
    if (row0 < 0 || !in_bounds(row0 + kTile - 1, total)) continue;
#pragma unroll 2
    for (int k = grp; k < kTile; k += 4) {
      const bool live = key0 + k < len;
      const int64_t row = row0 + k;
      LaneRow<TC, D> kr, vr;
      kr.zero();
      vr.zero();
      float ks = 1.f, vs = 1.f;
      if (live) {
        kr.load(reinterpret_cast<const TC*>(a.kc) + row * D, i);
        vr.load(reinterpret_cast<const TC*>(a.vc) + row * D, i);
        if (kQuant) { ks = __ldg(a.ks + row); vs = __ldg(a.vs + row); }
      }
      float f[E], s[HG];
      kr.get(f);
#pragma unroll
      for (int g = 0; g < HG; ++g) {
        s[g] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s[g] = fmaf(q[g][e], f[e], s[g]);
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1)
#pragma unroll
        for (int g = 0; g < HG; ++g) s[g] += __shfl_xor_sync(0xffffffffu, s[g], o);
      vr.get(f);
#pragma unroll
      for (int g = 0; g < HG; ++g) {
        float t = kQuant ? s[g] * ks : s[g];
        t = live ? t : -INFINITY;
        if (t > m[g] + kLazy) {
          const float w = exp2f(m[g] - t);
          m[g] = t;
          l[g] *= w;
#pragma unroll
          for (int e = 0; e < E; ++e) acc[g][e] *= w;
        }
        const float p = exp2f(t - m[g]);
        l[g] += p;
        const float pv = kQuant ? p * vs : p;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[g][e] = fmaf(pv, f[e], acc[g][e]);
      }
    }
  }
  // join the four groups of the warp
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {
#pragma unroll
    for (int g = 0; g < HG; ++g) {
      const float mo = __shfl_xor_sync(0xffffffffu, m[g], o), lo = __shfl_xor_sync(0xffffffffu, l[g], o);
      const float mm = fmaxf(m[g], mo), wa = exp2f(m[g] - mm), wb = exp2f(mo - mm);
      m[g] = mm;
      l[g] = l[g] * wa + lo * wb;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float x = __shfl_xor_sync(0xffffffffu, acc[g][e], o);
        acc[g][e] = acc[g][e] * wa + x * wb;
      }
    }
  }
  // join the warps
  __shared__ float so[kWarps][HG][D], sm[kWarps][HG], sl[kWarps][HG];
  if (grp == 0) {
#pragma unroll
    for (int g = 0; g < HG; ++g) {
      if (i == 0) { sm[warp][g] = m[g]; sl[warp][g] = l[g]; }
#pragma unroll
      for (int e = 0; e < E; ++e) so[warp][g][LaneRow<TC, D>::element(e, i)] = acc[g][e];
    }
  }
  __syncthreads();
  for (int x = threadIdx.x; x < gn * D; x += kWarps * 32) {
    const int g = x / D, d = x - g * D;
    float mm = kNoMax, ll = 0.f, o = 0.f;
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm[w][g]);
    for (int w = 0; w < kWarps; ++w) {
      const float f = exp2f(sm[w][g] - mm);
      ll += sl[w][g] * f;
      o += so[w][g][d] * f;
    }
    const int hq = h * a.G + g0 + g;
    reinterpret_cast<TQ*>(a.o)[(int64_t)b * a.o_b + (int64_t)hq * a.o_h + d] = from_f32<TQ>(len == 0 ? 0.f : o / ll);
    if (d == 0 && a.lse) a.lse[(int64_t)b * a.H_q + hq] = len == 0 ? -INFINITY : (mm + log2f(ll)) * kLn2;
  }
}

template <typename TQ, typename TC, int D, int HG>
int run_simt(const DecodeArgs& a, cudaStream_t st) {
  const unsigned grid = (unsigned)(a.B * a.H_kv * ((a.G + HG - 1) / HG));
  decode_simt_kernel<TQ, TC, D, HG><<<grid, kWarps * 32, 0, st>>>(a);
  count_launch();
  return check_launch("attn_decode");
}
template <typename TQ, typename TC, int D>
int run_simt_g(const DecodeArgs& a, cudaStream_t st) {
  if (a.G == 1) return run_simt<TQ, TC, D, 1>(a, st);
  if (a.G == 2) return run_simt<TQ, TC, D, 2>(a, st);
  return run_simt<TQ, TC, D, 4>(a, st);
}
template <typename TQ, typename TC>
int run_simt_d(const DecodeArgs& a, cudaStream_t st) {
  return a.D == 128 ? run_simt_g<TQ, TC, 128>(a, st) : run_simt_g<TQ, TC, 64>(a, st);
}

}  // namespace

size_t decode_workspace(const DecodeArgs&) { return 0; }

int launch_decode(const DecodeArgs& a, bool simt, cudaStream_t st) {
  (void)simt;
  const bool quant = a.cache_dtype == ULYSSES_E4M3;
  if (a.dtype == ULYSSES_BF16)
    return quant ? run_simt_d<__nv_bfloat16, uint8_t>(a, st) : run_simt_d<__nv_bfloat16, __nv_bfloat16>(a, st);
  return quant ? run_simt_d<float, uint8_t>(a, st) : run_simt_d<float, float>(a, st);
}

}  // namespace ulysses
