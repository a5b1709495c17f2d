// Rotary positions on several axes, forward and adjoint (include/ulysses.h,
// ulysses_rope_fwd / ulysses_rope_bwd).
//
//   (y1, y2) = (x1 cos a - x2 sin a, x1 sin a + x2 cos a),  a = pos * freq
//
// The angle of a far position needs more than fp32: at position 2^20 an fp32
// product is off by 0.06 rad.  Here it is a turn in 64-bit fixed point: freq is
// held as round(f / 2 pi * 2^64), the product with the integer position is
// taken mod 2^64, which drops whole turns exactly, and the top 32 bits are the
// turn in [-1/2, 1/2): two integer multiplies, no fp64 (which this GPU runs at
// 1/60 of its fp32 rate).  sincospif of that turn is off by at most ~1e-7.
//
// Bound by HBM: every row is read and written once.  A CTA takes TB tokens and
// a range of heads: it forms the tokens' TB * rot/2 sines and cosines once in
// shared memory, then streams the heads' rows; a thread moves two 8-element
// words, the two halves of 8 pairs.
#include "internal.h"
#include "rows.cuh"

namespace ulysses {

ULYSSES_ERROR_READER(read_error_rope)

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;   // tokens of one CTA

template <typename Tin, typename Tout>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a, int tb, int heads_cta) {
  using namespace rows;
  __shared__ __align__(16) float cos_s[kMaxTokens * kMaxRopePairs];
  __shared__ __align__(16) float sin_s[kMaxTokens * kMaxRopePairs];
  const int64_t n0 = (int64_t)blockIdx.x * tb;
  const int tokens = (int)(a.N - n0 < tb ? a.N - n0 : tb);
  const int half = a.half;
  for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
    const int t = i / half, p = i - t * half;
    const int32_t pos = __ldg(a.pos + (int64_t)a.axis[p] * a.N + n0 + t);
    const uint64_t turn = (uint64_t)(int64_t)pos * a.freq[p];
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &c);   // half turns: * 2^-31
    cos_s[i] = c;
    sin_s[i] = a.inverse ? -s : s;
  }
  __syncthreads();
  const int h0 = blockIdx.y * heads_cta;
  const int hn = a.heads - h0 < heads_cta ? a.heads - h0 : heads_cta;
  const int chunks = a.D / 16, c = threadIdx.x % chunks;
  const bool turned = c < half / 8;
  // the two words of this thread: 8 pairs, or 16 elements that are copied
  const int oa = (turned && a.pairs == ULYSSES_PAIRS_HALF) ? 8 * c : 16 * c;
  const int ob = (turned && a.pairs == ULYSSES_PAIRS_HALF) ? half + 8 * c : 16 * c + 8;
  for (int r = threadIdx.x / chunks; r < tokens * hn; r += kThreads / chunks) {
    int t, h;
    if (a.heads_fast) { t = r / hn; h = r - t * hn; } else { h = r / tokens; t = r - h * tokens; }
    h += h0;
    int j = 0;
#pragma unroll
    for (int k = 1; k < kMaxRopeItems; ++k)
      if (k < a.njobs && h >= a.job[k].head0) j = k;
    const RopeJob& jb = a.job[j];
    const int64_t n = n0 + t, b = n / a.S, s = n - b * a.S;
    const int64_t si = b * jb.src_b + s * jb.src_s + (int64_t)(h - jb.head0) * jb.src_h;
    const int64_t di = b * jb.dst_b + s * jb.dst_s + (int64_t)(h - jb.head0) * jb.dst_h;
    if (!in_bounds(si + ob + 7, jb.src_n) || !in_bounds(di + ob + 7, jb.dst_n)) continue;
    const Tin* src = reinterpret_cast<const Tin*>(jb.src) + si;
    Tout* dst = reinterpret_cast<Tout*>(jb.dst) + di;
    Row8<Tin> wa, wb;
    wa.load(src + oa);
    wb.load(src + ob);
    float x[16];
    wa.get(x);
    wb.get(x + 8);
    if (turned) {
      const float4* cp = reinterpret_cast<const float4*>(cos_s + t * half + 8 * c);
      const float4* sp = reinterpret_cast<const float4*>(sin_s + t * half + 8 * c);
      const float4 c0 = cp[0], c1 = cp[1], s0 = sp[0], s1 = sp[1];
      const float cs[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
      const float sn[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // half pairs: (x[i], x[i + 8]); adjacent pairs: (x[2i], x[2i + 1])
        if (a.pairs == ULYSSES_PAIRS_HALF) {
          const float u = x[i], v = x[i + 8];
          x[i] = u * cs[i] - v * sn[i];
          x[i + 8] = u * sn[i] + v * cs[i];
        } else {
          const float u = x[2 * i], v = x[2 * i + 1];
          x[2 * i] = u * cs[i] - v * sn[i];
          x[2 * i + 1] = u * sn[i] + v * cs[i];
        }
      }
    }
    Row8<Tout> ya, yb;
    ya.set(x);
    yb.set(x + 8);
    ya.store(dst + oa);
    yb.store(dst + ob);
  }
}

}  // namespace

int launch_rope(const RopeArgs& a, cudaStream_t st) {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  int tb = kMaxTokens;
  while (tb > 1 && (a.N + tb - 1) / tb < 4 * sms) tb /= 2;
  const int64_t gx = (a.N + tb - 1) / tb;
  // few tokens: split the heads too, down to 8 heads (one round of the CTA's threads or two)
  int hc = a.heads;
  while (hc > 8 && gx * ((a.heads + hc - 1) / hc) < sms) hc = (hc + 1) / 2;
  const dim3 grid((unsigned)gx, (unsigned)((a.heads + hc - 1) / hc));
  if (a.dtype == ULYSSES_BF16)
    rope_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, kThreads, 0, st>>>(a, tb, hc);
  else if (a.out_dtype == ULYSSES_FP32)
    rope_kernel<float, float><<<grid, kThreads, 0, st>>>(a, tb, hc);
  else
    rope_kernel<float, __nv_bfloat16><<<grid, kThreads, 0, st>>>(a, tb, hc);
  count_launch();
  return check_launch("rope");
}

}  // namespace ulysses
