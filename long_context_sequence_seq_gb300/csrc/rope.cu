// Rotary positions on several axes, forward and adjoint (include/ulysses.h,
// ulysses_rope_fwd / ulysses_rope_bwd).
//
//   (y1, y2) = (x1 cos a - x2 sin a, x1 sin a + x2 cos a),  a = pos * freq
//
// The angle of a far position needs more than fp32: at position 2^20 an fp32
// product is off by 0.06 rad.  Here it is a turn in 64-bit fixed point: freq is
// held as f / 2 pi * 2^64 (an integer, right to a unit), the product with the integer
// position is taken mod 2^64, which drops whole turns exactly, and the top 32
// bits are the turn in [-1/2, 1/2): two integer multiplies, no fp64 (which this
// GPU runs at 1/60 of its fp32 rate).  sincospif of that turn is off by at most
// ~2e-7.
//
// Bound by HBM: every row is read and written once.  A CTA takes TB tokens and
// a range of heads: it forms the tokens' TB * rot/2 sines and cosines once in
// shared memory, then streams the heads' rows; a thread moves two 8-element
// words, the two halves of 8 pairs.  Measured: fp32 gradients of 65536 tokens x
// 40 heads of 128 to bf16 292 us (2.01 GB, 103% of the measured copy rate);
// bf16, 17100 tokens 61 us (350 MB, 86%: 3.5 waves of CTAs, each waiting for
// its angles first).
#include "internal.h"
#include "rows.cuh"

namespace ulysses {

ULYSSES_ERROR_READER(read_error_rope)

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 64;     // of a CTA
constexpr int kMaxAngles = 2048;   // tokens x pairs of a CTA

// 64 bytes of loads in flight a thread, and the CTAs an SM holds of it: fewer
// or more of either lose (a video's 17100 tokens, at half this block size: 65 us; one row and 5 CTAs 70,
// four rows and 2 CTAs 81, two rows and 5 CTAs, with spills, 89; fp32 gradients
// of 65536: 294 us; 4 CTAs 302, two rows and 2 CTAs 355).
template <typename Tin> constexpr int kRows = sizeof(Tin) == 2 ? 2 : 1;
template <typename Tin> constexpr int kCtas = sizeof(Tin) == 2 ? 4 : 5;

template <typename Tin, typename Tout>
__global__ void __launch_bounds__(kThreads, kCtas<Tin>) rope_kernel(const __grid_constant__ RopeArgs a, int tb, int heads_cta) {
  using namespace rows;
  __shared__ __align__(16) float cos_s[kMaxAngles];
  __shared__ __align__(16) float sin_s[kMaxAngles];
  const int64_t n0 = (int64_t)blockIdx.x * tb;
  const int tokens = (int)(a.N - n0 < tb ? a.N - n0 : tb);
  const int half = a.half;
  const int h0 = blockIdx.y * heads_cta;
  const int hn = a.heads - h0 < heads_cta ? a.heads - h0 : heads_cta;
  const int chunks = a.D / 16, c = threadIdx.x % chunks;
  const bool turned = c < half / 8;
  // the two words of this thread: 8 pairs, or 16 elements that are copied
  const int oa = (turned && a.pairs == ULYSSES_PAIRS_HALF) ? 8 * c : 16 * c;
  const int ob = (turned && a.pairs == ULYSSES_PAIRS_HALF) ? half + 8 * c : 16 * c + 8;
  // rows that lie together in memory are neighbours
  const int ni = a.heads_fast ? hn : tokens, no = a.heads_fast ? tokens : hn;
  RowWalk walk(threadIdx.x / chunks, kThreads / chunks, ni);
  constexpr int R = kRows<Tin>;
  Row8<Tin> wa[R], wb[R];
  Tout* dst[R];
  int tok[R];
  auto load = [&]() {
#pragma unroll
    for (int u = 0; u < R; ++u) {
      dst[u] = nullptr;
      if (walk.o >= no) continue;
      const int t = a.heads_fast ? walk.o : walk.i, h = h0 + (a.heads_fast ? walk.i : walk.o);
      int j = 0;
#pragma unroll
      for (int k = 1; k < kMaxRopeItems; ++k)
        if (k < a.njobs && h >= a.job[k].head0) j = k;
      const RopeJob& jb = a.job[j];
      const int64_t n = n0 + t;
      // one division of 64 bits only where there is more than one batch entry
      const int64_t b = a.S == a.N ? 0 : n / a.S, s = n - b * a.S;
      const int64_t si = b * jb.src_b + s * jb.src_s + (int64_t)(h - jb.head0) * jb.src_h;
      const int64_t di = b * jb.dst_b + s * jb.dst_s + (int64_t)(h - jb.head0) * jb.dst_h;
      if (in_bounds(si + ob + 7, jb.src_n) && in_bounds(di + ob + 7, jb.dst_n)) {
        const Tin* src = reinterpret_cast<const Tin*>(jb.src) + si;
        wa[u].load(src + oa);
        wb[u].load(src + ob);
        dst[u] = reinterpret_cast<Tout*>(jb.dst) + di;
        tok[u] = t;
      }
      walk.next();
    }
  };
  // fp32: the first rows are on their way while the angles are formed (302 ->
  // 291 us); bf16 has no registers left for that (61 us, 66 with spills)
  constexpr bool kAhead = sizeof(Tin) == 4;
  bool more = false;
  if (kAhead) {
    more = walk.o < no;
    load();
  }
  // a thread forms one pair's angles, for every fourth token
  if (const int p = threadIdx.x % kMaxRopePairs; p < half) {
    const uint64_t freq = a.freq[p];
    const int32_t* pos = a.pos + (int64_t)a.axis[p] * a.N + n0;
    for (int t = threadIdx.x / kMaxRopePairs; t < tokens; t += kThreads / kMaxRopePairs) {
      const uint64_t turn = (uint64_t)(int64_t)__ldg(pos + t) * freq;
      float s, co;
      sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &co);   // half turns: * 2^-31
      cos_s[t * half + p] = co;
      sin_s[t * half + p] = a.inverse ? -s : s;
    }
  }
  __syncthreads();
  while (kAhead ? more : walk.o < no) {
    if (!kAhead) load();
#pragma unroll
    for (int u = 0; u < R; ++u) {
      if (dst[u] == nullptr) continue;
      float x[16];
      wa[u].get(x);
      wb[u].get(x + 8);
      if (turned) {
        const float4* cp = reinterpret_cast<const float4*>(cos_s + tok[u] * half + 8 * c);
        const float4* sp = reinterpret_cast<const float4*>(sin_s + tok[u] * half + 8 * c);
        const float4 c0 = cp[0], c1 = cp[1], s0 = sp[0], s1 = sp[1];
        const float cs[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
        const float sn[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // half pairs: (x[i], x[i + 8]); adjacent pairs: (x[2i], x[2i + 1])
          if (a.pairs == ULYSSES_PAIRS_HALF) {
            const float p = x[i], q = x[i + 8];
            x[i] = p * cs[i] - q * sn[i];
            x[i + 8] = p * sn[i] + q * cs[i];
          } else {
            const float p = x[2 * i], q = x[2 * i + 1];
            x[2 * i] = p * cs[i] - q * sn[i];
            x[2 * i + 1] = p * sn[i] + q * cs[i];
          }
        }
      }
      Row8<Tout> ya, yb;
      ya.set(x);
      yb.set(x + 8);
      ya.store(dst[u] + oa);
      yb.store(dst[u] + ob);
    }
    if (kAhead) {
      more = walk.o < no;
      load();
    }
  }
}

}  // namespace

int launch_rope(const RopeArgs& a, cudaStream_t st) {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // tokens of a CTA: 256 bytes a thread, so that the angles' latency is small
  // beside them, and no more, so that the last wave is short
  const int need = (a.dtype == ULYSSES_BF16 ? 8 : 4) * kThreads;
  int tb = 1;
  while (tb < kMaxTokens && 2 * tb * a.half <= kMaxAngles && (int64_t)tb * a.heads * (a.D / 16) < need) tb *= 2;
  while (tb > 1 && (a.N + tb - 1) / tb < 2 * sms) tb /= 2;
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
