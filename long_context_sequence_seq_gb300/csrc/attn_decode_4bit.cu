// Attention of one new token per sequence over a 4-bit paged cache: an engine of
// its own for bf16 queries, beside those of attn_decode.cuh for fp32 ones.
//
// A key's K and V are 152 bytes at D = 128, 13 flops a byte with 4 query heads a
// kv head, so the copy rate leaves 6.6 clocks of an SM for a key and kv head: 26
// warp instructions.  Most of those go into making f16 operands of the codes
// (conversion and block scale, 12 a key), so everything beside that is kept short.
//
// A unit's codes are one block of memory (1 KB of K, 1 KB of V), and so are its
// block scales: each warp copies them, 16 bytes a lane, into a ring of its own in
// shared memory, a step ahead; a step's rows need no registers until they are
// multiplied.  From there the operands are loaded as the matrix engine does from global
// memory: lane (g, j) has
//   K   of rows g and g + 8 the j-th quarter of the codes: one or two blocks
//   V   of rows 2j, 2j+1, 2j+8, 2j+9 the g-th eighth: a block, or half of one.
//       The codes of two rows are interleaved (two logical operations for eight
//       codes) before they are converted, so that pairs come out as operands
// (16-byte words change places within 128 bytes, so that neither load meets a
// bank twice).  code * block scale is exact in f16 (2 + 4 significant bits, 2^-10
// to 2688 or 0).  K's row scale multiplies the score, V's goes into the weight,
// which enters as an f16 value and its f16 rest (attn_decode.cuh).
//
// Up to 4 query heads (kTwice): each has two of the product's 8 columns.  A lane
// then works on one key of a unit (lanes j < 2 on key g, the others on g + 8)
// and the two exchange the weights' parts: half of the softmax's instructions.
//
// Measured, a million keys of 8 kv heads of 128 with 4 query heads each (1.28 GB,
// 188 us at the copy rate): 225 us, 84%; 64 ragged sequences of up to 32768, 0.62
// GB: 120 us.  Rows held in registers as in the matrix engine took 296 us, with
// the two points above 272, through shared memory 226.  What bounds it now are
// the pipes: 296 warp instructions a unit, of which a unit's 64 conversions, 64
// block scales and 16 products alone take 320 of the 520 clocks that it takes (the
// f16 products share the issue with the products of the matrix pipe, 8 clocks
// each).  Set aside: four CTAs an SM 231 us, three units a step 222 (but ragged
// batches and 8 heads a kv head slower), one unit a step 255, three steps in the
// ring 226, the next step's scores formed beside this one's sums 225.
#include "attn_decode.cuh"

namespace ulysses {

ULYSSES_ERROR_READER(read_error_attn_decode_4bit)

namespace {

__device__ __forceinline__ float log2_fast(float x) {   // of a normal number (row scales are at least 2^-111)
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(to), "l"(from) : "memory");
}
// `n` bytes, the rest zeros
__device__ __forceinline__ void copy16(uint32_t to, const void* from, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(to), "l"(from), "r"(n) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from, int n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" :: "r"(to), "l"(from), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the last N groups of this thread's copies have arrived
template <int N>
__device__ __forceinline__ void copies_arrived() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

template <int D, int NT, bool kTwice, bool kSeen_>
struct FourEngine {
  using TQ = __nv_bfloat16;
  static constexpr bool kSeen = kSeen_;
  static constexpr int kHeads = kTwice ? 4 : 8 * NT;
  static constexpr int kRowB = D / 2;                     // bytes of a row's codes
  static constexpr int kSub = 2;                          // units of a step
  static constexpr int kStages = 2;                       // steps in the ring
  static constexpr int kKR = D / 32, kVR = D / 64;        // registers of a row's codes per lane
  static constexpr int kX = kTwice ? 1 : 2;               // keys of a unit that a lane has the weights of
  static constexpr int kMT = D / 16;                      // M tiles of O^T
  // a unit in the ring: codes of K and of V, block scales of both, row scales of both, and how many keys it has
  static constexpr int kCodes = kUnit * kRowB, kBlocks = kUnit * D / 16;
  static constexpr int kAtBlocks = 2 * kCodes, kAtScales = kAtBlocks + 2 * kBlocks, kAtKeys = kAtScales + 2 * kUnit * 4;
  static constexpr int kUnitB = kAtKeys + 16;
  static constexpr int kRing = kStages * kSub * kUnitB;   // bytes of a warp

  uint32_t q[NT][D / 8];
  float acc[NT][kMT][4];
  float m[NT][2], l[NT][2], mw[NT][2], sc[NT][2];
  int lane, g, j;
  char* ring;

  __device__ __forceinline__ FourEngine(int lane_, char* ring_) : lane(lane_), g(lane_ >> 2), j(lane_ & 3), ring(ring_) {}

  __device__ __forceinline__ int key_of(int x) const { return kTwice ? g + 8 * (j >> 1) : g + 8 * x; }
  __device__ __forceinline__ int head_of(int t, int c) const { return kTwice ? 2 * (j & 1) + c : t * 8 + 2 * j + c; }

  __device__ __forceinline__ void begin(const DecodeArgs& a, const Piece& p) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int hl = kTwice ? g & 3 : t * 8 + g;
      const bool live = hl < p.gn;
      const TQ* qp = reinterpret_cast<const TQ*>(a.q) + (int64_t)p.b * a.q_b + (int64_t)(p.h * a.G + p.g0 + (live ? hl : 0)) * a.q_h +
                     j * (D / 4);
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        const uint4 v = live ? ld16(qp + x * 8) : make_uint4(0, 0, 0, 0);
        q[t][4 * x] = v.x; q[t][4 * x + 1] = v.y; q[t][4 * x + 2] = v.z; q[t][4 * x + 3] = v.w;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) { m[t][c] = kNoMax; l[t][c] = 0.f; mw[t][c] = kNoMax; sc[t][c] = a.scale_log2; }
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[t][i][c] = 0.f;
    }
  }
  // q to f16, its largest element at 2^14 to 2^15 (the scores' scale takes the power of two back)
  __device__ __forceinline__ void scale_q() {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float big = 0.f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        float e[2];
        bf16x2_to_f32(q[t][i], e);
        big = fmaxf(big, fmaxf(fabsf(e[0]), fabsf(e[1])));
      }
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      int e = (int)(__float_as_uint(big) >> 23) - 127;
      e = (e < -100 ? -100 : (e > 126 ? 126 : e)) - 14;
      const float down = __int_as_float((127 - e) << 23), up = __int_as_float((127 + e) << 23);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        float x[2];
        bf16x2_to_f32(q[t][i], x);
        q[t][i] = f32_to_f16x2(x[0] * down, x[1] * down);
      }
      // from head g's lanes to those that hold the scores of heads 2j, 2j + 1
      sc[t][0] *= __shfl_sync(0xffffffffu, up, 8 * j);
      sc[t][1] *= __shfl_sync(0xffffffffu, up, 8 * j + 4);
    }
  }

  // Offset of the 16-byte word `w` of a unit's codes in the ring: words change places within 128 bytes.
  __device__ __forceinline__ static int place(int w) { return 16 * (w ^ (2 * (w >> 3 & (D == 128 ? 3 : 1)))); }

  // Walks a piece's units and copies them into the ring.
  struct Feed {
    const char *kp, *vp, *bp;                             // the lane's words of codes, of block scales
    const float* sp;                                      // the lane's row scale
    const int32_t* row;
    int64_t total;
    int per, col, off, last_col, pg, ahead, to, num_pages, per_page, head;
    __device__ __forceinline__ Feed(const DecodeArgs& a, const Piece& p, int lane) {
      constexpr int kW = kBlocks / 16;                    // words of K's (and of V's) block scales
      kp = static_cast<const char*>(a.kc) + lane * 16;
      vp = static_cast<const char*>(a.vc) + lane * 16;
      bp = static_cast<const char*>(lane < kW ? a.kc : a.vc) + a.page * kRowB + lane % kW * 16;
      sp = (lane < kUnit ? a.ks : a.vs) + lane % kUnit;
      row = a.table + (int64_t)p.b * a.cols;
      per = a.page / kUnit;
      last_col = (p.unit0 + p.units - 1) / per;
      col = p.unit0 / per;
      off = p.unit0 - col * per;
      // page ids are read a page ahead
      pg = __ldg(row + col);
      ahead = col < last_col ? __ldg(row + col + 1) : 0;
      to = place(lane);
      total = a.num_pages * a.H_kv * a.page;
      num_pages = (int)a.num_pages;
      per_page = a.H_kv * per;
      head = p.h * per;
    }
    // the next kSub units, whole and of one page, to `at`; false where they are not
    __device__ __forceinline__ bool whole_step(char* at, int keys, int lane) {
      if (off + kSub > per || keys < kSub * kUnit || (unsigned)pg >= (unsigned)num_pages) return false;
      const int first = pg * per_page + head;             // the head's first unit in the page
      if (!in_bounds((int64_t)(first + off + kSub) * kUnit - 1, total)) return false;
      const int64_t page = (int64_t)first * (9 * D);
      const char *k = kp + page + off * kCodes, *v = vp + page + off * kCodes, *b = bp + page + off * kBlocks;
      const float* s = sp + (int64_t)(first + off) * kUnit;
      const uint32_t d = tc::smem_u32(at), c = d + to;
      constexpr int kW = kBlocks / 16;
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
#pragma unroll
        for (int x = 0; x < kCodes / 512; ++x) {
          copy16(c + u * kUnitB + x * 512, k + u * kCodes + x * 512);
          copy16(c + u * kUnitB + x * 512 + kCodes, v + u * kCodes + x * 512);
        }
        copy4(d + u * kUnitB + kAtScales + lane * 4, s + u * kUnit);
      }
      if (lane < 2 * kW) {
#pragma unroll
        for (int u = 0; u < kSub; ++u) copy16(d + u * kUnitB + kAtBlocks + lane * 16, b + u * kBlocks);
      }
      off += kSub;
      if (off == per) turn();
      return true;
    }
    // on to the next page
    __device__ __forceinline__ void turn() {
      off = 0;
      ++col;
      pg = ahead;
      ahead = col < last_col ? __ldg(row + col + 1) : 0;
    }
    // the next unit, of `keys` keys, to `at`: rows behind the last are zeros
    __device__ __forceinline__ void unit(char* at, int keys, int lane) {
      if ((unsigned)pg >= (unsigned)num_pages) {
        if (keys > 0) raise_error(kErrPages);
        keys = 0;
      }
      const int first = keys > 0 ? pg * per_page + head : 0;
      if (!in_bounds(keys > 0 ? (int64_t)(first + off) * kUnit + kUnit - 1 : 0, total)) keys = 0;
      const int64_t codes = (int64_t)first * (9 * D) + off * kCodes, blocks = (int64_t)first * (9 * D) + off * kBlocks;
      const uint32_t d = tc::smem_u32(at);
      constexpr int kW = kBlocks / 16;
#pragma unroll
      for (int x = 0; x < kCodes / 512; ++x) {
        const int n = (lane + 32 * x) * 16 / kRowB < keys ? 16 : 0;
        copy16(d + to + x * 512, kp + codes + x * 512, n);
        copy16(d + to + x * 512 + kCodes, vp + codes + x * 512, n);
      }
      if (lane < 2 * kW) copy16(d + kAtBlocks + lane * 16, bp + blocks, min(max(keys * (D / 16) - lane % kW * 16, 0), 16));
      copy4(d + kAtScales + lane * 4, sp + (int64_t)(first + off) * kUnit, lane % kUnit < keys ? 4 : 0);
      if (lane == 0) *reinterpret_cast<int*>(at + kAtKeys) = keys;
      if (++off == per) turn();
    }
  };

  // the scores of the lane's keys of the unit at `at`, in two sums of half the row each
  __device__ __forceinline__ void scores(const char* at, float (&s)[NT][2 * kX]) {
    float h[2][NT][4];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < 4; ++c) h[k][t][c] = 0.f;
    uint32_t w[2][kKR], b[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int n = (g + 8 * x) * kRowB + j * (kRowB / 4);
      const char* p = at + place(n / 16) + n % 16;
      const char* bs = at + kAtBlocks + (g + 8 * x) * (D / 16) + j * (D / 64);
      if (D == 128) {
        const uint4 t = *reinterpret_cast<const uint4*>(p);
        w[x][0] = t.x; w[x][1] = t.y; w[x][kKR - 2] = t.z; w[x][kKR - 1] = t.w;
        b[x] = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(bs));
      } else {
        const uint2 t = *reinterpret_cast<const uint2*>(p);
        w[x][0] = t.x; w[x][1] = t.y;
        b[x] = e4m3x2_to_f16x2(*reinterpret_cast<const uint8_t*>(bs));
      }
    }
#pragma unroll
    for (int i = 0; i < kKR; ++i) {
      const uint32_t s0 = __byte_perm(b[0], b[0], i < 2 ? 0x1010 : 0x3232), s1 = __byte_perm(b[1], b[1], i < 2 ? 0x1010 : 0x3232);
      uint32_t f0[4], f1[4];
      e2m1x8_to_f16x2(w[0][i], f0);
      e2m1x8_to_f16x2(w[1][i], f1);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t f[4] = {hmul2(f0[2 * x], s0), hmul2(f1[2 * x], s1), hmul2(f0[2 * x + 1], s0), hmul2(f1[2 * x + 1], s1)};
#pragma unroll
        for (int t = 0; t < NT; ++t) mma_f16(h[x][t], f, q[t][i * 4 + 2 * x], q[t][i * 4 + 2 * x + 1]);
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2 * kX; ++c) {
        if (kTwice) s[t][c] = j < 2 ? h[0][t][c] + h[1][t][c] : h[0][t][c + 2] + h[1][t][c + 2];
        else s[t][c] = h[0][t][c] + h[1][t][c];
      }
  }

  // the maximum of x over the lanes of a head
  __device__ __forceinline__ static float max_keys(float x) {
    if (kTwice) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
  }
  __device__ __forceinline__ void rescale(int t, int c, float f) {
#pragma unroll
    for (int i = 0; i < kMT; ++i) { acc[t][i][c] *= f; acc[t][i][c + 2] *= f; }
  }

  // one step: the kSub units at `at` (whole: all of their keys count)
  __device__ __forceinline__ void step(const Piece& p, float* to, const char* at, bool whole) {
    float s[kSub][NT][2 * kX], w[kSub][NT][2 * kX];       // scores and weighted scores, base 2
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
      const char* unit = at + u * kUnitB;
      const float* rs = reinterpret_cast<const float*>(unit + kAtScales);
      const int keys = whole ? kUnit : *reinterpret_cast<const int*>(unit + kAtKeys);
      scores(unit, s[u]);
#pragma unroll
      for (int x = 0; x < kX; ++x) {
        const float ks = rs[key_of(x)], lv = log2_fast(rs[kUnit + key_of(x)]);
        const bool live = key_of(x) < keys;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float v = s[u][t][c + 2 * x] * (sc[t][c] * ks);
            v = live ? v : -INFINITY;
            s[u][t][c + 2 * x] = v;
            w[u][t][c + 2 * x] = v + lv;
            if (kSeen && live && head_of(t, c) < p.gn) to[(u * p.heads + head_of(t, c)) * kUnit + key_of(x)] = v;
          }
      }
    }
    // maxima move when exceeded by 2^8; mw is kLift below the weighted scores' maximum
    float top[NT][2], topw[NT][2];
    bool moves = false;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        top[t][c] = s[0][t][c];
        topw[t][c] = w[0][t][c];
#pragma unroll
        for (int i = 1; i < kSub * kX; ++i) {
          top[t][c] = fmaxf(top[t][c], s[i / kX][t][c + 2 * (i % kX)]);
          topw[t][c] = fmaxf(topw[t][c], w[i / kX][t][c + 2 * (i % kX)]);
        }
        moves = moves || top[t][c] > m[t][c] + kLazy || topw[t][c] > mw[t][c] + (kLift + kLazy);
      }
    if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float mm = fmaxf(m[t][c], max_keys(top[t][c]));
          l[t][c] *= exp2_fast(m[t][c] - mm);
          m[t][c] = mm;
          const float mmw = fmaxf(mw[t][c], max_keys(topw[t][c]) - kLift);
          rescale(t, c, exp2_fast(mw[t][c] - mmw));
          mw[t][c] = mmw;
        }
    }
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
      uint32_t pw[2][NT][2];                               // the weights' parts, as operands
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int x = 0; x < kX; ++x) {
          float e[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            l[t][c] += exp2_fast(s[u][t][c + 2 * x] - m[t][c]);
            e[c] = exp2_fast(w[u][t][c + 2 * x] - mw[t][c]);
          }
          const uint32_t value = f32_to_f16x2(e[0], e[1]);
          const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&value));
          const uint32_t rest = f32_to_f16x2(e[0] - h.x, e[1] - h.y);
          if (kTwice) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, j < 2 ? rest : value, 2);
            pw[0][t][0] = transpose8x8(j < 2 ? value : other);
            pw[0][t][1] = transpose8x8(j < 2 ? other : rest);
          } else {
            pw[0][t][x] = transpose8x8(value);
            pw[1][t][x] = transpose8x8(rest);
          }
        }
      }
      const char* unit = at + u * kUnitB;
      uint32_t v[4][kVR], vb[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int row = 2 * j + (x & 1) + (x >> 1) * 8, n = row * kRowB + g * (kRowB / 8);
        const char* src = unit + kCodes + place(n / 16) + n % 16;
        if (D == 128) {
          const uint2 t = *reinterpret_cast<const uint2*>(src);
          v[x][0] = t.x; v[x][kVR - 1] = t.y;
        } else {
          v[x][0] = *reinterpret_cast<const uint32_t*>(src);
        }
        vb[x] = *reinterpret_cast<const uint8_t*>(unit + kAtBlocks + kBlocks + row * (D / 16) + g * (D / 8) / 16);
      }
      const uint32_t s0 = e4m3x2_to_f16x2((uint16_t)(vb[0] | vb[1] << 8)), s1 = e4m3x2_to_f16x2((uint16_t)(vb[2] | vb[3] << 8));
#pragma unroll
      for (int i = 0; i < kVR; ++i) {
        const uint32_t low = 0x0f0f0f0fu;
        const uint32_t w0 = v[0][i], w1 = v[1][i], w2 = v[2][i], w3 = v[3][i];
        uint32_t e0[4], o0[4], e1[4], o1[4];               // even and odd elements, of rows 2j, 2j + 1 and of 2j + 8, 2j + 9
        e2m1x8_to_f16x2((w0 & low) | ((w1 << 4) & ~low), e0);
        e2m1x8_to_f16x2(((w0 >> 4) & low) | (w1 & ~low), o0);
        e2m1x8_to_f16x2((w2 & low) | ((w3 << 4) & ~low), e1);
        e2m1x8_to_f16x2(((w2 >> 4) & low) | (w3 & ~low), o1);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t f[4] = {hmul2(e0[x], s0), hmul2(o0[x], s0), hmul2(e1[x], s1), hmul2(o1[x], s1)};
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < (kTwice ? 1 : 2); ++k) mma_f16(acc[t][i * 4 + x], f, pw[k][t][0], pw[k][t][1]);
        }
      }
    }
  }

  __device__ __forceinline__ void run(const DecodeArgs& a, const Piece& p) {
    Feed feed(a, p, lane);
    const int keys = min(p.len - p.unit0 * kUnit, p.units * kUnit);
    int fed = 0;                                          // keys of the piece that have been asked for
    auto stage = [&](int at) {                            // whether the step is whole
      bool whole = false;
      if (fed < keys) {
        char* const to = ring + at * kSub * kUnitB;
        whole = feed.whole_step(to, keys - fed, lane);
        if (!whole) {
#pragma unroll 1
          for (int u = 0; u < kSub; ++u) feed.unit(to + u * kUnitB, min(max(keys - fed - u * kUnit, 0), kUnit), lane);
        }
        fed += kSub * kUnit;
      }
      copies_issued();                                    // a group a step, an empty one too
      return whole;
    };
    __syncwarp();                                         // the last piece's reads are over
    bool whole = stage(0);
    scale_q();
    float* to = p.scores;
    int at = 0;
    for (int done = 0; done < keys; done += kSub * kUnit) {
      const bool next = stage(at ^ 1);
      copies_arrived<1>();
      __syncwarp();                                       // everyone's part of the step is there
      step(p, to, ring + at * kSub * kUnitB, whole);
      __syncwarp();                                       // it is read
      at ^= 1;
      whole = next;
      if (kSeen) to += kSub * p.heads * kUnit;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (kTwice) l[t][c] += __shfl_xor_sync(0xffffffffu, l[t][c], 2);
        l[t][c] += __shfl_xor_sync(0xffffffffu, l[t][c], 4);
        l[t][c] += __shfl_xor_sync(0xffffffffu, l[t][c], 8);
        l[t][c] += __shfl_xor_sync(0xffffffffu, l[t][c], 16);
        if (kTwice) {
#pragma unroll
          for (int i = 0; i < kMT; ++i) {
            acc[t][i][c] += __shfl_xor_sync(0xffffffffu, acc[t][i][c], 2);
            acc[t][i][c + 2] += __shfl_xor_sync(0xffffffffu, acc[t][i][c + 2], 2);
          }
        }
        rescale(t, c, exp2f(mw[t][c] - m[t][c]));         // sums in units of 2^m again
      }
  }

  // the lane's values of head (t, c): D / 8 consecutive ones, from g * D / 8 on
  __device__ __forceinline__ void values(int t, int c, float (&f)[D / 8]) const {
#pragma unroll
    for (int e = 0; e < D / 16; ++e) {
      f[2 * e] = acc[t][e][c];
      f[2 * e + 1] = acc[t][e][c + 2];
    }
  }
  __device__ __forceinline__ void partial(float2* ml, float* o, int gn) const {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int hl = t * 8 + 2 * j + c;
        if (hl >= gn) continue;
        if (g == 0) ml[hl] = make_float2(m[t][c], l[t][c]);
        float f[D / 8];
        values(t, c, f);
        float* d = o + hl * D + g * (D / 8);
#pragma unroll
        for (int e = 0; e < D / 8; e += 4) *reinterpret_cast<float4*>(d + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
      }
  }
  __device__ __forceinline__ void result(const DecodeArgs& a, const Piece& p) const {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int hl = t * 8 + 2 * j + c;
        if (hl >= p.gn) continue;
        const int hq = p.h * a.G + p.g0 + hl;
        const float inv = 1.f / l[t][c];
        if (kSeen && g == 0) finish(a, p.b, hq, m[t][c], l[t][c]);
        if (g == 0 && a.lse) a.lse[(int64_t)p.b * a.H_q + hq] = (m[t][c] + log2f(l[t][c])) * kLn2;
        float f[D / 8];
        values(t, c, f);
#pragma unroll
        for (int e = 0; e < D / 8; ++e) f[e] = l[t][c] == 0.f ? 0.f : f[e] * inv;
        TQ* d = reinterpret_cast<TQ*>(a.o) + (int64_t)p.b * a.o_b + (int64_t)hq * a.o_h + g * (D / 8);
#pragma unroll
        for (int e = 0; e < D / 8; e += 8) {
          Row8<TQ> y;
          y.set(f + e);
          y.store(d + e);
        }
      }
  }
};

template <int D, bool kSeen>
int run_four(const DecodeArgs& a, bool simt, cudaStream_t st) {
  if (use_simt(a, simt)) {
    if (a.dtype == ULYSSES_BF16) return run_simt<__nv_bfloat16, Codes4, D, kSeen>(a, st);
    return run_simt<float, Codes4, D, kSeen>(a, st);
  }
  if (a.dtype != ULYSSES_BF16) return run<SplitEngine<kE2m1, D, kSeen>, D, D == 128 ? 2 : 3>(a, st);
  if (a.G <= 4) return run<FourEngine<D, 1, true, kSeen>, D, 3>(a, st);
  if (a.G <= 8) return run<FourEngine<D, 1, false, kSeen>, D, 3>(a, st);
  return run<FourEngine<D, 2, false, kSeen>, D, 2>(a, st);
}
template <bool kSeen>
int run_widths(const DecodeArgs& a, bool simt, cudaStream_t st) {
  return a.D == 128 ? run_four<128, kSeen>(a, simt, st) : run_four<64, kSeen>(a, simt, st);
}

}  // namespace

int launch_decode_4bit(const DecodeArgs& a, bool simt, cudaStream_t st) {
  return a.seen ? run_widths<true>(a, simt, st) : run_widths<false>(a, simt, st);
}

}  // namespace ulysses
