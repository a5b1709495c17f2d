// Attention of one new token per sequence over the paged cache
// (include/ulysses.h, ulysses_attn_decode): the engines and kernels.  They are
// compiled in attn_decode.cu (16- and 32-bit and e4m3 caches), attn_decode_4bit.cu
// (e2m1) and attn_decode_seen.cu (with the tokens' attention weights).
//
//   s_j = scale * q . k_j,  o = sum_j softmax(s)_j v_j,  lse = log sum_j e^{s_j}
//
// in one pass with a running maximum m (base-2 exponents): a key with
// s > m + 8 moves m and rescales the sums, otherwise m stays, which is exact
// because o = acc / l and lse = m + log l hold for any m.
//
// Bound by HBM: every cached row is read once and costs 4 flops a byte at 4
// query heads a kv head in bf16, 27 TFLOP/s at the copy rate, 1.4% of the dense
// tensor peak.  So the work is to keep enough loads in flight (about 64 KB an
// SM) and to waste no time at either end.
//
// Split.  An item is (sequence, kv head, group of its query heads); its keys
// come in units of 16, which lie in one page.  The units of all items, one
// after the other, are dealt to the launch's warps in equal contiguous ranges,
// whatever the lengths: the warps read the lengths, no host knows them.  An
// item inside one warp's range is finished there; the pieces of the others go
// to the workspace, two slots a warp (the piece that its range begins in and
// the one that it ends in), and the join kernel, launched behind with a
// programmatic dependency so that its launch overlaps, adds each item's pieces
// in the order of the warps.  No atomics, nothing to initialise.  (Measured:
// one CTA an item instead, 64 ragged sequences of 512 to 32768 keys, bf16: 1846
// us; this way 305 to 314 us for 2.10 GB, 100 to 103% of the measured copy rate.
// A million keys of one sequence in e4m3: 57.3 ms and 337 us for 2.21 GB, 98%, or
// 344 as a call among others.)
// Where the page table has room for a few units a warp only, a cluster of CTAs
// takes each item and joins through distributed shared memory: one launch.
// With weights (kSeen) the engines keep each key's scores, and once the heads'
// maxima and sums are final a pass over the scores adds exp2(s - m) / l to the
// keys' slots: in the cluster from shared memory (500 bf16 keys 9.5 us and 8.7 without,
// 4099 12.9 and 13.5), else in a third kernel from the workspace.  Scores and not weights
// are kept, because a weight's maximum and sum are known last; recomputing the
// scores would read K again, 128 bytes a key in e4m3 and D = 128 against 32.
//
// Three engines walk a piece.
//   Matrix engine (bf16 queries): keys are the M = 16 side of mma m16n8k16 and
//   the query heads of the group (up to 8 or 16) the N side.  The warp-level
//   instruction leaves the pipe 83% idle or more, which is all that is asked of
//   it, and its register operands take rows straight from global memory, since
//   the contraction may run over d in any order that Q shares: no shared memory,
//   no barrier, no copy (tcgen05 reads its operands from shared memory).  Rows
//   stay in the lanes that loaded them:
//     S = K Q^T   lane (g, j) holds rows g and g + 8, the 16-byte words j, j+4, ..
//     O^T += V^T P^T   it holds rows 2j, 2j+1, 2j+8, 2j+9, words g, g+8, ..; pairs
//                 of rows are interleaved by byte permutes, and P turns from
//                 S's layout to the operand's by movmatrix
//   bf16 weights go in as three parts, which hold all 24 bits: the output is then
//   off by fp32 arithmetic and its own rounding alone, and the pipe has room.  The
//   parts are cut, not rounded, and at least 2^-126 for a weight that is not zero:
//   all are positive then, so an infinite V element gives infinity, as a part of
//   zero or below would not (0 x inf, inf - inf).
//   E4m3 codes become f16 exactly.  q is scaled by a power of two to the top of
//   f16's range (exact but for elements 2^-31 below its largest, which are off by
//   2^-39 of that); the rows' scales enter in fp32: K's times the score, V's in
//   the weight, as 2^(s + log2 vs - M + 7) with a running maximum M of its own, so
//   that the largest weights of a piece, whatever the rows' scales are, lie at 2^7
//   to 2^15 of f16's range (below 2^16), and those 2^-32 below are still held.
//   They go in as a value and its rounding error too, 2^-22: the output of a
//   million keys differs from fp32 arithmetic's by 1.6e-4 in norm, roundings of
//   the output itself; as a value alone (2^-12) by 8.8e-4.
//   Sums stay in the pipe's fp32 accumulators over a piece, which it cuts where an
//   fp32 addition rounds: after thousands of keys that shows in the last rounding
//   of some outputs (64 x 16384 keys: 1.9e-4 in norm off the definition rounded to
//   bf16, plain fp32 1.0e-4, beside the rounding's own 1.7e-3).  A step's sums added
//   in fp32 instead, 4.4e-5, cost registers: a million e4m3 keys 396 us, not 343,
//   16 bf16 heads a kv head 70, not 66.
//   Split engine (fp32 queries, from two or three heads on): fp32 operands as two
//   11-bit parts on the tf32 pipe; heads are the M side, the high parts of up
//   to 8 in its rows 0-7 and their low parts in rows 8-15, so one instruction
//   multiplies both by a part of K or V, and two make the product to 2^-21.  A
//   step's products are summed from zero and added in fp32: left to accumulate
//   in the pipe, which cuts instead of rounding, 8 x 30000 keys (8 kv heads of
//   128, 4 query heads each: 1.97 GB) were 7.5e-6 off (2-norm) in 338 us; this way
//   7.8e-7, less than plain fp32, in 394 us (75% of the copy rate).
//   SIMT engine (fp32 queries of one head or two, and by choice): FMA
//   throughout, 8 lanes a key.  (8 x 8000 keys, 8 kv heads of 128 with a query
//   head each, 0.52 GB: 81 us, 97%.)
#pragma once

#include <type_traits>

#include "internal.h"
#include "rows.cuh"
#include "tc_ptx.cuh"

namespace ulysses {

namespace {

using namespace rows;

constexpr int kUnit = 16;                       // keys of a unit
constexpr float kNoMax = -3.4028234663852886e38f;
constexpr float kLazy = 8.f;                    // a maximum moves when exceeded by 2^8
constexpr float kLift = 7.f;                    // f16 weights are 2^7 at the maximum, so at most 2^15
constexpr float kTiny = 1.17549435082228751e-38f;   // 2^-126
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWarps = 4;                       // of a CTA
constexpr int kMinUnits = 2;                    // of a warp, where there are enough for all
constexpr int kClusterUnits = 16;               // of a warp of a cluster, at most
constexpr int kWideUnits = 64;                  // of a CTA of the wider clusters, at most
constexpr int kMaxBatch = 2048;                 // sequences of one launch (their prefix sums sit in shared memory)

// How a launch is split (host), the same for both of its kernels.
struct Plan {
  int groups;       // query-head groups of a kv head
  int heads;        // query heads of a group (the last may have fewer)
  int warps;        // of the launch
  int* prefix;      // [B + 1] units before each sequence (one head); workspace
  float2* ml;       // [2 * warps][heads] (m, l); workspace
  float* o;         // [2 * warps][heads][D] sums; workspace
};

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

// Warps that share `total` units (each at least kMinUnits), the first unit of
// warp w, and the warp that has a unit.  The host keeps a launch's units below
// 2^31: 64-bit divisions here cost a microsecond of every call.
__device__ __forceinline__ int active_warps(const Plan& p, int total) {
  return min(p.warps, (total - 1) / kMinUnits + 1);
}
__device__ __forceinline__ int first_unit(int w, int active, int total) {
  const int each = (unsigned)total / (unsigned)active, rest = total - each * active;
  return w * each + min(w, rest);
}
__device__ __forceinline__ int warp_of(int unit, int active, int total) {
  const int each = (unsigned)total / (unsigned)active, rest = total - each * active;
  const int longer = rest * (each + 1);                    // units of the warps that have one more
  return unit < longer ? (unsigned)unit / (unsigned)(each + 1) : rest + (unsigned)(unit - longer) / (unsigned)each;
}

// The piece of an item that a warp walks.
struct Piece {
  int b, h, g0, gn;      // sequence, kv head, first query head of the group and how many
  int unit0, units;      // units of the item
  int len;               // the sequence's keys
  float* scores;         // kSeen: where the piece's scores go, [units][heads][16]
  int heads;             // heads of a unit there
};

// Walks the pages of a piece, a unit at a time.  Units of the cache are
// numbered ([num_pages][H_kv][page / 16]); the host keeps that below 2^31.
struct Walk {
  const int32_t* row;    // the sequence's table row
  int col, off, per, last_col, head, base, num_pages;
  __device__ __forceinline__ Walk(const DecodeArgs& a, const Piece& p) {
    row = a.table + (int64_t)p.b * a.cols;
    per = a.page / kUnit;
    col = p.unit0 / per;
    off = p.unit0 - col * per;
    last_col = (p.unit0 + p.units - 1) / per;
    head = p.h * per;
    base = a.H_kv * per;
    num_pages = (int)a.num_pages;
  }
  // page id of the current unit (0 behind the piece: its units are not loaded)
  __device__ __forceinline__ int fetch() const { return col <= last_col ? __ldg(row + col) : 0; }
  // number of the current unit, given its page id; -1 (reported) where that is out of range
  __device__ __forceinline__ int unit(int pg) const {
    if ((unsigned)pg >= (unsigned)num_pages) {
      if (col <= last_col) raise_error(kErrPages);
      return -1;
    }
    return pg * base + head + off;
  }
  __device__ __forceinline__ void next() {
    if (++off == per) { off = 0; ++col; }
  }
};

// The scores of an item's keys (in units of log 2), kept for the pass that adds
// the weights up: a full table's units for every item.
__device__ __forceinline__ float* scores_of(const DecodeArgs& a, int64_t item, int heads) {
  const int64_t units = ((int64_t)a.cols * a.page + kUnit - 1) / kUnit;
  return a.scores + item * units * heads * kUnit;
}
// Row number in the cache ([num_pages][H_kv][page]) of the first key of a unit of an
// item; -1: its page is out of range (reported where its scores were to be formed).
__device__ __forceinline__ int64_t row_of_unit(const DecodeArgs& a, int b, int h, int unit) {
  const int per = a.page / kUnit, col = unit / per;
  const int pg = __ldg(a.table + (int64_t)b * a.cols + col);
  if ((unsigned)pg >= (unsigned)a.num_pages) return -1;
  return ((pg * (int64_t)a.H_kv + h) * per + (unit - col * per)) * kUnit;
}
// Adds to a slot's weight.  One addition a slot and call, unless sequences share a
// page: then it gathers from all of them.
__device__ __forceinline__ void add_weight(const DecodeArgs& a, int64_t row, float x) {
  if (in_bounds(row, a.num_pages * a.H_kv * a.page)) atomicAdd(a.seen + row, x);
}
// The head's maximum and the inverse of its sum, for the same pass.
__device__ __forceinline__ void finish(const DecodeArgs& a, int b, int hq, float m, float l) {
  a.fin[(int64_t)b * a.H_q + hq] = make_float2(m, l == 0.f ? 0.f : 1.f / l);
}

// A sum over keys by the weights' sum.  Where no key counts (none on a good page,
// or every score -inf) l is 0 and the output 0, as of a sequence without keys;
// the sum itself may hold 0 x inf then.
__device__ __forceinline__ float quotient(float s, float l) { return l == 0.f ? 0.f : s / l; }

// ------------------------------------------------------------------ matrix engine

__device__ __forceinline__ void mma_bf16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t f32_to_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {   // 2 ulp, as exp2f, without its handling of tiny results
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// kTwice: up to 4 heads a group, each in two columns of the N side, h and h + 4;
// the scores of both are the same, and the first takes the weights' first part
// and the second their second, so one product has both (in bf16 a further one the
// third).  (A million e4m3 keys, 4 heads a kv head: 343 us; with two products 390,
// and with weights as a value alone 339.  Groups of more heads have no columns
// left: 8 ragged sequences of up to 30000 e4m3 keys, 8 heads a kv head, 45 us, a
// value alone 42; 16 heads 54 and 50.  In bf16 parts cost no time.)
template <bool kQuant, int D, int NT, bool kTwice, bool kSeen_>
struct MatrixEngine {
  using TQ = __nv_bfloat16;
  static constexpr bool kSeen = kSeen_;
  static constexpr int kHeads = kTwice ? 4 : 8 * NT;
  static constexpr int kProducts = (kQuant ? 2 : 3) - (kTwice ? 1 : 0);   // with V for a step's weights
  static constexpr int kRowB = kQuant ? D : 2 * D;        // bytes of a row
  static constexpr int kSub = kRowB == 256 ? 1 : 2;       // units of a step: 32 registers of K and of V, or 16
  static constexpr int kKW = kRowB / 64;                  // K: 16-byte words of a row per lane
  static constexpr int kVB = kRowB / 8 < 16 ? 8 : 16;     // V: bytes of a word
  static constexpr int kVW = kRowB / (8 * kVB);           //    words of a row per lane
  static constexpr int kVE = kQuant ? kVB : kVB / 2;      //    elements of a word
  static constexpr int kMT = D / 16;                      // M tiles of O^T

  uint32_t q[NT][kKW * 4 * (kQuant ? 2 : 1)];
  float acc[NT][kMT][4];
  float m[NT][2], l[NT][2], mw[NT][2], sc[NT][2];
  int lane, g, j;

  __device__ __forceinline__ MatrixEngine(int lane_) : lane(lane_), g(lane_ >> 2), j(lane_ & 3) {}

  // q as it is; scale_q() makes it the operand, behind the first rows' loads
  __device__ __forceinline__ void begin(const DecodeArgs& a, const Piece& p) {
    constexpr int kE = kQuant ? 16 : 8;                    // elements of a K word
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int hl = kTwice ? g & 3 : t * 8 + g;
      const bool live = hl < p.gn;
      const TQ* qp = reinterpret_cast<const TQ*>(a.q) + (int64_t)p.b * a.q_b + (int64_t)(p.h * a.G + p.g0 + (live ? hl : 0)) * a.q_h;
#pragma unroll
      for (int w = 0; w < kKW; ++w) {
#pragma unroll
        for (int x = 0; x < kE / 8; ++x) {
          const uint4 v = live ? ld16(qp + (w * 4 + j) * kE + x * 8) : make_uint4(0, 0, 0, 0);
          uint32_t* d = &q[t][(w * (kE / 8) + x) * 4];
          d[0] = v.x; d[1] = v.y; d[2] = v.z; d[3] = v.w;
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) { m[t][c] = kNoMax; l[t][c] = 0.f; mw[t][c] = kNoMax; sc[t][c] = a.scale_log2; }
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[t][i][c] = 0.f;
    }
  }
  __device__ __forceinline__ void scale_q() {
    if (!kQuant) return;
    constexpr int kN = sizeof(q[0]) / 4;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float big = 0.f;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        float e[2];
        bf16x2_to_f32(q[t][i], e);
        big = fmaxf(big, fmaxf(fabsf(e[0]), fabsf(e[1])));
      }
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // the power of two below the head's largest element comes to 2^14 (2^127 to 2^15: bf16 ends at 65280 then)
      int e = (int)(__float_as_uint(big) >> 23) - 127;
      e = (e < -100 ? -100 : (e > 126 ? 126 : e)) - 14;
      const float down = __int_as_float((127 - e) << 23), up = __int_as_float((127 + e) << 23);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        float x[2];
        bf16x2_to_f32(q[t][i], x);
        q[t][i] = f32_to_f16x2(x[0] * down, x[1] * down);
      }
      // from head g's lanes to those that hold the scores of heads 2j, 2j + 1
      sc[t][0] *= __shfl_sync(0xffffffffu, up, 8 * j);
      sc[t][1] *= __shfl_sync(0xffffffffu, up, 8 * j + 4);
    }
  }

  // rows of the units of a step; `unit` is its number in the cache, `keys` how
  // many of its 16 the piece has (0: none)
  struct Rows { uint4 k[kSub][2][kKW]; uint32_t v[kSub][4][kVW * kVB / 4]; float ks[kSub][2], vs[kSub][2]; };

  template <bool kAll>
  __device__ __forceinline__ void load_k(const DecodeArgs& a, Rows& r, int u, int unit, int keys) {
    const char* p = reinterpret_cast<const char*>(a.kc) + ((int64_t)unit * kUnit + g) * kRowB + j * 16;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const bool ok = kAll || g + 8 * x < keys;
#pragma unroll
      for (int w = 0; w < kKW; ++w) r.k[u][x][w] = ok ? ld16(p + x * 8 * kRowB + w * 64) : make_uint4(0, 0, 0, 0);
    }
    if (kQuant) {
      const int64_t s = (int64_t)unit * kUnit + g;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const bool ok = kAll || g + 8 * x < keys;
        r.ks[u][x] = ok ? __ldg(a.ks + s + 8 * x) : 0.f;
        r.vs[u][x] = ok ? __ldg(a.vs + s + 8 * x) : 0.f;
      }
    }
  }
  template <bool kAll>
  __device__ __forceinline__ void load_v(const DecodeArgs& a, Rows& r, int u, int unit, int keys) {
    const char* p = reinterpret_cast<const char*>(a.vc) + ((int64_t)unit * kUnit + 2 * j) * kRowB + g * kVB;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int key = (x & 1) + (x >> 1) * 8;              // from 2 j on
      const bool ok = kAll || 2 * j + key < keys;
#pragma unroll
      for (int w = 0; w < kVW; ++w) {
        if (kVB == 16) {
          const uint4 t = ok ? ld16(p + key * kRowB + w * 128) : make_uint4(0, 0, 0, 0);
          r.v[u][x][w * 4] = t.x; r.v[u][x][w * 4 + 1] = t.y; r.v[u][x][w * 4 + 2] = t.z; r.v[u][x][w * 4 + 3] = t.w;
        } else {
          const uint2 t = ok ? ld8(p + key * kRowB) : make_uint2(0, 0);
          r.v[u][x][0] = t.x; r.v[u][x][1] = t.y;
        }
      }
    }
  }
  // whole units take the path without predicates (warp-uniform)
  struct Next {
    MatrixEngine& e; const DecodeArgs& a; const int (&unit)[kSub]; const int (&keys)[kSub];
    __device__ __forceinline__ void load_k(Rows& r) {
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        if (keys[u] == kUnit) e.template load_k<true>(a, r, u, unit[u], kUnit);
        else e.template load_k<false>(a, r, u, unit[u], keys[u]);
      }
    }
    __device__ __forceinline__ void load_v(Rows& r) {
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        if (keys[u] == kUnit) e.template load_v<true>(a, r, u, unit[u], kUnit);
        else e.template load_v<false>(a, r, u, unit[u], keys[u]);
      }
    }
  };

  // two elements (x, x + 1 for e = 2x) of V's word registers as 16-bit pairs
  __device__ __forceinline__ static uint32_t v_pair(const uint32_t* w, int e2) {   // elements 2 e2, 2 e2 + 1
    if (!kQuant) return w[e2];
    return e4m3x2_to_f16x2((uint16_t)(w[e2 >> 1] >> (16 * (e2 & 1))));
  }

  // The 16-bit parts of two weights, largest first: they add up to the weight.
  // The third goes into both columns of a head with kTwice, so half of it.
  __device__ __forceinline__ static void parts(float p0, float p1, uint32_t (&part)[3]) {
    if (kQuant) {
      part[0] = f32_to_f16x2(p0, p1);
      const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&part[0]));
      part[1] = f32_to_f16x2(p0 - h.x, p1 - h.y);
      return;
    }
    const float t0 = fminf(p0, kTiny), t1 = fminf(p1, kTiny);
    float h[2];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (k == 2 && kTwice) { p0 = fmaxf(0.5f * p0, t0); p1 = fmaxf(0.5f * p1, t1); }
      part[k] = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);   // cut to bf16
      bf16x2_to_f32(part[k], h);
      p0 = fmaxf(p0 - h[0], t0);
      p1 = fmaxf(p1 - h[1], t1);
    }
  }

  // two sums of half the row each: half the chain of dependent products
  __device__ __forceinline__ void scores(const Rows& r, int u, float (&s)[NT][4]) {
    float h[2][NT][4];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < 4; ++c) h[k][t][c] = 0.f;
#pragma unroll
    for (int w = 0; w < kKW; ++w) {
      const uint32_t lo[4] = {r.k[u][0][w].x, r.k[u][0][w].y, r.k[u][0][w].z, r.k[u][0][w].w};
      const uint32_t hi[4] = {r.k[u][1][w].x, r.k[u][1][w].y, r.k[u][1][w].z, r.k[u][1][w].w};
      if (!kQuant) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t f[4] = {lo[2 * x], hi[2 * x], lo[2 * x + 1], hi[2 * x + 1]};
#pragma unroll
          for (int t = 0; t < NT; ++t) mma_bf16(h[x & 1][t], f, q[t][w * 4 + 2 * x], q[t][w * 4 + 2 * x + 1]);
        }
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t f[4] = {e4m3x2_to_f16x2((uint16_t)lo[x]), e4m3x2_to_f16x2((uint16_t)hi[x]),
                                 e4m3x2_to_f16x2((uint16_t)(lo[x] >> 16)), e4m3x2_to_f16x2((uint16_t)(hi[x] >> 16))};
#pragma unroll
          for (int t = 0; t < NT; ++t) mma_f16(h[x & 1][t], f, q[t][w * 8 + 2 * x], q[t][w * 8 + 2 * x + 1]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 4; ++c) s[t][c] = h[0][t][c] + h[1][t][c];
  }

  // the maximum of x over the lanes of a head (equal j)
  __device__ __forceinline__ static float max_keys(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
  }

  __device__ __forceinline__ void rescale(int t, int c, float f) {
#pragma unroll
    for (int i = 0; i < kMT; ++i) { acc[t][i][c] *= f; acc[t][i][c + 2] *= f; }
  }

  // one step of kSub units; `next` loads the next one's rows as the registers come free
  template <class Next>
  __device__ __forceinline__ void step(const DecodeArgs& a, const Piece& p, float* to, Rows& r, const int (&keys)[kSub], Next&& next) {
    float s[kSub][NT][4], tw[kSub][NT][4];
#pragma unroll
    for (int u = 0; u < kSub; ++u) scores(r, u, s[u]);
    float lvs[kSub][2], ks[kSub][2];
    if (kQuant) {
#pragma unroll
      for (int u = 0; u < kSub; ++u)
#pragma unroll
        for (int x = 0; x < 2; ++x) { lvs[u][x] = __log2f(r.vs[u][x]); ks[u][x] = r.ks[u][x]; }
    }
    next.load_k(r);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float top = kNoMax, topw = kNoMax;
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float v = s[u][t][c + 2 * x] * (kQuant ? sc[t][c] * ks[u][x] : sc[t][c]);
            v = g + 8 * x < keys[u] ? v : -INFINITY;
            s[u][t][c + 2 * x] = v;
            if (kSeen && g + 8 * x < keys[u] && t * 8 + 2 * j + c < p.gn)
              to[(u * p.heads + t * 8 + 2 * j + c) * kUnit + g + 8 * x] = v;
            top = fmaxf(top, v);
            if (kQuant) { tw[u][t][c + 2 * x] = v + lvs[u][x]; topw = fmaxf(topw, v + lvs[u][x]); }
          }
        if (__any_sync(0xffffffffu, top > m[t][c] + kLazy)) {
          const float mm = fmaxf(m[t][c], max_keys(top)), f = exp2_fast(m[t][c] - mm);
          m[t][c] = mm;
          l[t][c] *= f;
          if (!kQuant) rescale(t, c, f);
        }
        // mw is kLift below the maximum
        if (kQuant && __any_sync(0xffffffffu, topw > mw[t][c] + (kLift + kLazy))) {
          const float mm = fmaxf(mw[t][c], max_keys(topw) - kLift), f = exp2_fast(mw[t][c] - mm);
          mw[t][c] = mm;
          rescale(t, c, f);
        }
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float p = exp2_fast(s[u][t][c + 2 * x] - m[t][c]);
            l[t][c] += p;
            s[u][t][c + 2 * x] = kQuant ? exp2_fast(tw[u][t][c + 2 * x] - mw[t][c]) : p;
          }
      }
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
      uint32_t pw[kProducts][NT][2];                       // the weights' parts
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float p0 = s[u][t][2 * x], p1 = s[u][t][2 * x + 1];
          uint32_t part[3];
          parts(p0, p1, part);
          if (kTwice) {
            pw[0][t][x] = transpose8x8(j < 2 ? part[0] : part[1]);
            if (!kQuant) pw[kProducts - 1][t][x] = transpose8x8(part[2]);
          } else {
#pragma unroll
            for (int k = 0; k < kProducts; ++k) pw[k][t][x] = transpose8x8(part[k]);
          }
        }
#pragma unroll
      for (int w = 0; w < kVW; ++w)
#pragma unroll
        for (int e = 0; e < kVE / 2; ++e) {
          uint32_t v[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) v[x] = v_pair(&r.v[u][x][w * 4], e);
          const uint32_t f[4] = {__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[0], v[1], 0x7632),
                                 __byte_perm(v[2], v[3], 0x5410), __byte_perm(v[2], v[3], 0x7632)};
#pragma unroll
          for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int k = 0; k < kProducts; ++k) {
              if (kQuant) mma_f16(acc[t][w * (kVE / 2) + e], f, pw[k][t][0], pw[k][t][1]);
              else mma_bf16(acc[t][w * (kVE / 2) + e], f, pw[k][t][0], pw[k][t][1]);
            }
          }
        }
    }
    next.load_v(r);
  }

  __device__ __forceinline__ void run(const DecodeArgs& a, const Piece& p) {
    const int64_t total = a.num_pages * a.H_kv * a.page;
    Walk walk(a, p);
    Rows r;
    int unit[kSub], keys[kSub], nkeys[kSub], pg[kSub];
    float* to = p.scores;
    int left = min(p.len - p.unit0 * kUnit, p.units * kUnit);   // keys of the piece from the step on
    // page ids are read a step ahead of the rows, rows a step ahead of their use
    auto places = [&](int keys_left, int (&n)[kSub]) {
      Walk w = walk;
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        unit[u] = w.unit(pg[u]);
        n[u] = unit[u] >= 0 && in_bounds((int64_t)unit[u] * kUnit + kUnit - 1, total)
                   ? min(max(keys_left - u * kUnit, 0), kUnit) : 0;
        w.next();
      }
      walk = w;
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        pg[u] = w.fetch();
        w.next();
      }
    };
    {
      Walk w = walk;
#pragma unroll
      for (int u = 0; u < kSub; ++u) { pg[u] = w.fetch(); w.next(); }
    }
    places(left, keys);
    Next now{*this, a, unit, keys};
    now.load_k(r);
    now.load_v(r);
    scale_q();
    while (left > 0) {
      left -= kSub * kUnit;
      places(left, nkeys);
      Next next{*this, a, unit, nkeys};
      step(a, p, to, r, keys, next);
      if (kSeen) to += kSub * p.heads * kUnit;
#pragma unroll
      for (int u = 0; u < kSub; ++u) keys[u] = nkeys[u];
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
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
        if (kQuant) rescale(t, c, exp2f(mw[t][c] - m[t][c]));   // sums in units of 2^m again
      }
  }

  // element 0 of word w of head (t, c): kVE consecutive values of this lane
  __device__ __forceinline__ void values(int t, int c, int w, float* f) const {
#pragma unroll
    for (int e = 0; e < kVE / 2; ++e) {
      f[2 * e] = acc[t][w * (kVE / 2) + e][c];
      f[2 * e + 1] = acc[t][w * (kVE / 2) + e][c + 2];
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
#pragma unroll
        for (int w = 0; w < kVW; ++w) {
          float f[kVE];
          values(t, c, w, f);
          float* d = o + hl * D + (w * 8 + g) * kVE;
#pragma unroll
          for (int e = 0; e < kVE; e += 4) *reinterpret_cast<float4*>(d + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
        }
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
        TQ* d = reinterpret_cast<TQ*>(a.o) + (int64_t)p.b * a.o_b + (int64_t)hq * a.o_h;
#pragma unroll
        for (int w = 0; w < kVW; ++w) {
          float f[kVE];
          values(t, c, w, f);
#pragma unroll
          for (int e = 0; e < kVE; ++e) f[e] = l[t][c] == 0.f ? 0.f : f[e] * inv;
#pragma unroll
          for (int e = 0; e < kVE; e += 8) {
            Row8<TQ> y;
            y.set(f + e);
            y.store(d + (w * 8 + g) * kVE + e);
          }
        }
      }
  }
};

// ------------------------------------------------------------------ fp32 matrix engine

__device__ __forceinline__ void mma_tf32(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t to_tf32(float x) {   // nearest, 11 significant bits
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = to_tf32(x);
  lo = to_tf32(x - __uint_as_float(hi));
}

template <Held kHeld, int D, bool kSeen_>
struct SplitEngine {
  using TQ = float;
  static constexpr bool kSeen = kSeen_;
  static constexpr bool kQuant = kHeld != kAsIs, kFour = kHeld == kE2m1;
  static constexpr int kHeads = 8;
  static constexpr int kHalf = 8;                         // keys of a step
  static constexpr int kRowB = kFour ? D / 2 : (kQuant ? D : 4 * D);
  static constexpr int kKW = kRowB < 64 ? 1 : kRowB / 64; // K: words of a row per lane, of 16 bytes
  static constexpr int kKE = D / 4;                       //    elements of a row per lane
  static constexpr int kVB = kRowB / 8 < 16 ? kRowB / 8 : 16;   // V: bytes of a word
  static constexpr int kVW = kRowB / (8 * kVB);
  static constexpr int kVE = D / 8;                       //    elements of a row per lane
  static constexpr int kWE = kVE / kVW;                   //    elements of a word

  uint32_t q[kKE / 2][4];
  float acc[kVE][4];
  float m, l;
  int lane, g, j;

  struct Rows { uint4 k[kKW]; uint32_t v[2][kVW * kVB / 4]; float2 ks, vs; uint32_t kb, vb[2]; };

  __device__ __forceinline__ SplitEngine(int lane_) : lane(lane_), g(lane_ >> 2), j(lane_ & 3) {}

  // the d of K's element e in lane j
  __device__ __forceinline__ static int k_index(int e, int j) {
    constexpr int w = kKE / kKW;
    return (e / w * 4 + j) * w + e % w;
  }
  __device__ __forceinline__ void begin(const DecodeArgs& a, const Piece& p) {
    const bool live = g < p.gn;
    const float* qp = reinterpret_cast<const float*>(a.q) + (int64_t)p.b * a.q_b + (int64_t)(p.h * a.G + p.g0 + (live ? g : 0)) * a.q_h;
#pragma unroll
    for (int i = 0; i < kKE / 2; ++i)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        q[i][2 * x] = __float_as_uint(live ? qp[k_index(2 * i + x, j)] : 0.f);   // split behind the first rows' loads
#pragma unroll
    for (int i = 0; i < kVE; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[i][c] = 0.f;
    m = kNoMax;
    l = 0.f;
  }
  // slot: the row's in its page
  __device__ __forceinline__ void load_k(const DecodeArgs& a, Rows& r, int64_t row, int slot, int keys) {
    const bool ok = g < keys;
    if (kFour) {
      const char* p = reinterpret_cast<const char*>(a.kc) + e2m1_codes(row, slot, D) + g * kRowB + j * (kKE / 2);
      const uint8_t* s = reinterpret_cast<const uint8_t*>(a.kc) + e2m1_blocks(row, slot, a.page, D) + g * (D / 16) + j * (D / 64);
      if (kKE == 32) {
        r.k[0] = ok ? ld16(p) : make_uint4(0, 0, 0, 0);
        r.kb = ok ? __ldg(reinterpret_cast<const uint16_t*>(s)) : 0;
      } else {
        const uint2 t = ok ? ld8(p) : make_uint2(0, 0);
        r.k[0] = make_uint4(t.x, t.y, 0, 0);
        r.kb = ok ? __ldg(s) : 0;
      }
    }
    const char* p = reinterpret_cast<const char*>(a.kc) + (row + g) * kRowB + j * 16;
#pragma unroll
    for (int w = 0; w < (kFour ? 0 : kKW); ++w) r.k[w] = ok ? ld16(p + w * 64) : make_uint4(0, 0, 0, 0);
    if (kQuant) {
      r.ks.x = 2 * j < keys ? __ldg(a.ks + row + 2 * j) : 0.f;
      r.ks.y = 2 * j + 1 < keys ? __ldg(a.ks + row + 2 * j + 1) : 0.f;
      r.vs.x = 2 * j < keys ? __ldg(a.vs + row + 2 * j) : 0.f;
      r.vs.y = 2 * j + 1 < keys ? __ldg(a.vs + row + 2 * j + 1) : 0.f;
    }
  }
  __device__ __forceinline__ void load_v(const DecodeArgs& a, Rows& r, int64_t row, int slot, int keys) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const bool ok = 2 * j + x < keys;
      if constexpr (kFour) {
        const char* p = reinterpret_cast<const char*>(a.vc) + e2m1_codes(row, slot, D) + (2 * j + x) * kRowB + g * kVB;
        const uint8_t* s = reinterpret_cast<const uint8_t*>(a.vc) + e2m1_blocks(row, slot, a.page, D) + (2 * j + x) * (D / 16) + g * kVE / 16;
        if (kVB == 8) {
          const uint2 t = ok ? ld8(p) : make_uint2(0, 0);
          r.v[x][0] = t.x; r.v[x][kVB / 4 - 1] = t.y;
        } else {
          r.v[x][0] = ok ? ld4(p) : 0;
        }
        r.vb[x] = ok ? __ldg(s) : 0;
        continue;
      }
      const char* p = reinterpret_cast<const char*>(a.vc) + (row + 2 * j + x) * kRowB + g * kVB;
#pragma unroll
      for (int w = 0; w < kVW; ++w) {
        if constexpr (kVB == 16) {
          const uint4 t = ok ? ld16(p + w * 128) : make_uint4(0, 0, 0, 0);
          r.v[x][w * 4] = t.x; r.v[x][w * 4 + 1] = t.y; r.v[x][w * 4 + 2] = t.z; r.v[x][w * 4 + 3] = t.w;
        } else if constexpr (!kFour) {
          const uint2 t = ok ? ld8(p) : make_uint2(0, 0);
          r.v[x][0] = t.x; r.v[x][1] = t.y;
        }
      }
    }
  }
  // elements e, e + 1 of a lane's words (4 bits: block scales in the bytes of b)
  __device__ __forceinline__ static void pair(const uint32_t* w, uint32_t b, int e, float* f) {
    if (kFour) {
      uint32_t h[4];
      e2m1x8_to_f16x2(w[e / 8], h);
      const uint32_t s = e4m3x2_to_f16x2((uint16_t)((b >> (8 * (e / 16)) & 0xffu) * 0x101u)), y = hmul2(h[e % 8 / 2], s);   // exact
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&y));
      f[0] = v.x;
      f[1] = v.y;
    } else if (!kQuant) {
      f[0] = __uint_as_float(w[e]);
      f[1] = __uint_as_float(w[e + 1]);
    } else {
      const uint32_t h = e4m3x2_to_f16x2((uint16_t)(w[e / 4] >> (8 * (e % 4))));
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
      f[0] = v.x;
      f[1] = v.y;
    }
  }
  __device__ __forceinline__ void run(const DecodeArgs& a, const Piece& p) {
    const int64_t total = a.num_pages * a.H_kv * a.page;
    Walk walk(a, p);
    Rows r;
    // steps are half units: `half` is the one that `row` and `keys` stand for
    int half = 0, left = min(p.len - p.unit0 * kUnit, p.units * kUnit);
    int64_t row = 0;
    int slot = 0;
    int keys = 0, pg = walk.fetch();
    auto place = [&]() {
      if ((half & 1) == 0) {
        const int n = walk.unit(pg);
        row = (int64_t)n * kUnit;
        slot = walk.off * kUnit;
        keys = n >= 0 && in_bounds(row + kUnit - 1, total) ? min(max(left - half * kHalf, 0), kUnit) : 0;
        walk.next();
        pg = walk.fetch();
      } else {
        row += kHalf;
        slot += kHalf;
        keys = max(keys - kHalf, 0);
      }
      ++half;
    };
    place();
    load_k(a, r, row, slot, keys);
    load_v(a, r, row, slot, keys);
#pragma unroll
    for (int i = 0; i < kKE / 2; ++i)
#pragma unroll
      for (int x = 0; x < 2; ++x) split_tf32(__uint_as_float(q[i][2 * x]) * a.scale_log2, q[i][2 * x], q[i][2 * x + 1]);
    for (int at = 0; at < left; at += kHalf) {
      const int mine = min(keys, kHalf);
      // four sums: a quarter of the chain of dependent products
      float s[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[k][c] = 0.f;
      {
        uint32_t kw[kKW * 4];
#pragma unroll
        for (int w = 0; w < kKW; ++w) { kw[4 * w] = r.k[w].x; kw[4 * w + 1] = r.k[w].y; kw[4 * w + 2] = r.k[w].z; kw[4 * w + 3] = r.k[w].w; }
#pragma unroll
        for (int i = 0; i < kKE / 2; ++i) {
          float f[2];
          pair(kw, r.kb, 2 * i, f);
          if (kQuant) {
            mma_tf32(s[i % 4], q[i], __float_as_uint(f[0]), __float_as_uint(f[1]));
          } else {
            uint32_t h0, l0, h1, l1;
            split_tf32(f[0], h0, l0);
            split_tf32(f[1], h1, l1);
            mma_tf32(s[i % 2], q[i], h0, h1);
            mma_tf32(s[2 + i % 2], q[i], l0, l1);
          }
        }
      }
      const float2 ks = r.ks, vs = r.vs;
      place();
      load_k(a, r, row, slot, keys);
      // rows g and g + 8 of the product: the high and the low parts of head g
      float t0 = (s[0][0] + s[1][0]) + (s[2][0] + s[3][0]) + ((s[0][2] + s[1][2]) + (s[2][2] + s[3][2]));
      float t1 = (s[0][1] + s[1][1]) + (s[2][1] + s[3][1]) + ((s[0][3] + s[1][3]) + (s[2][3] + s[3][3]));
      if (kQuant) { t0 *= ks.x; t1 *= ks.y; }
      t0 = 2 * j < mine ? t0 : -INFINITY;
      t1 = 2 * j + 1 < mine ? t1 : -INFINITY;
      if (kSeen && g < p.gn) {
        float* to = p.scores + ((at / kUnit) * p.heads + g) * kUnit + at % kUnit + 2 * j;
        if (2 * j < mine) to[0] = t0;
        if (2 * j + 1 < mine) to[1] = t1;
      }
      if (__any_sync(0xffffffffu, fmaxf(t0, t1) > m + kLazy)) {
        float mm = fmaxf(t0, t1);
        mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, 1));
        mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, 2));
        mm = fmaxf(mm, m);
        const float f = exp2f(m - mm);
        m = mm;
        l *= f;
#pragma unroll
        for (int i = 0; i < kVE; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[i][c] *= f;
      }
      float p0 = exp2f(t0 - m), p1 = exp2f(t1 - m);
      l += p0 + p1;
      if (kQuant) { p0 *= vs.x; p1 *= vs.y; }
      uint32_t w[4];
      split_tf32(p0, w[0], w[1]);
      split_tf32(p1, w[2], w[3]);
#pragma unroll
      for (int e = 0; e < kVE; e += 2) {
        float a0[2], a1[2];                               // elements e, e + 1 of rows 2j, 2j + 1
        pair(r.v[0], r.vb[0], e, a0);
        pair(r.v[1], r.vb[1], e, a1);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          // a step's sum from zero, added in fp32: the pipe cuts what it accumulates
          float t[4] = {0.f, 0.f, 0.f, 0.f};
          if (kQuant) {
            mma_tf32(t, w, __float_as_uint(a0[x]), __float_as_uint(a1[x]));
          } else {
            uint32_t h0, l0, h1, l1;
            split_tf32(a0[x], h0, l0);
            split_tf32(a1[x], h1, l1);
            mma_tf32(t, w, l0, l1);
            mma_tf32(t, w, h0, h1);
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[e + x][c] += t[c];
        }
      }
      load_v(a, r, row, slot, keys);
    }
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
  }
  // the sums of head g: element e of V's lanes 2j + x
  template <class Store>
  __device__ __forceinline__ void each_word(float by, Store&& store) const {
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int e = 0; e < kVE; e += 4) {
        const int d = ((e / kWE) * 8 + 2 * j + x) * kWE + e % kWE;
        store(d, make_float4((acc[e][x] + acc[e][x + 2]) * by, (acc[e + 1][x] + acc[e + 1][x + 2]) * by,
                             (acc[e + 2][x] + acc[e + 2][x + 2]) * by, (acc[e + 3][x] + acc[e + 3][x + 2]) * by));
      }
  }
  __device__ __forceinline__ void partial(float2* ml, float* o, int gn) const {
    if (g >= gn) return;
    if (j == 0) ml[g] = make_float2(m, l);
    each_word(1.f, [&](int d, float4 v) { *reinterpret_cast<float4*>(o + g * D + d) = v; });
  }
  __device__ __forceinline__ void result(const DecodeArgs& a, const Piece& p) const {
    if (g >= p.gn) return;
    const int hq = p.h * a.G + p.g0 + g;
    if (kSeen && j == 0) finish(a, p.b, hq, m, l);
    if (j == 0 && a.lse) a.lse[(int64_t)p.b * a.H_q + hq] = (m + log2f(l)) * kLn2;
    float* out = reinterpret_cast<float*>(a.o) + (int64_t)p.b * a.o_b + (int64_t)hq * a.o_h;
    const bool none = l == 0.f;
    each_word(1.f / l, [&](int d, float4 v) {
      *reinterpret_cast<float4*>(out + d) = none ? make_float4(0.f, 0.f, 0.f, 0.f) : v;
    });
  }
};

// ------------------------------------------------------------------ SIMT engine

// One lane's part of a row: 8 lanes hold D values, lane i the 16-byte words
// i, i + 8, ...  (for 8-bit rows of 64 values: 8-byte words).
// load: row `row` of the cache, whose slot in its page is `slot`.
struct Codes4 {};       // a 4-bit row's element type
template <typename TC, int D> struct LaneRow;
template <int D> struct LaneRow<Codes4, D> {
  uint32_t w[D / 64], b;
  __device__ __forceinline__ void load(const void* cache, int64_t row, int slot, int page, int i) {
    const char* p = static_cast<const char*>(cache) + e2m1_codes(row, slot, D) + i * (D / 16);
    if (D == 128) {
      const uint2 v = ld8(p);
      w[0] = v.x; w[D / 64 - 1] = v.y;
    } else {
      w[0] = ld4(p);
    }
    b = __ldg(static_cast<const uint8_t*>(cache) + e2m1_blocks(row, slot, page, D) + i * (D / 8) / 16);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < D / 64; ++k) w[k] = 0;
    b = 0;
  }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t s = e4m3x2_to_f16x2((uint16_t)(b * 0x101u));
#pragma unroll
    for (int k = 0; k < D / 64; ++k) {
      uint32_t h[4];
      e2m1x8_to_f16x2(w[k], h);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint32_t y = hmul2(h[x], s);             // exact
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&y));
        f[8 * k + 2 * x] = v.x;
        f[8 * k + 2 * x + 1] = v.y;
      }
    }
  }
  __device__ static __forceinline__ int element(int e, int i) { return i * (D / 8) + e; }
};
template <int D> struct LaneRow<float, D> {
  static constexpr int kWords = D / 32;
  uint4 w[kWords];
  __device__ __forceinline__ void load(const void* cache, int64_t row, int, int, int i) {
    const float* p = static_cast<const float*>(cache) + row * D;
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
  __device__ __forceinline__ void load(const void* cache, int64_t row, int, int, int i) {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(cache) + row * D;
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
  __device__ __forceinline__ void load(const void* cache, int64_t row, int, int, int i) {
    const uint8_t* p = static_cast<const uint8_t*>(cache) + row * D;
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


template <typename TQ_, typename TC, int D, int HG, bool kSeen_>
struct SimtEngine {
  using TQ = TQ_;
  static constexpr bool kSeen = kSeen_;
  static constexpr bool kQuant = !std::is_same<TC, TQ>::value;
  static constexpr int kHeads = HG;
  static constexpr int E = D / 8;               // elements of a row per lane
  float q[HG][E], acc[HG][E], m[HG], l[HG];
  int lane, i, grp;

  __device__ __forceinline__ SimtEngine(int lane_) : lane(lane_), i(lane_ & 7), grp(lane_ >> 3) {}

  __device__ __forceinline__ void begin(const DecodeArgs& a, const Piece& p) {
#pragma unroll
    for (int g = 0; g < HG; ++g) {
      m[g] = kNoMax;
      l[g] = 0.f;
      const TQ* qp = reinterpret_cast<const TQ*>(a.q) + (int64_t)p.b * a.q_b +
                     (int64_t)(p.h * a.G + p.g0 + (g < p.gn ? g : 0)) * a.q_h;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        q[g][e] = to_f32<TQ>(qp[LaneRow<TC, D>::element(e, i)]);
        acc[g][e] = 0.f;
      }
    }
  }
  __device__ __forceinline__ void run(const DecodeArgs& a, const Piece& p) {
    const int64_t total = a.num_pages * a.H_kv * a.page;
    Walk walk(a, p);
    constexpr int kAtOnce = HG * E <= 16 && sizeof(LaneRow<TC, D>) <= 32 ? 4 : 2;   // keys of a lane group whose rows load together
    int pg = walk.fetch();
    for (int u = 0; u < p.units; ++u) {
      const int n = walk.unit(pg);
      const int64_t row0 = (int64_t)n * kUnit;
      const int slot0 = walk.off * kUnit;
      walk.next();
      pg = walk.fetch();
      if (n < 0 || !in_bounds(row0 + kUnit - 1, total)) continue;
      const int left = p.len - (p.unit0 + u) * kUnit;
#pragma unroll kAtOnce
      for (int k = grp; k < kUnit; k += 4) {
        const bool live = k < left;
        const int64_t row = row0 + k;
        LaneRow<TC, D> kr, vr;
        kr.zero();
        vr.zero();
        float ks = 1.f, vs = 1.f;
        if (live) {
          kr.load(a.kc, row, slot0 + k, a.page, i);
          vr.load(a.vc, row, slot0 + k, a.page, i);
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
          float t = s[g] * (kQuant ? a.scale_log2 * ks : a.scale_log2);
          t = live ? t : -INFINITY;
          if (kSeen && live && i == 0 && g < p.gn) p.scores[(u * p.heads + g) * kUnit + k] = t;
          if (t > m[g] + kLazy) {
            const float w = exp2f(m[g] - t);
            m[g] = t;
            l[g] *= w;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[g][e] *= w;
          }
          const float x = exp2f(t - m[g]);
          l[g] += x;
          const float pv = kQuant ? x * vs : x;
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
  }
  __device__ __forceinline__ void partial(float2* ml, float* o, int gn) const {
    if (grp != 0) return;
#pragma unroll
    for (int g = 0; g < HG; ++g) {
      if (g >= gn) break;
      if (i == 0) ml[g] = make_float2(m[g], l[g]);
#pragma unroll
      for (int e = 0; e < E; ++e) o[g * D + LaneRow<TC, D>::element(e, i)] = acc[g][e];
    }
  }
  __device__ __forceinline__ void result(const DecodeArgs& a, const Piece& p) const {
    if (grp != 0) return;
#pragma unroll
    for (int g = 0; g < HG; ++g) {
      if (g >= p.gn) break;
      const int hq = p.h * a.G + p.g0 + g;
      if (kSeen && i == 0) finish(a, p.b, hq, m[g], l[g]);
      if (i == 0 && a.lse) a.lse[(int64_t)p.b * a.H_q + hq] = (m[g] + log2f(l[g])) * kLn2;
      TQ* d = reinterpret_cast<TQ*>(a.o) + (int64_t)p.b * a.o_b + (int64_t)hq * a.o_h;
#pragma unroll
      for (int e = 0; e < E; ++e) d[LaneRow<TC, D>::element(e, i)] = from_f32<TQ>(quotient(acc[g][e], l[g]));
    }
  }
};

// ------------------------------------------------------------------ the two kernels

// Shared memory of CTA `rank` of the cluster, at this CTA's address `at`.
__device__ __forceinline__ float2 cluster_ld2(uint32_t at, int rank) {
  uint32_t p;
  float2 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t at, int rank) {
  uint32_t p;
  float4 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(p) : "memory");
  return v;
}

// Shared memory that a warp of the engine copies rows through (Engine::kRing bytes; most have none).
template <class Engine, class = void> struct Ring { static constexpr int kBytes = 0; };
template <class Engine> struct Ring<Engine, std::enable_if_t<(Engine::kRing > 0)>> { static constexpr int kBytes = Engine::kRing; };
template <class Engine>
__host__ __device__ constexpr int ring_bytes() { return Ring<Engine>::kBytes; }
template <class Engine>
__device__ __forceinline__ Engine make_engine(int lane, char* ring) {
  if constexpr (ring_bytes<Engine>() > 0) return Engine(lane, ring);
  else return Engine(lane);
}

template <class Engine, int D, int kCtas>
__global__ void __launch_bounds__(kWarps * 32, kCtas) decode_kernel(const __grid_constant__ DecodeArgs a,
                                                                    const __grid_constant__ Plan p) {
  // the engines' rings, and prefix[b]: units of the sequences before b (of one head)
  extern __shared__ __align__(16) char shared[];
  int* const prefix = reinterpret_cast<int*>(shared + kWarps * ring_bytes<Engine>());
  __shared__ int sums[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int carry = 0;
  for (int b0 = 0; b0 < a.B; b0 += kWarps * 32) {
    const int b = b0 + threadIdx.x;
    int x = b < a.B ? (length_of(a, b) + kUnit - 1) / kUnit : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sums[w];
      carry += sums[w];
    }
    if (b < a.B) prefix[b + 1] = before + x;
    __syncthreads();
  }
  if (threadIdx.x == 0) prefix[0] = 0;
  __syncthreads();
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b <= a.B; b += kWarps * 32) p.prefix[b] = prefix[b];
  // the join may be launched: it waits for the whole of this grid
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int per = a.H_kv * p.groups;                       // items of a sequence
  const int total = carry * per;
  if (total == 0) return;
  const int active = active_warps(p, total), w = blockIdx.x * kWarps + warp;
  if (w >= active) return;
  const int begin = first_unit(w, active, total), end = first_unit(w + 1, active, total);
  int b = 0;
  {
    int lo = 0, hi = a.B - 1;                              // the last b with prefix[b] * per <= begin
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] * per <= begin) lo = mid; else hi = mid - 1;
    }
    b = lo;
  }
  Engine e = make_engine<Engine>(lane, shared + warp * ring_bytes<Engine>());
  int at = begin;
  while (at < end) {
    while (prefix[b + 1] * per <= at) ++b;
    const int units = prefix[b + 1] - prefix[b], in_seq = at - prefix[b] * per;
    const int item = (unsigned)in_seq / (unsigned)units;
    const int item0 = prefix[b] * per + item * units;      // the item's first unit
    Piece pc;
    pc.b = b;
    pc.h = item / p.groups;
    pc.g0 = (item - pc.h * p.groups) * p.heads;
    pc.gn = min(a.G - pc.g0, p.heads);
    pc.unit0 = at - item0;
    pc.units = min(end, item0 + units) - at;
    pc.len = length_of(a, b);
    if (Engine::kSeen) {
      pc.heads = p.heads;
      pc.scores = scores_of(a, (int64_t)b * per + item, p.heads) + (int64_t)pc.unit0 * p.heads * kUnit;
    }
    e.begin(a, pc);
    e.run(a, pc);
    if (pc.units == units) {
      e.result(a, pc);
    } else {
      const int64_t slot = 2 * w + (at == begin ? 0 : 1);
      e.partial(p.ml + slot * p.heads, p.o + slot * p.heads * D, pc.gn);
    }
    at += pc.units;
  }
}

// Adds the attention weights of every cached token up, from the scores that the
// split launch left and the heads' final maxima and sums:
//   weights[place of key j] += sum_h exp2(s_hj - m_h) / l_h
// the query heads h of the kv head in their order.  The units of all (sequence,
// kv head) are dealt to the warps in equal ranges, a lane a key of four pairs of
// units at a time.  Bound by what the scores and the weights take (4 G + 8 bytes a
// key and kv head, from L2 for the most part) and the chain of table and scores:
// 64 ragged sequences of up to 16384 bf16 keys, 8 kv heads of 128 with 4 query
// heads each (1.06 GB of rows): 19 us behind the split kernel's 162 and the join's
// 7; a pair of units at a time 30.
constexpr int kSeenThreads = 256;
__global__ void __launch_bounds__(kSeenThreads) decode_weights_kernel(const __grid_constant__ DecodeArgs a,
                                                                      const __grid_constant__ Plan p) {
  extern __shared__ int prefix[];
  const int lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int b = threadIdx.x; b <= a.B; b += kSeenThreads) prefix[b] = p.prefix[b];
  __syncthreads();
  const int total = prefix[a.B] * a.H_kv;
  if (total == 0) return;
  const int warps = gridDim.x * (kSeenThreads / 32), active = min(warps, (total - 1) / kMinUnits + 1);
  const int w = blockIdx.x * (kSeenThreads / 32) + (threadIdx.x >> 5);
  if (w >= active) return;
  const int begin = first_unit(w, active, total), end = first_unit(w + 1, active, total);
  int lo = 0, hi = a.B - 1;                                // the last b with prefix[b] * H_kv <= begin
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] * a.H_kv <= begin) lo = mid; else hi = mid - 1;
  }
  int b = lo, at = begin;
  while (at < end) {
    while (prefix[b + 1] * a.H_kv <= at) ++b;
    const int units = prefix[b + 1] - prefix[b], h = (at - prefix[b] * a.H_kv) / units;
    const int item0 = prefix[b] * a.H_kv + h * units, unit0 = at - item0;
    const int n = min(end, item0 + units) - at, len = length_of(a, b);
    const float2* fin = a.fin + (int64_t)b * a.H_q + h * a.G;
    // a lane a key of four pairs of units at a time: their loads do not wait for each other
    constexpr int kPairs = 4;
    for (int u = 0; u < n; u += 2 * kPairs) {
      const int key = lane & 15;
      int unit[kPairs];
      int64_t row[kPairs];
      float x[kPairs];
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const int v = u + 2 * i + (lane >> 4);
        unit[i] = unit0 + v;
        const bool live = v < n && unit[i] * kUnit + key < len;
        row[i] = live ? row_of_unit(a, b, h, unit[i]) : -1;
        if (!live) unit[i] = unit0;
        x[i] = 0.f;
      }
      for (int g = 0; g < p.groups; ++g) {
        const int g0 = g * p.heads, gn = min(a.G - g0, p.heads);
        const float* s = scores_of(a, ((int64_t)b * a.H_kv + h) * p.groups + g, p.heads) + key;
#pragma unroll 4
        for (int k = 0; k < gn; ++k) {
          const float2 f = fin[g0 + k];
#pragma unroll
          for (int i = 0; i < kPairs; ++i) x[i] += exp2f(s[((int64_t)unit[i] * p.heads + k) * kUnit] - f.x) * f.y;
        }
      }
#pragma unroll
      for (int i = 0; i < kPairs; ++i)
        if (row[i] >= 0) add_weight(a, row[i] + key, x[i]);
    }
    at += n;
  }
}

// Short caches: a cluster per item.  Its warps take equal ranges of the item's
// units and leave their sums in shared memory; each CTA joins a part of the
// item's outputs from the shared memories of all.  One launch, no workspace.
template <class Engine, int D, int kCtas>
__global__ void __launch_bounds__(kWarps * 32, kCtas) decode_cluster_kernel(const __grid_constant__ DecodeArgs a,
                                                                            int groups, int heads, int ctas) {
  constexpr int kH = Engine::kHeads;
  __shared__ __align__(16) float so[kWarps][kH][D];
  __shared__ __align__(8) float2 sml[kWarps][kH];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)tc::cluster_ctarank(), item = blockIdx.x / ctas;
  Piece pc;
  const int hg = item % (a.H_kv * groups);
  pc.b = item / (a.H_kv * groups);
  pc.h = hg / groups;
  pc.g0 = (hg - pc.h * groups) * heads;
  pc.gn = min(a.G - pc.g0, heads);
  pc.len = length_of(a, pc.b);
  const int units = (pc.len + kUnit - 1) / kUnit, warps = ctas * kWarps, w = rank * kWarps + warp;
  pc.unit0 = first_unit(w, warps, units);
  pc.units = first_unit(w + 1, warps, units) - pc.unit0;
  Engine e = make_engine<Engine>(lane, nullptr);
  e.begin(a, pc);
  if (pc.units > 0) e.run(a, pc);
  e.partial(sml[warp], &so[warp][0][0], pc.gn);
  __syncwarp();
  tc::cluster_sync();
  const int total = pc.gn * D / 4, each = (total + ctas - 1) / ctas;
  const uint32_t o_at = tc::smem_u32(&so[0][0][0]), ml_at = tc::smem_u32(&sml[0][0]);
  for (int i = rank * each + threadIdx.x; i < min(total, (rank + 1) * each); i += kWarps * 32) {
    const int hl = i / (D / 4), c = i - hl * (D / 4);
    float m = kNoMax, l = 0.f;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r = 0; r < ctas; ++r) {
#pragma unroll
      for (int k = 0; k < kWarps; ++k) m = fmaxf(m, cluster_ld2(ml_at + (k * kH + hl) * 8, r).x);
    }
    for (int r = 0; r < ctas; ++r) {
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float2 ml = cluster_ld2(ml_at + (k * kH + hl) * 8, r);
        const float4 x = cluster_ld4(o_at + ((k * kH + hl) * D + c * 4) * 4, r);
        const float f = exp2f(ml.x - m);
        l += ml.y * f;
        s.x += x.x * f; s.y += x.y * f; s.z += x.z * f; s.w += x.w * f;
      }
    }
    using TQ = typename Engine::TQ;
    const int hq = pc.h * a.G + pc.g0 + hl;
    TQ* d = reinterpret_cast<TQ*>(a.o) + (int64_t)pc.b * a.o_b + (int64_t)hq * a.o_h + c * 4;
    d[0] = from_f32<TQ>(quotient(s.x, l));
    d[1] = from_f32<TQ>(quotient(s.y, l));
    d[2] = from_f32<TQ>(quotient(s.z, l));
    d[3] = from_f32<TQ>(quotient(s.w, l));
    if (c == 0 && a.lse) a.lse[(int64_t)pc.b * a.H_q + hq] = (m + log2f(l)) * kLn2;   // l = 0: -inf
  }
  __syncwarp();
  tc::cluster_sync();                                      // no CTA leaves while another reads its sums
}

// The same for the 4-bit engine, and with weights.  Pieces are joined in their CTA
// first and then over the cluster, so a CTA may have eight warps (kW) of half as
// many units; each warp then adds its own keys' weights to their slots, from its
// scores in shared memory.  Bound by the chain length -> page -> K -> V -> joins:
// 4099 bf16 keys of 8 kv heads of 128, 4 query heads each, with weights 12.9 us, 777
// 4-bit ones without 8.0.  Joined over all warps of the cluster at once, by four
// warps a CTA, with the heads' maxima and sums found one after the other, it was
// 17.3 and 9.2.
template <class Engine, int D, int kW, int kCtas>
__global__ void __launch_bounds__(kW * 32, kCtas) decode_wide_cluster_kernel(const __grid_constant__ DecodeArgs a,
                                                                              int groups, int heads, int ctas) {
  constexpr int kH = Engine::kHeads, kUnits = kWideUnits / kW;
  extern __shared__ __align__(16) char shared[];           // rings, sums, scores
  __shared__ __align__(8) float2 sml[kW][kH], all_ml[kH];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)tc::cluster_ctarank(), item = blockIdx.x / ctas;
  Piece pc;
  const int hg = item % (a.H_kv * groups);
  pc.b = item / (a.H_kv * groups);
  pc.h = hg / groups;
  pc.g0 = (hg - pc.h * groups) * heads;
  pc.gn = min(a.G - pc.g0, heads);
  pc.len = length_of(a, pc.b);
  const int units = (pc.len + kUnit - 1) / kUnit, warps = ctas * kW, w = rank * kW + warp;
  pc.unit0 = first_unit(w, warps, units);
  pc.units = first_unit(w + 1, warps, units) - pc.unit0;
  float* const so = reinterpret_cast<float*>(shared + kW * ring_bytes<Engine>());   // [warps][kH][D]
  if (Engine::kSeen) {
    pc.heads = heads;
    pc.scores = so + kW * kH * D + warp * (kUnits * heads * kUnit);
  }
  Engine e = make_engine<Engine>(lane, shared + warp * ring_bytes<Engine>());
  e.begin(a, pc);
  if (pc.units > 0) e.run(a, pc);
  constexpr int kPairs = kUnits / 2;                       // of units, a lane a key
  const int key = lane & 15;
  int64_t row[kPairs];                                     // kSeen: of the lane's keys
  if (Engine::kSeen) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int unit = 2 * i + (lane >> 4);
      const bool live = unit < pc.units && (pc.unit0 + unit) * kUnit + key < pc.len;
      row[i] = live ? row_of_unit(a, pc.b, pc.h, pc.unit0 + unit) : -1;
    }
  }
  e.partial(sml[warp], so + warp * kH * D, pc.gn);
  __syncthreads();
  const int total = pc.gn * D / 4;
  for (int i = threadIdx.x; i < total; i += kW * 32) {
    const int hl = i / (D / 4), c = i - hl * (D / 4);
    float m = kNoMax, l = 0.f;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kW; ++k) m = fmaxf(m, sml[k][hl].x);
#pragma unroll
    for (int k = 0; k < kW; ++k) {
      const float2 ml = sml[k][hl];
      const float4 x = *reinterpret_cast<const float4*>(so + (k * kH + hl) * D + c * 4);
      const float f = exp2f(ml.x - m);
      l += ml.y * f;
      s.x += x.x * f; s.y += x.y * f; s.z += x.z * f; s.w += x.w * f;
    }
    *reinterpret_cast<float4*>(so + hl * D + c * 4) = s;   // nobody else has read or will read this place
    if (c == 0) all_ml[hl] = make_float2(m, l);
  }
  __syncwarp();
  tc::cluster_sync();
  const uint32_t o_at = tc::smem_u32(so), ml_at = tc::smem_u32(all_ml);
  if (Engine::kSeen) {                                     // (one group: the item has all of the kv head's query heads)
    constexpr int kRounds = (kH + 3) / 4;                  // a lane a CTA of four heads
    float top[kRounds], inv[kRounds], x[kPairs];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const float2 ml = cluster_ld2(ml_at + min(4 * r + (lane >> 3), pc.gn - 1) * 8, min(lane & 7, ctas - 1));
      float t = ml.x;
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
      float l = (lane & 7) < ctas ? ml.y * exp2f(ml.x - t) : 0.f;
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      top[r] = t;
      inv[r] = l == 0.f ? 0.f : 1.f / l;
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) x[i] = 0.f;
#pragma unroll
    for (int h = 0; h < kH; ++h) {
      if (h >= pc.gn) break;
      const float mh = __shfl_sync(0xffffffffu, top[h / 4], h % 4 * 8), ih = __shfl_sync(0xffffffffu, inv[h / 4], h % 4 * 8);
#pragma unroll
      for (int i = 0; i < kPairs; ++i)
        if (row[i] >= 0) x[i] += exp2f(pc.scores[((2 * i + (lane >> 4)) * heads + h) * kUnit + key] - mh) * ih;
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
      if (row[i] >= 0) add_weight(a, row[i] + key, x[i]);
  }
  const int each = (total + ctas - 1) / ctas;
  for (int i = rank * each + threadIdx.x; i < min(total, (rank + 1) * each); i += kW * 32) {
    const int hl = i / (D / 4), c = i - hl * (D / 4);
    float2 ml[8];
    float4 x[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      ml[r] = make_float2(kNoMax, 0.f);
      x[r] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < ctas) {
        ml[r] = cluster_ld2(ml_at + hl * 8, r);
        x[r] = cluster_ld4(o_at + (hl * D + c * 4) * 4, r);
      }
    }
    float m = kNoMax, l = 0.f;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < 8; ++r) m = fmaxf(m, ml[r].x);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const float f = exp2f(ml[r].x - m);
      l += ml[r].y * f;
      s.x += x[r].x * f; s.y += x[r].y * f; s.z += x[r].z * f; s.w += x[r].w * f;
    }
    using TQ = typename Engine::TQ;
    const int hq = pc.h * a.G + pc.g0 + hl;
    TQ* d = reinterpret_cast<TQ*>(a.o) + (int64_t)pc.b * a.o_b + (int64_t)hq * a.o_h + c * 4;
    d[0] = from_f32<TQ>(quotient(s.x, l));
    d[1] = from_f32<TQ>(quotient(s.y, l));
    d[2] = from_f32<TQ>(quotient(s.z, l));
    d[3] = from_f32<TQ>(quotient(s.w, l));
    if (c == 0 && a.lse) a.lse[(int64_t)pc.b * a.H_q + hq] = (m + log2f(l)) * kLn2;   // l = 0: -inf
  }
  __syncwarp();
  tc::cluster_sync();                                      // no CTA leaves while another reads its sums
}

// Running sum of pieces: the largest m so far, and l and the values in its units.
struct Sum { float m, l; float4 s; };
__device__ __forceinline__ void add_piece(Sum& x, float m, float l, float4 s) {
  const float top = fmaxf(x.m, m), fa = exp2f(x.m - top), fb = exp2f(m - top);
  x.m = top;
  x.l = x.l * fa + l * fb;
  x.s.x = x.s.x * fa + s.x * fb;
  x.s.y = x.s.y * fa + s.y * fb;
  x.s.z = x.s.z * fa + s.z * fb;
  x.s.w = x.s.w * fa + s.w * fb;
}
__device__ __forceinline__ void add_lanes(Sum& x, int o) {   // with lane ^ o, in one order on both
  Sum y;
  y.m = __shfl_xor_sync(0xffffffffu, x.m, o);
  y.l = __shfl_xor_sync(0xffffffffu, x.l, o);
  y.s.x = __shfl_xor_sync(0xffffffffu, x.s.x, o);
  y.s.y = __shfl_xor_sync(0xffffffffu, x.s.y, o);
  y.s.z = __shfl_xor_sync(0xffffffffu, x.s.z, o);
  y.s.w = __shfl_xor_sync(0xffffffffu, x.s.w, o);
  if (threadIdx.x & o) {
    add_piece(y, x.m, x.l, x.s);
    x = y;
  } else {
    add_piece(x, y.m, y.l, y.s);
  }
}

// Adds the pieces of an item, for one of its heads, or writes the result of a
// sequence without keys.  kPart: a CTA for 32 of the head's values, 32 pieces
// at a time (few items, hundreds of pieces each); kRow: a CTA for the head;
// kWarp: a warp for it (many items, of a few pieces or none).
enum Join { kPart, kRow, kWarp };
template <typename TQ, int D, Join kHow, int kJoin, bool kSeen>
__global__ void __launch_bounds__(kJoin) decode_join_kernel(const __grid_constant__ DecodeArgs a,
                                                            const __grid_constant__ Plan p) {
  constexpr int kLanes = kHow == kPart ? 8 : D / 4;                // threads across the values, four each
  constexpr int kParts = (kHow == kWarp ? 32 : kJoin) / kLanes;    // pieces at a time
  __shared__ Sum sums[kJoin / 32][kLanes];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int bh = kHow == kPart ? blockIdx.x / (D / 32) : (kHow == kRow ? blockIdx.x : blockIdx.x * (kJoin / 32) + warp);
  const int c = (kHow == kPart ? (blockIdx.x % (D / 32)) * 8 : 0) + threadIdx.x % kLanes;
  const int part = (kHow == kWarp ? lane : threadIdx.x) / kLanes;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (bh >= a.B * a.H_q) return;                           // a whole warp (or CTA)
  const int b = bh / a.H_q, hq = bh - b * a.H_q;
  const int h = hq / a.G, gi = (hq - h * a.G) / p.heads, hl = hq - h * a.G - gi * p.heads;
  TQ* d = reinterpret_cast<TQ*>(a.o) + (int64_t)b * a.o_b + (int64_t)hq * a.o_h + c * 4;
  const int before = p.prefix[b], after = p.prefix[b + 1], all = p.prefix[a.B];
  const int units = after - before;
  Sum x{kNoMax, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  if (units > 0) {
    const int per = a.H_kv * p.groups;
    const int total = all * per, active = active_warps(p, total);
    const int first = before * per + (h * p.groups + gi) * units;
    const int w0 = warp_of(first, active, total), w1 = warp_of(first + units - 1, active, total);
    if (w0 == w1) return;                                  // finished where it was walked
    // the piece of warp w: in its first slot unless the item begins inside w's range
    const int skip = first_unit(w0, active, total) == first ? 0 : 1;
    // kBatch pieces load before the first is added: hundreds of pieces are one or two waits
    constexpr int kBatch = kHow == kPart ? 8 : 4;
    const int n = w1 - w0 + 1;
    const float2* ml = p.ml + 2 * w0 * p.heads + hl;
    const float* o = p.o + (int64_t)(2 * w0 * p.heads + hl) * D + c * 4;
    for (int i0 = part; i0 < n; i0 += kBatch * kParts) {
      float2 t[kBatch];
      float4 v[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * kParts;
        const int at = (2 * i + (i == 0 ? skip : 0)) * p.heads;
        t[k] = i < n ? ml[at] : make_float2(kNoMax, 0.f);
        v[k] = i < n ? *reinterpret_cast<const float4*>(o + (int64_t)at * D) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float top = x.m;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) top = fmaxf(top, t[k].x);
      const float f = exp2f(x.m - top);
      x.m = top;
      x.l *= f;
      x.s = make_float4(x.s.x * f, x.s.y * f, x.s.z * f, x.s.w * f);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float u = exp2f(t[k].x - top);
        x.l += t[k].y * u;
        x.s.x += v[k].x * u; x.s.y += v[k].y * u; x.s.z += v[k].z * u; x.s.w += v[k].w * u;
      }
    }
  }
#pragma unroll
  for (int o = kLanes; o < 32; o <<= 1) add_lanes(x, o);
  if (kHow != kWarp) {
    if (lane < kLanes) sums[warp][lane] = x;
    __syncthreads();
    if (threadIdx.x >= kLanes) return;
    float top = x.m;
#pragma unroll
    for (int k = 1; k < kJoin / 32; ++k) top = fmaxf(top, sums[k][lane].m);
    x = Sum{top, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll
    for (int k = 0; k < kJoin / 32; ++k) {
      const Sum y = sums[k][lane];
      const float u = exp2f(y.m - top);
      x.l += y.l * u;
      x.s.x += y.s.x * u; x.s.y += y.s.y * u; x.s.z += y.s.z * u; x.s.w += y.s.w * u;
    }
  } else if (lane >= kLanes) {
    return;
  }
  if (kSeen && c == 0) finish(a, b, hq, x.m, x.l);
  if (x.l == 0.f) {   // no key that counts; a branch: selects at each quotient made 25.9 us of 24 ragged x 4096 27.0
    d[0] = d[1] = d[2] = d[3] = from_f32<TQ>(0.f);
    if (c == 0 && a.lse) a.lse[(int64_t)b * a.H_q + hq] = -INFINITY;
    return;
  }
  d[0] = from_f32<TQ>(x.s.x / x.l);
  d[1] = from_f32<TQ>(x.s.y / x.l);
  d[2] = from_f32<TQ>(x.s.z / x.l);
  d[3] = from_f32<TQ>(x.s.w / x.l);
  if (c == 0 && a.lse) a.lse[(int64_t)b * a.H_q + hq] = (x.m + log2f(x.l)) * kLn2;
}

// ------------------------------------------------------------------ host

constexpr int kMaxWarps = 152 * 16;              // of a launch: slots of the workspace

// fp32 queries of few heads a key are SIMT work: at 1-2 flops a byte the FMA
// pipe keeps up.  8 kv heads, 8 x 30000 keys, 1.97 GB of D = 128: 1 query head a
// kv head 279 us (105% of the copy rate), 2 291 (101%; 8 x 8000 keys 85, and 98 by
// the fp32 matrix engine); 3 heads 569 by SIMT and 394 by the matrix engine, 4 374
// and 394, 8 734 and 394.  0.98 GB of D = 64: 1 head 166, 2 205 and 186, 4 304 and
// 186.
inline bool use_simt(const DecodeArgs& a, bool chosen) {
  return chosen || (a.dtype == ULYSSES_FP32 && a.G <= (a.D == 128 ? 2 : 1));
}

// query heads of a group
inline int heads_of(const DecodeArgs& a, bool simt) {
  const int most = a.dtype == ULYSSES_BF16 ? 16 : 8;
  if (!use_simt(a, simt)) return a.G < most ? a.G : most;
  return a.G < 4 ? (a.G < 2 ? 1 : 2) : 4;
}

// CTAs of a cluster for each item, or 0: split the keys over the whole launch.
// A cluster saves the join, its launch and a workspace, but waits for the longest
// item: it is taken while its warps have at most kClusterUnits units when the
// table is full and all clusters are resident at once.  (8 kv heads of 4, one
// sequence, clusters and split: 777 keys 7.2 and 9.2 us, 3000 9.5 and 10.8, 4500
// 11.3 and 11.8, 6000 13.6 and 13.1, 8000 17.0 and 13.6: on time alone they part at
// 5000 keys.  16 x 4000 ragged 32.7 and 19.5, 4 x 16000 ragged 37.0 and 22.2, which
// twice as many units would take.)  152 SMs and not the device's: the workspace is
// asked for without one, and both have to choose alike.
inline int cluster_of(const DecodeArgs& a, int heads) {
  if (a.seen && a.G > heads) return 0;              // groups of one kv head add to the same weights
  const int64_t items = (int64_t)a.B * a.H_kv * ((a.G + heads - 1) / heads);
  const int64_t units = ((int64_t)a.cols * a.page + kUnit - 1) / kUnit;
  int c = 8;
  while (c > 1 && items * c > 152 * 2) c /= 2;
  if (items * c > 152 * 2 || units > (int64_t)c * kWarps * kClusterUnits) return 0;
  while (c > 1 && units <= (int64_t)(c / 2) * kWarps) c /= 2;   // no more warps than units
  return c;
}
// CTAs of eight warps for each item, one an SM, or 0: four warps.  Twice the warps
// are taken where they hold the table too and four in each of eight CTAs would have
// more than `most` units.  (8 kv heads of 4, one sequence, 8 warps and 4: with weights
// 1000 bf16 keys 9.4 and 10.7 us, 1000 4-bit ones 9.6 and 10.7, 4 x 1500 bf16 11.4 and
// 13.0; without, of 4-bit ones, which are walked two units a step, 777 8.6 and 8.0,
// 1500 8.7 and 10.  Few: 100 keys 8.5 and 7.6.  Two CTAs an SM: 4 x 1500 with weights
// 23.3 and 11.4.)  16 clusters of eight CTAs run at once, and not 19, as a GPC's SMs are
// no multiple of eight: 3 x 1500 of 6 kv heads with weights 17.4 us, 11.6 in fours.
inline int wide_cluster_of(const DecodeArgs& a, int heads, int most) {
  const int64_t items = (int64_t)a.B * a.H_kv * ((a.G + heads - 1) / heads);
  const int64_t units = ((int64_t)a.cols * a.page + kUnit - 1) / kUnit;
  int c = items > 16 ? 4 : 8;
  while (c > 1 && items * c > 152) c /= 2;
  return items * c > 152 || units > (int64_t)c * kWideUnits || units <= 8 * kWarps * most ? 0 : c;
}

struct WsLayout { size_t prefix, ml, o, fin, scores, total; };
inline WsLayout ws_layout(const DecodeArgs& a, int heads) {
  WsLayout w{};
  const int b = a.B < kMaxBatch ? a.B : kMaxBatch;
  w.ml = align256((size_t)(b + 1) * sizeof(int));
  w.o = w.ml + align256((size_t)2 * kMaxWarps * heads * 8);
  w.fin = w.o + align256((size_t)2 * kMaxWarps * heads * a.D * 4);
  w.scores = w.fin + (a.seen ? align256((size_t)b * a.H_q * 8) : 0);
  const size_t units = ((size_t)a.cols * a.page + kUnit - 1) / kUnit, groups = (a.G + heads - 1) / heads;
  w.total = w.scores + (a.seen ? align256((size_t)b * a.H_kv * groups * units * heads * kUnit * 4) : 0);
  return w;
}

// Reported here, and not left for the next call's check to find.
inline int launch_failed(const char* what, cudaError_t err) {
  (void)cudaGetLastError();
  return set_error(ULYSSES_ERR_CUDA, "%s: launch failed: %s", what, cudaGetErrorString(err));
}

template <class Kernel>
int launch_cluster(Kernel kernel, int warps, int bytes, const DecodeArgs& a, const Plan& p, int c, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.B * a.H_kv * p.groups * c));
  cfg.blockDim = dim3(warps * 32);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)c;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, a, p.groups, p.heads, c);
  if (err != cudaSuccess) return launch_failed("attn_decode", err);
  count_launch();
  return ULYSSES_OK;
}
template <class Engine, int D, int kW, int kCtas>
int run_cluster(const DecodeArgs& a, const Plan& p, int c, cudaStream_t st) {
  constexpr int kSums = kW * (ring_bytes<Engine>() + Engine::kHeads * D * 4);
  constexpr int kScores = Engine::kSeen ? kWideUnits * kUnit * 4 : 0;   // bytes of a head
  const auto kernel = decode_wide_cluster_kernel<Engine, D, kW, kCtas>;
  static PerDeviceOnce<> once;
  if (const int rc = opt_in_smem(once, (const void*)kernel, kSums + kScores * Engine::kHeads, "attn_decode")) return rc;
  return launch_cluster(kernel, kW, kSums + kScores * p.heads, a, p, c, st);
}

// kEight: clusters may have eight warps a CTA.
template <class Engine, int D, int kCtas, bool kEight = Engine::kSeen || (ring_bytes<Engine>() > 0)>
int run(const DecodeArgs& a, cudaStream_t st) {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  int ctas = sms * kCtas;
  if (ctas * kWarps > kMaxWarps) ctas = kMaxWarps / kWarps;
  Plan p{};
  p.heads = a.G < Engine::kHeads ? a.G : Engine::kHeads;
  p.groups = (a.G + p.heads - 1) / p.heads;
  p.warps = ctas * kWarps;
  if (const int c = cluster_of(a, p.heads)) {
    if constexpr (Engine::kSeen || ring_bytes<Engine>() > 0) {
      if constexpr (kEight)
        if (const int wide = wide_cluster_of(a, p.heads, Engine::kSeen ? 1 : 2)) return run_cluster<Engine, D, 8, 1>(a, p, wide, st);
      return run_cluster<Engine, D, kWarps, kCtas < 3 ? kCtas : 2>(a, p, c, st);
    } else {
      return launch_cluster(decode_cluster_kernel<Engine, D, kCtas>, kWarps, 0, a, p, c, st);
    }
  }
  const WsLayout w = ws_layout(a, p.heads);
  char* ws = (char*)a.ws;
  p.prefix = (int*)(ws + w.prefix);
  p.ml = (float2*)(ws + w.ml);
  p.o = (float*)(ws + w.o);
  // sequences of a launch: their prefix sums fit shared memory, their units 31 bits with every table full
  const int64_t full = ((int64_t)a.cols * a.page + kUnit - 1) / kUnit * a.H_kv * p.groups;
  int batch = kMaxBatch;
  if (full > 0 && 2147483647 / full < batch) batch = (int)(2147483647 / full);
  if (batch == 0)
    return set_error(ULYSSES_ERR_UNSUPPORTED, "attn_decode: table_cols * page_size * H_kv * groups of one sequence at or above 2^35");
  for (int b0 = 0; b0 < a.B; b0 += batch) {
    DecodeArgs x = a;
    x.B = a.B - b0 < batch ? a.B - b0 : batch;
    x.q = (const char*)a.q + (int64_t)b0 * a.q_b * sizeof(typename Engine::TQ);
    x.o = (char*)a.o + (int64_t)b0 * a.o_b * sizeof(typename Engine::TQ);
    x.lse = a.lse ? a.lse + (int64_t)b0 * a.H_q : nullptr;
    x.table = a.table + (int64_t)b0 * a.cols;
    x.lens = a.lens + b0;
    if (Engine::kSeen) {
      x.fin = (float2*)(ws + w.fin);
      x.scores = (float*)(ws + w.scores);
    }
    if (ring_bytes<Engine>() > 0) {
      static PerDeviceOnce<> once;
      if (const int rc = opt_in_smem(once, (const void*)decode_kernel<Engine, D, kCtas>,
                                     kWarps * ring_bytes<Engine>() + (kMaxBatch + 1) * (int)sizeof(int), "attn_decode"))
        return rc;
    }
    decode_kernel<Engine, D, kCtas><<<ctas, kWarps * 32, kWarps * ring_bytes<Engine>() + (x.B + 1) * sizeof(int), st>>>(x, p);
    count_launch();
    int rc = check_launch("attn_decode");
    if (rc) return rc;
    const int rows = x.B * a.H_q;
    // 1 x 48000 keys (32 rows): 37.0 us by parts, 46.2 by rows, 78.1 by warps; 16 x 4000 (512 rows): 53.5, 46.8,
    // 48.9; 95 ragged of up to 8096, D = 64 (3040 rows): 89.4, 75.9, 70.8.  CTAs of 256 threads take more pieces
    // at a time, of 128 find room beside the last of the split kernel's: by parts 1 x 48000 37.0 and 38.6 us, 30
    // ragged of up to 8000 (240 rows) 21.0 and 18.7; by rows 16 x 4000 ragged (512 rows) 20.4 and 22.0, 37 x 4000
    // ragged (1184 rows) 32.4 and 31.9
    const Join how = rows <= 256 ? kPart : (rows <= 152 * 16 ? kRow : kWarp);
    const int threads = how == kWarp || (how == kPart ? rows <= 128 : rows <= 608) ? 256 : 128;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(how == kPart ? rows * (D / 32) : (how == kRow ? rows : (rows + 7) / 8)));
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    using TQ = typename Engine::TQ;
    constexpr bool kSeen = Engine::kSeen;
    const auto join = how == kWarp                      ? decode_join_kernel<TQ, D, kWarp, 256, kSeen>
                      : how == kPart && threads == 256 ? decode_join_kernel<TQ, D, kPart, 256, kSeen>
                      : how == kPart                   ? decode_join_kernel<TQ, D, kPart, 128, kSeen>
                      : threads == 256                 ? decode_join_kernel<TQ, D, kRow, 256, kSeen>
                                                       : decode_join_kernel<TQ, D, kRow, 128, kSeen>;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, join, x, p);
    if (err != cudaSuccess) return launch_failed("attn_decode join", err);
    count_launch();
    if constexpr (Engine::kSeen) {
      cfg.gridDim = dim3((unsigned)(sms * 4));
      cfg.blockDim = dim3(kSeenThreads);
      cfg.dynamicSmemBytes = (x.B + 1) * sizeof(int);
      const cudaError_t err2 = cudaLaunchKernelEx(&cfg, decode_weights_kernel, x, p);
      if (err2 != cudaSuccess) return launch_failed("attn_decode weights", err2);
      count_launch();
    }
  }
  return ULYSSES_OK;
}

template <bool kQuant, int D, bool kSeen>
int run_matrix(const DecodeArgs& a, cudaStream_t st) {
  if (a.G <= 4) return run<MatrixEngine<kQuant, D, 1, true, kSeen>, D, 3>(a, st);
  if (a.G <= 8) return run<MatrixEngine<kQuant, D, 1, false, kSeen>, D, 3>(a, st);
  return run<MatrixEngine<kQuant, D, 2, false, kSeen>, D, 2>(a, st);
}
template <typename TQ, typename TC, int D, bool kSeen>
int run_simt(const DecodeArgs& a, cudaStream_t st) {
  if (a.G == 1) return run<SimtEngine<TQ, TC, D, 1, kSeen>, D, 4, false>(a, st);
  if (a.G <= 3) return run<SimtEngine<TQ, TC, D, 2, kSeen>, D, 3, false>(a, st);
  return run<SimtEngine<TQ, TC, D, 4, kSeen>, D, 2, false>(a, st);
}

template <bool kQuant, int D, bool kSeen>
int run_engine(const DecodeArgs& a, bool simt, cudaStream_t st) {
  if (use_simt(a, simt)) {
    if (a.dtype == ULYSSES_BF16)
      return run_simt<__nv_bfloat16, std::conditional_t<kQuant, uint8_t, __nv_bfloat16>, D, kSeen>(a, st);
    return run_simt<float, std::conditional_t<kQuant, uint8_t, float>, D, kSeen>(a, st);
  }
  if (a.dtype == ULYSSES_BF16) return run_matrix<kQuant, D, kSeen>(a, st);
  return run<SplitEngine<kQuant ? kE4m3 : kAsIs, D, kSeen>, D, D == 128 ? 2 : 3>(a, st);
}
// Caches as they are (kQuant: in e4m3).
template <bool kQuant, bool kSeen>
int run_decode(const DecodeArgs& a, bool simt, cudaStream_t st) {
  return a.D == 128 ? run_engine<kQuant, 128, kSeen>(a, simt, st) : run_engine<kQuant, 64, kSeen>(a, simt, st);
}

}  // namespace
}  // namespace ulysses
