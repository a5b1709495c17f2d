// Eviction from the paged cache by accumulated attention weight
// (include/ulysses.h, ulysses_cache_evict).
//
// Of a sequence's n tokens m = min(n, keep) stay, for every kv head its own: the
// last r = min(m, recent), and of the n - r before them the m - r of greatest
// weight (the lower position first among equals).  They close up in their order,
// so position i of what is left is the i-th token that stays, and the places from
// m on are left as they were.
//
// Two kernels.  The first selects: a cluster of CTAs for each (sequence, kv head)
// finds the smallest weight that stays by its bits, three digits from the top, each
// from a histogram over the cluster, and writes the list of the rows that stay.
// Weights are ordered as unsigned numbers (sign and magnitude made monotone; -0 as
// +0, NaN above everything).  Up to 16384 positions a CTA stay in registers from
// digit to digit.  Bound by latencies: launch, lengths, table, weights, and about
// 1.5 us a digit (10 us for a few positions, 25 for 131072 in 8 CTAs a head, of
// which 2.5 would be reading them).  Where at most 32 positions are left to choose
// from, they are put in order one against the other instead.
//
// The second moves rows, in place: a chunk of rows, K, V, scales and weights, is
// read into shared memory and then written.  A row never moves up, so what a chunk
// of C rows overwrites are rows of itself and of at most two chunks before it (the
// C places hold at most C kept rows, neighbours in rank): it waits until those have
// been read.  CTAs take chunks by a counter, in order.  A chunk's reading waits for
// writes of chunks before it alone, and those for reading of chunks before them, so
// the first chunk that is not done can always go on.  Every kept row is read and
// written once, which is all the memory traffic there is beside the weights'.
// Bound by HBM: 65536 rows of 8 heads of 128 in bf16 (537 MB) move in 91 us, 87% of
// the copy rate.  Through registers, a chunk at a time, it was 128 us (a CTA's
// loads, waits and stores one after the other); with a fence before each chunk's
// flag, which waits for the stores before it, 139 us; one chunk ahead in shared
// memory 118, of which 25 were waits for neighbours that read no earlier than they
// wrote; as it is, two to five chunks ahead, the flags are there when they are
// asked for.
#include "internal.h"
#include "rows.cuh"
#include "tc_ptx.cuh"

namespace ulysses {

ULYSSES_ERROR_READER(read_error_cache_evict)

namespace {

using namespace rows;

constexpr int kUnit = 16;          // positions of one thread at a time
constexpr int kThreads = 512;      // of a selecting CTA
constexpr int kMoveThreads = 256;  // that move rows, of a CTA
constexpr int kMaxBatch = 2048;    // sequences of one launch (their prefix sums sit in shared memory)
constexpr int kBins = 2048;        // of a digit of 11 bits

// What the selection leaves for the move (workspace).
struct Lists {
  int2* size;      // [B] (tokens before, tokens that stay); equal where nothing moves
  int* ticket;     // chunks taken
  int64_t* src;    // [B][H][positions] rows of the positions that stay, rising (rows: [num_pages][H][page])
  int* before;     // [B][H][chunks] how many of those lie before position chunk * c
  int* read;       // [B][H][chunks] 1: the chunk's rows have been read
  int64_t positions, chunks;
  int chunk;       // rows moved together: 16 KB of K and of V, at most 128
};
constexpr int chunk_of(int row_bytes) { return row_bytes >= 128 ? 16384 / row_bytes : 128; }

// A weight as a number whose order is the weights'.
__device__ __forceinline__ uint32_t order_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);             // -0 + 0 = +0
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct Size { int n, m, r; };
// Tokens, those that stay, those of them that stay for their age.  A length that
// the table cannot hold is reported, and such a sequence is left as it is.
__device__ __forceinline__ Size size_of(const EvictArgs& a, int b) {
  const int n = __ldg(a.lens + b), keep = __ldg(a.keep + b);
  if (n < 0 || n > (int64_t)a.cols * a.page) {
    raise_error(kErrPages);
    return Size{n, n, 0};
  }
  const int m = keep < 0 || keep > n ? n : keep;
  return Size{n, m, min(m, a.recent)};
}

// The orders of the 16 weights of unit `unit` of a sequence's head.
__device__ __forceinline__ void load_unit(const EvictArgs& a, const int32_t* row, int h, int unit, uint32_t (&key)[kUnit]) {
  const int per = a.page / kUnit, col = unit / per;
  const int64_t at = ((int64_t)__ldg(row + col) * a.H + h) * a.page + (unit - col * per) * kUnit;
  const float4* p = reinterpret_cast<const float4*>(a.w + at);
  if (!in_bounds(at, a.num_pages * a.H * a.page)) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = p[i];
    key[4 * i] = order_of(v.x); key[4 * i + 1] = order_of(v.y); key[4 * i + 2] = order_of(v.z); key[4 * i + 3] = order_of(v.w);
  }
}

__device__ __forceinline__ int ld_cluster(uint32_t at, int rank) {
  uint32_t p;
  int v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(p) : "memory");
  return v;
}

// Inclusive sums over the block's threads; `sums` holds a number for each warp.
__device__ __forceinline__ int block_scan(int x, int* sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();                                         // the last use of sums is over
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int s = lane < kThreads / 32 ? sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < kThreads / 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  total = __shfl_sync(0xffffffffu, s, kThreads / 32 - 1);
  const int below = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
  return x + (warp > 0 ? below : 0);
}

// A barrier of the cluster's threads, or of the one CTA's.
__device__ __forceinline__ void sync_all(int ctas) {
  if (ctas > 1) {
    __syncwarp();
    tc::cluster_sync();
  } else {
    __syncthreads();
  }
}
// An int of every CTA's shared memory, at this CTA's address of it (0 of those there
// are not); the loads do not wait for each other.
constexpr int kMaxCtas = 8;
__device__ __forceinline__ void ld_ranks(const int* p, int ctas, int (&v)[kMaxCtas]) {
#pragma unroll
  for (int c = 0; c < kMaxCtas; ++c) v[c] = c < ctas ? ld_cluster(tc::smem_u32(p), c) : 0;
}

// Units a thread holds in registers from one digit to the next; those of longer
// sequences are loaded again (from L2).
constexpr int kHold = 2;

__global__ void __launch_bounds__(kThreads, 2) evict_select_kernel(const __grid_constant__ EvictArgs a,
                                                                const __grid_constant__ Lists l, int ctas) {
  __shared__ int hist[kBins];
  __shared__ int part[kBins];                              // totals over the cluster, of this CTA's bins
  __shared__ int part_sum[3];                              // theirs, for each digit
  __shared__ int sums[kThreads / 32];
  __shared__ int found[3];                                 // the digit, the positions in the digits above it, in it
  __shared__ int mine[2];                                  // of this CTA's positions: above the threshold, at it
  __shared__ int few;                                      // positions left to choose from, when they are few: how many
  __shared__ int few_key[32], few_at[32];                  // of this CTA's, their orders and places
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int rank = ctas > 1 ? (int)tc::cluster_ctarank() : 0, item = blockIdx.x / ctas;
  const int b = item / a.H, h = item - b * a.H;
  const int32_t* row = a.table + (int64_t)b * a.cols;
  int page = (int)threadIdx.x < a.cols ? __ldg(row + threadIdx.x) : 0;   // on its way beside the lengths
  Size z = size_of(a, b);
  if (blockIdx.x == 0 && threadIdx.x == 0) *l.ticket = 0;
  // a page out of range: the sequence is left as it is, all of its heads (each looks at the whole row)
  int bad = 0;
  if (z.m < z.n)
    for (int c = threadIdx.x, last = (z.n - 1) / a.page; c <= last; c += kThreads) {
      bad |= (unsigned)page >= (unsigned)a.num_pages;
      if (c + kThreads <= last) page = __ldg(row + c + kThreads);
    }
  for (int i = threadIdx.x; i < kBins; i += kThreads) hist[i] = 0;
  if (threadIdx.x < 2) mine[threadIdx.x] = 0;
  if (threadIdx.x == 0) few = 0;
  if (threadIdx.x < 3) part_sum[threadIdx.x] = 0;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) raise_error(kErrPages);
    z.m = z.n;
  }
  if (h == 0 && rank == 0 && threadIdx.x == 0) l.size[b] = make_int2(z.n, z.m);
  if (z.m >= z.n) return;                                  // the whole cluster
  int64_t* src = l.src + item * l.positions;
  int* before = l.before + item * l.chunks;
  const int old = z.n - z.r, k = z.m - z.r;                // k of `old` positions stay
  for (int i = rank * kThreads + threadIdx.x; i < (z.m + l.chunk - 1) / l.chunk; i += ctas * kThreads) l.read[item * l.chunks + i] = 0;
  for (int i = rank * kThreads + threadIdx.x; i < z.r; i += ctas * kThreads) {
    const int p = old + i, col = p / a.page;
    src[k + i] = ((int64_t)__ldg(row + col) * a.H + h) * a.page + (p - col * a.page);
  }
  const int units = (old + kUnit - 1) / kUnit, each = (units + ctas - 1) / ctas;
  const int u0 = min(rank * each, units), u1 = min(u0 + each, units);
  uint32_t held[kHold][kUnit];
  if (k > 0) {
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      const int u = u0 + i * kThreads + threadIdx.x;
      if (u < u1) load_unit(a, row, h, u, held[i]);
    }
  }

  // the threshold, digit by digit: `prefix` holds the bits found, k_left of the
  // positions that have them are to stay
  uint32_t prefix = 0;
  int k_left = k;
  if (k > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
      auto count_unit = [&](const uint32_t (&key)[kUnit], int u) {
        const int live = old - u * kUnit;
        if (pass > 0) {                                    // few: those with the digits found so far
          uint32_t some = 0;
#pragma unroll
          for (int i = 0; i < kUnit; ++i) some |= (uint32_t)(key[i] >> (shift + bits) == prefix) << i;
          if (live < kUnit) some &= (1u << live) - 1;
          if (!some) return;
#pragma unroll
          for (int i = 0; i < kUnit; ++i)
            if (some >> i & 1) atomicAdd(hist + ((key[i] >> shift) & ((1 << bits) - 1)), 1);
          return;
        }
        // neighbours of one bin are counted together: tokens nobody looked at are alike
        int bin = -1, count = 0;
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
          if (i >= live) continue;
          const int d = (int)(key[i] >> shift);
          if (d == bin) { ++count; continue; }
          if (count) atomicAdd(hist + bin, count);
          bin = d;
          count = 1;
        }
        if (count) atomicAdd(hist + bin, count);
      };
#pragma unroll
      for (int i = 0; i < kHold; ++i) {
        const int u = u0 + i * kThreads + threadIdx.x;
        if (u < u1) count_unit(held[i], u);
      }
      for (int u = u0 + kHold * kThreads + threadIdx.x; u < u1; u += kThreads) {
        uint32_t key[kUnit];
        load_unit(a, row, h, u, key);
        count_unit(key, u);
      }
      sync_all(ctas);
      const int share = kBins / ctas;
      int above = 0, owner = 0, sum = 0, total;
      if (ctas > 1) {
        // each CTA adds up its share of the bins over the cluster ..
        for (int i = threadIdx.x; i < share; i += kThreads) {
          int v[kMaxCtas], n = 0;
          ld_ranks(hist + rank * share + i, ctas, v);
#pragma unroll
          for (int c = 0; c < kMaxCtas; ++c) n += v[c];
          part[i] = n;
          sum += n;
        }
        sum = __reduce_add_sync(0xffffffffu, sum);
        if ((threadIdx.x & 31) == 0 && sum) atomicAdd(part_sum + pass, sum);
        sync_all(ctas);
        // .. all find the share that has the digit ..
        int v[kMaxCtas];
        ld_ranks(part_sum + pass, ctas, v);
        bool passed = false;
#pragma unroll
        for (int c = kMaxCtas - 1; c >= 0; --c) {
          if (!passed && (above + v[c] >= k_left || c == 0)) {
            owner = c;
            passed = true;
          }
          above += passed ? 0 : v[c];
        }
      }
      // .. and the digit in it, from the top
      constexpr int kOwn = kBins / kThreads;               // bins of a thread, at most
      int n[kOwn];
      sum = 0;
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int bin = share - 1 - ((int)threadIdx.x * kOwn + i);
        n[i] = bin >= 0 ? (ctas > 1 ? ld_cluster(tc::smem_u32(part + bin), owner) : hist[bin]) : 0;
        sum += n[i];
      }
      int upto = above + block_scan(sum, sums, total) - sum;   // positions in the bins above
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        if (upto < k_left && upto + n[i] >= k_left) {      // one thread, once
          found[0] = owner * share + share - 1 - ((int)threadIdx.x * kOwn + i);
          found[1] = upto;
          found[2] = n[i];
        }
        upto += n[i];
      }
      __syncthreads();
      const int digit = found[0];
      k_left -= found[1];
      prefix = prefix << bits | (uint32_t)digit;
      if (ctas > 1) {                                      // of this CTA's: those above, at last those at it
        int own = 0;
        for (int i = threadIdx.x; i < kBins; i += kThreads) {
          own += i > digit ? hist[i] : 0;
          if (i == digit && pass == 2) mine[1] = hist[i];
        }
        own = __reduce_add_sync(0xffffffffu, own);
        if ((threadIdx.x & 31) == 0 && own) atomicAdd(mine, own);
      }
      if (pass < 2 && found[2] <= 32) {
        // few have the digits so far: they are put in order one against the other
        auto keep_few = [&](const uint32_t (&key)[kUnit], int u) {
          const int live = old - u * kUnit;
          uint32_t some = 0;
#pragma unroll
          for (int i = 0; i < kUnit; ++i) some |= (uint32_t)(i < live && key[i] >> shift == prefix) << i;
          if (!some) return;
          const int x = atomicAdd(&few, __popc(some));
#pragma unroll
          for (int i = 0; i < kUnit; ++i)
            if (some >> i & 1) {
              const int at = x + __popc(some & ((1u << i) - 1));
              few_key[at] = (int)key[i];
              few_at[at] = u * kUnit + i;
            }
        };
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
          const int u = u0 + i * kThreads + threadIdx.x;
          if (u < u1) keep_few(held[i], u);
        }
        for (int u = u0 + kHold * kThreads + threadIdx.x; u < u1; u += kThreads) {
          uint32_t key[kUnit];
          load_unit(a, row, h, u, key);
          keep_few(key, u);
        }
        sync_all(ctas);
        if (threadIdx.x < 32) {
          int v[kMaxCtas], at = threadIdx.x, owner = -1;   // lane i has the i-th of all CTAs'
          if (ctas > 1) ld_ranks(&few, ctas, v);
#pragma unroll
          for (int c = 0; c < kMaxCtas; ++c) {
            const int n = ctas > 1 ? v[c] : (c == 0 ? few : 0);
            if (owner < 0) {
              if (at < n) owner = c;
              else at -= n;
            }
          }
          uint32_t key = 0;
          int place = 0, ahead = 0;
          if (owner >= 0) {
            key = (uint32_t)(ctas > 1 ? ld_cluster(tc::smem_u32(few_key + at), owner) : few_key[at]);
            place = ctas > 1 ? ld_cluster(tc::smem_u32(few_at + at), owner) : few_at[at];
          }
          for (int i = 0; i < found[2]; ++i) {
            const uint32_t other = __shfl_sync(0xffffffffu, key, i);
            const int its = __shfl_sync(0xffffffffu, place, i);
            ahead += other > key || (other == key && its < place);
          }
          const uint32_t last = __ballot_sync(0xffffffffu, owner >= 0 && ahead == k_left - 1);   // one lane: the last that stays
          const uint32_t edge = __shfl_sync(0xffffffffu, key, __ffs(last) - 1);
          const uint32_t over = __ballot_sync(0xffffffffu, owner >= 0 && key > edge);
          const bool own = owner == rank;
          const uint32_t own_over = __ballot_sync(0xffffffffu, own && key > edge), own_at = __ballot_sync(0xffffffffu, own && key == edge);
          if (threadIdx.x == 0) {
            found[0] = (int)edge;
            found[1] = __popc(over);
            if (ctas > 1) {
              mine[0] += __popc(own_over);
              mine[1] = __popc(own_at);
            }
          }
        }
        __syncthreads();
        prefix = (uint32_t)found[0];
        k_left -= found[1];
        break;
      }
      if (pass < 2) {                                      // cleared for the next digit
        for (int i = threadIdx.x; i < kBins; i += kThreads) hist[i] = 0;
        __syncthreads();
      }
    }
  }
  // positions that stay before this CTA's: those above the threshold and the first k_left at it
  int gt0 = 0, eq0 = 0;
  if (ctas > 1) {
    __syncthreads();
    sync_all(ctas);
    int g[kMaxCtas], e[kMaxCtas];
    ld_ranks(mine, ctas, g);
    ld_ranks(mine + 1, ctas, e);
#pragma unroll
    for (int c = 0; c < kMaxCtas; ++c) {
      gt0 += c < rank ? g[c] : 0;
      eq0 += c < rank ? e[c] : 0;
    }
  }
  auto list_units = [&](const uint32_t (&key)[kUnit], int u) {
    uint32_t gt = 0, eq = 0;                               // a bit a position
    if (u < u1 && k > 0) {
      const int live = old - u * kUnit;
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
        gt |= (uint32_t)(i < live && key[i] > prefix) << i;
        eq |= (uint32_t)(i < live && key[i] == prefix) << i;
      }
    }
    int total;
    const int counts = __popc(gt) | __popc(eq) << 16;      // at most 8192 of each
    const int upto = block_scan(counts, sums, total) - counts;
    const int g = gt0 + (upto & 0xffff), e = eq0 + (upto >> 16);
    if (u < u1) {
      const int at = g + min(e, k_left);
      if ((u * kUnit & (l.chunk - 1)) == 0) before[u * kUnit / l.chunk] = at;
      // the first of those at it, as many as are left
      for (int over = __popc(eq) - max(k_left - e, 0); over > 0; --over) eq &= ~(0x80000000u >> __clz(eq));
      const uint32_t stay = gt | eq;
      if (stay) {
        const int per = a.page / kUnit, col = u / per;
        const int64_t first = ((int64_t)__ldg(row + col) * a.H + h) * a.page + (u - col * per) * kUnit;
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
          const int to = at + __popc(stay & ((1u << i) - 1));
          if ((stay >> i & 1) && in_bounds(to, k)) src[to] = first + i;
        }
      }
    }
    gt0 += total & 0xffff;
    eq0 += total >> 16;
  };
#pragma unroll
  for (int i = 0; i < kHold; ++i)
    if (u0 + i * kThreads < u1) list_units(held[i], u0 + i * kThreads + threadIdx.x);
  for (int t = u0 + kHold * kThreads; t < u1; t += kThreads) {
    uint32_t key[kUnit];
    const int u = t + threadIdx.x;
    if (u < u1 && k > 0) load_unit(a, row, h, u, key);
    list_units(key, u);
  }
  if (ctas > 1) sync_all(ctas);                            // no CTA leaves while another reads its shared memory
}

// Where a chunk's rows are and where they go; -1: a row that does not move.
template <int kChunk>
struct Places {
  int64_t from[kChunk], to[kChunk];
  int* flags;                                              // the item's; NULL: there is no chunk
  int c, first, last;                                      // the chunk, and those that have rows in its places
};

// Of a thread, in a chunk: words of K's and V's rows; weights and row scales; block scales.
constexpr int own_words(int row_bytes) { return 2 * chunk_of(row_bytes) * (row_bytes / 16) / kMoveThreads; }
constexpr int own_scalars(int row_bytes, bool scales) { return ((scales ? 3 : 1) * chunk_of(row_bytes) + kMoveThreads - 1) / kMoveThreads; }
constexpr int own_blocks(int row_bytes, bool four) { return four ? 2 * chunk_of(row_bytes) / kMoveThreads : 0; }
constexpr int stage_bytes(int row_bytes, bool four, bool scales) {
  return (own_words(row_bytes) * 16 + own_scalars(row_bytes, scales) * 4 + own_blocks(row_bytes, four) * 8) * kMoveThreads;
}
// Chunks on their way through shared memory, two CTAs an SM.
constexpr int stages_of(int row_bytes, bool four, bool scales) {
  const int n = 102400 / stage_bytes(row_bytes, four, scales);
  return n < 6 ? n : 6;
}
constexpr int kMovers = kMoveThreads + 96;

// A slot of a ring and the phase of its barriers.
struct Turn {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++at == n) { at = 0; phase ^= 1; }
  }
};

// Moves the rows that stay.  Eight warps copy a chunk's rows to shared memory,
// kStages - 1 chunks ahead, and from there to their places.  A ninth warp finds the
// places of the chunks to come.  A tenth tells the other CTAs that a chunk's rows
// have been read, as soon as they have arrived, and an eleventh waits for the
// chunks whose rows lie in this one's places: each on its own, so that no chunk's
// reading waits for another chunk.  kRowB: bytes of a row's values or codes.
template <int kRowB, bool kFour, bool kScales>
__global__ void __launch_bounds__(kMovers, 2) evict_move_kernel(const __grid_constant__ EvictArgs a,
                                                                const __grid_constant__ Lists l) {
  constexpr int kChunk = chunk_of(kRowB);
  constexpr int kW = kRowB / 16;                           // words of a row
  constexpr int kOwn = own_words(kRowB), kScalars = own_scalars(kRowB, kScales), kBlocks = own_blocks(kRowB, kFour);
  constexpr int kStages = stages_of(kRowB, kFour, kScales), kStageB = stage_bytes(kRowB, kFour, kScales);
  constexpr int kRing = kStages + 2;                       // chunks whose places are known
  constexpr int D = kRowB * 2;                             // kFour
  static_assert(kOwn >= 1 && kStages >= 2 && (kChunk & (kChunk - 1)) == 0 && kChunk % kUnit == 0, "");
  using Place = Places<kChunk>;
  extern __shared__ __align__(16) char stages[];           // kStages, for the rows on their way
  int2* const size = reinterpret_cast<int2*>(stages + kStages * kStageB);   // [B], and chunks of the sequences before, of one head
  int* const prefix = reinterpret_cast<int*>(size + a.B);
  __shared__ Place places[kRing];
  __shared__ __align__(8) uint64_t placed[kRing], read[kRing], free_[kRing], done[kRing];
  __shared__ int stop;                                     // a wait gave up: all leave
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      tc::mbar_init(placed + i, 1);                        // its places are known
      tc::mbar_init(read + i, kMoveThreads);               // its rows have arrived
      tc::mbar_init(free_ + i, 1);                         // those of others in its places too
      tc::mbar_init(done + i, kMoveThreads / 32 + 2);      // nobody looks at its places any more
    }
    stop = 0;
    tc::fence_barrier_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int ticket = 0;                                          // the ninth warp's first lane's: the next chunk
  if (threadIdx.x == kMoveThreads) ticket = atomicAdd(l.ticket, 1);
  for (int b = threadIdx.x; b < a.B; b += kMovers) {
    const int2 z = l.size[b];
    size[b] = z;
    if (blockIdx.x == 0) a.out[b] = z.y;
  }
  __syncthreads();

  if (warp < kMoveThreads / 32) {                          // ---- the rows
    // a thread copies its words of a chunk to places of its own in a stage, and from there; words, weights and row
    // scales, block scales are numbered through the chunk, K's before V's
    const auto scalar = [&](int i) { return i < kChunk ? a.w : (kScales && i < 3 * kChunk ? (i < 2 * kChunk ? a.ks : a.vs) : nullptr); };
    const auto slot_of = [&](int64_t row) {                // of its page
      const unsigned unit = (unsigned)(row / kUnit);
      return (int)(unit % (unsigned)(a.page / kUnit)) * kUnit + (int)(row % kUnit);
    };
    const auto word_at = [&](int i, int64_t row) {
      char* base = static_cast<char*>(i >= kChunk * kW ? a.vc : a.kc);
      return base + (kFour ? e2m1_codes(row, slot_of(row), D) : row * kRowB) + i % kW * 16;
    };
    const auto block_at = [&](int i, int64_t row) {
      return static_cast<char*>(i >= kChunk ? a.vc : a.kc) + e2m1_blocks(row, slot_of(row), a.page, D);
    };
    constexpr int kAtScalars = kOwn * kMoveThreads * 16, kAtBlocks = kAtScalars + kScalars * kMoveThreads * 4;
    const auto load = [&](const Place& p, int stage, uint64_t* arrived) {
      const uint32_t to = tc::smem_u32(stages + stage * kStageB);
#pragma unroll
      for (int x = 0; x < kOwn; ++x) {
        const int i = x * kMoveThreads + threadIdx.x;
        const int64_t from = p.from[i / kW % kChunk];
        if (from >= 0) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(to + i * 16), "l"(word_at(i, from)) : "memory");
      }
#pragma unroll
      for (int x = 0; x < kScalars; ++x) {
        const int i = x * kMoveThreads + threadIdx.x;
        const int64_t from = p.from[i % kChunk];
        if (scalar(i) && from >= 0)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(to + kAtScalars + i * 4), "l"(scalar(i) + from) : "memory");
      }
#pragma unroll
      for (int x = 0; x < kBlocks; ++x) {
        const int i = x * kMoveThreads + threadIdx.x;
        const int64_t from = p.from[i % kChunk];
        if (from >= 0)
          asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" :: "r"(to + kAtBlocks + i * 8), "l"(block_at(i, from)), "n"(D == 128 ? 8 : 4) : "memory");
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" :: "r"(tc::smem_u32(arrived)) : "memory");
    };
    Turn ahead, now;
    int to_stage = 0, stage = 0, more = 1;                 // more: of the chunk that is loaded next
    const auto load_next = [&]() {
      if (!more) return true;
      if (!tc::mbar_wait(placed + ahead.at, ahead.phase, &stop)) return false;
      more = places[ahead.at].flags != nullptr;
      if (more) load(places[ahead.at], to_stage, read + ahead.at);
      ahead.next(kRing);
      to_stage = to_stage + 1 == kStages ? 0 : to_stage + 1;
      return true;
    };
    bool ok = true;
    for (int i = 0; i < kStages - 1; ++i) ok = ok && load_next();
    while (ok) {
      const Place& p = places[now.at];
      if (!p.flags) break;
      ok = load_next() && tc::mbar_wait(read + now.at, now.phase, &stop) && tc::mbar_wait(free_ + now.at, now.phase, &stop);
      if (ok) {
        const char* from = stages + stage * kStageB;
#pragma unroll
        for (int x = 0; x < kOwn; ++x) {
          const int i = x * kMoveThreads + threadIdx.x;
          const int64_t to = p.to[i / kW % kChunk];
          if (to >= 0) st16(word_at(i, to), *reinterpret_cast<const uint4*>(from + i * 16));
        }
#pragma unroll
        for (int x = 0; x < kScalars; ++x) {
          const int i = x * kMoveThreads + threadIdx.x;
          const int64_t to = p.to[i % kChunk];
          if (scalar(i) && to >= 0) scalar(i)[to] = *reinterpret_cast<const float*>(from + kAtScalars + i * 4);
        }
#pragma unroll
        for (int x = 0; x < kBlocks; ++x) {
          const int i = x * kMoveThreads + threadIdx.x;
          const int64_t to = p.to[i % kChunk];
          if (to >= 0) {
            const uint32_t* b = reinterpret_cast<const uint32_t*>(from + kAtBlocks + i * 8);
            uint32_t* q = reinterpret_cast<uint32_t*>(block_at(i, to));
            q[0] = b[0];
            if (D == 128) q[1] = b[1];
          }
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(done + now.at);
      now.next(kRing);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  if (warp == kMoveThreads / 32 + 1) {                     // ---- the tenth warp
    if (lane != 0) return;
    for (Turn now; tc::mbar_wait(placed + now.at, now.phase, &stop); now.next(kRing)) {
      int* const flags = places[now.at].flags;
      const int c = places[now.at].c;
      if (!flags || !tc::mbar_wait(read + now.at, now.phase, &stop)) return;
      // no fence: the copies have arrived, so no later write can reach them, and one would wait for the stores of
      // the chunks before
      asm volatile("st.relaxed.gpu.global.s32 [%0], %1;" :: "l"(flags + c), "r"(1) : "memory");
      tc::mbar_arrive(done + now.at);
    }
    return;
  }
  if (warp == kMoveThreads / 32 + 2) {                     // ---- the eleventh
    if (lane != 0) return;
    for (Turn now; tc::mbar_wait(placed + now.at, now.phase, &stop); now.next(kRing)) {
      Place& p = places[now.at];
      if (!p.flags) return;
      // at most two, and chunks before this one: their reading waits for nothing
      int ok = 1;
      uint64_t begin = 0;
      for (int x = p.first; x <= p.last && x < p.c && ok; ++x) {
        while (true) {
          asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(ok) : "l"(p.flags + x) : "memory");
          if (ok) break;
          const uint64_t t = global_timer_ns();
          if (begin == 0) begin = t;
          if (t - begin > kWaitLimitNs) break;
        }
      }
      if (!ok) {                                           // the CTA leaves: others wait as long at most
        raise_error(kErrTimeout);
        *(volatile int*)&stop = 1;
        return;
      }
      tc::mbar_arrive(free_ + now.at);
      tc::mbar_arrive(done + now.at);
    }
    return;
  }
  // ---- the ninth
  {
    int carry = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + lane;
      const int chunks = b < a.B && size[b].y < size[b].x ? (size[b].y + kChunk - 1) / kChunk : 0;
      int x = chunks;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b < a.B) prefix[b] = carry + x - chunks;
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) prefix[a.B] = carry;
    __syncwarp();
  }
  constexpr int kMine = (kChunk + 31) / 32;                // rows of a lane
  const int64_t total = (int64_t)prefix[a.B] * a.H, rows = a.num_pages * a.H * a.page;
  int round = 0;
#pragma unroll 1
  for (Turn now;; now.next(kRing), ++round) {
    if (round >= kRing && !tc::mbar_wait_warp(done + now.at, now.phase ^ 1, &stop)) return;
    Place& p = places[now.at];
    while (true) {
      const int t = __shfl_sync(0xffffffffu, ticket, 0);
      if (t >= total) {
        __syncwarp();
        if (lane == 0) {
          p.flags = nullptr;
          tc::mbar_arrive(placed + now.at);
        }
        return;
      }
      if (lane == 0) ticket = atomicAdd(l.ticket, 1);
      int lo = 0, hi = a.B - 1;                            // the last b with prefix[b] * H <= t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int64_t)prefix[mid] * a.H <= t) lo = mid; else hi = mid - 1;
      }
      const int b = lo, chunks = prefix[b + 1] - prefix[b], in_seq = t - prefix[b] * a.H;
      const int h = in_seq / chunks, c = in_seq - h * chunks;
      const int64_t item = (int64_t)b * a.H + h;
      const int2 z = size[b];
      const int r0 = c * kChunk, n = min(kChunk, z.y - r0);
      const int64_t* src = l.src + item * l.positions + r0;
      const int32_t* row = a.table + (int64_t)b * a.cols;
      const int* before = l.before + item * l.chunks + c;
      int64_t from[kMine], to[kMine];
#pragma unroll
      for (int x = 0; x < kMine; ++x) {
        const int i = min(lane + 32 * x, n - 1), col = (r0 + i) / a.page;
        from[x] = __ldg(src + i);
        to[x] = ((int64_t)__ldg(row + col) * a.H + h) * a.page + (r0 + i - col * a.page);
      }
      // ranks of the rows that lie in the chunk's places
      const int r = min(z.y, a.recent), old = z.x - r, k0 = z.y - r, end = min(r0 + kChunk, z.x);
      const int first = r0 < old ? __ldg(before) : k0 + r0 - old, last = (end < old ? __ldg(before + 1) : k0 + end - old) - 1;
      // positions rise and none lies below its rank: if the last stays where it is, all do
      if (__shfl_sync(0xffffffffu, from[kMine - 1] == to[kMine - 1], 31)) {
        if (lane == 0) asm volatile("st.relaxed.gpu.global.s32 [%0], %1;" :: "l"(l.read + item * l.chunks + c), "r"(1) : "memory");
        continue;
      }
#pragma unroll
      for (int x = 0; x < kMine; ++x) {
        const int i = lane + 32 * x;
        const bool moves = i < n && from[x] != to[x] && in_bounds(from[x], rows) && in_bounds(to[x], rows);
        if (i < kChunk) {
          p.from[i] = moves ? from[x] : -1;
          p.to[i] = moves ? to[x] : -1;
        }
      }
      __syncwarp();
      if (lane == 0) {
        p.flags = l.read + item * l.chunks;
        p.c = c;
        p.first = first / kChunk;
        p.last = last / kChunk;
        tc::mbar_arrive(placed + now.at);
      }
      break;
    }
  }
}

// ------------------------------------------------------------------ host

struct WsLayout { size_t size, ticket, before, read, src, total; int64_t positions, chunks; };
WsLayout ws_layout(const EvictArgs& a) {
  WsLayout w{};
  const int64_t b = a.B < kMaxBatch ? a.B : kMaxBatch, items = b * a.H;
  w.positions = (int64_t)a.cols * a.page;
  w.chunks = w.positions / 32 + 2;               // of the smallest chunk
  w.ticket = align256((size_t)b * sizeof(int2));
  w.before = w.ticket + 256;
  w.read = w.before + align256((size_t)(items * w.chunks) * 4);
  w.src = w.read + align256((size_t)(items * w.chunks) * 4);
  w.total = w.src + align256((size_t)(items * w.positions) * 8);
  return w;
}

// CTAs of a cluster for each (sequence, kv head): a unit a thread where two CTAs an
// SM allow it.
int cluster_of(const EvictArgs& a) {
  int c = 1;
  while (c < kMaxCtas && (int64_t)a.cols * a.page > (int64_t)c * kThreads * kUnit && (int64_t)a.B * a.H * c * 2 <= 152 * 2) c *= 2;
  return c;
}

int launch_failed(const char* what, cudaError_t err) {
  (void)cudaGetLastError();
  return set_error(ULYSSES_ERR_CUDA, "%s: launch failed: %s", what, cudaGetErrorString(err));
}

template <int kRowB, bool kFour, bool kScales>
cudaError_t move(const EvictArgs& a, const Lists& l, cudaStream_t st) {
  constexpr int kStages = stages_of(kRowB, kFour, kScales) * stage_bytes(kRowB, kFour, kScales);
  static PerDeviceOnce<> once;
  if (opt_in_smem(once, (const void*)evict_move_kernel<kRowB, kFour, kScales>,
                  kStages + kMaxBatch * (int)(sizeof(int2) + sizeof(int)) + 4, "cache_evict"))
    return cudaErrorInvalidValue;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(sms * 2));
  cfg.blockDim = dim3(kMovers);
  cfg.dynamicSmemBytes = kStages + a.B * sizeof(int2) + (a.B + 1) * sizeof(int);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_move_kernel<kRowB, kFour, kScales>, a, l);
}

cudaError_t move_rows(const EvictArgs& a, const Lists& l, cudaStream_t st) {
  const bool wide = a.D == 128;
  switch (a.cache_dtype) {
    case ULYSSES_E2M1: return wide ? move<64, true, true>(a, l, st) : move<32, true, true>(a, l, st);
    case ULYSSES_E4M3: return wide ? move<128, false, true>(a, l, st) : move<64, false, true>(a, l, st);
    case ULYSSES_BF16: return wide ? move<256, false, false>(a, l, st) : move<128, false, false>(a, l, st);
    default: return wide ? move<512, false, false>(a, l, st) : move<256, false, false>(a, l, st);
  }
}

}  // namespace

size_t evict_workspace(const EvictArgs& a) { return a.B == 0 ? 0 : ws_layout(a).total; }

int launch_evict(const EvictArgs& a, cudaStream_t st) {
  const WsLayout w = ws_layout(a);
  char* ws = (char*)a.ws;
  const int row_bytes = a.cache_dtype == ULYSSES_E2M1 ? a.D / 2 : (a.cache_dtype == ULYSSES_E4M3 ? a.D : elt_size(a.cache_dtype) * a.D);
  const Lists l{(int2*)(ws + w.size), (int*)(ws + w.ticket), (int64_t*)(ws + w.src), (int*)(ws + w.before), (int*)(ws + w.read),
                w.positions, w.chunks, chunk_of(row_bytes)};
  for (int b0 = 0; b0 < a.B; b0 += kMaxBatch) {
    EvictArgs x = a;
    x.B = a.B - b0 < kMaxBatch ? a.B - b0 : kMaxBatch;
    x.table = a.table + (int64_t)b0 * a.cols;
    x.lens = a.lens + b0;
    x.keep = a.keep + b0;
    x.out = a.out + b0;
    const int c = cluster_of(x);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((int64_t)x.B * x.H * c));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)c;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaError_t err = cudaLaunchKernelEx(&cfg, evict_select_kernel, x, l, c);
    if (err != cudaSuccess) return launch_failed("cache_evict", err);
    count_launch();
    err = move_rows(x, l, st);
    if (err != cudaSuccess) return launch_failed("cache_evict move", err);
    count_launch();
  }
  return ULYSSES_OK;
}

}  // namespace ulysses
