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
// finds the smallest weight that stays by its bits, three digits from the top (10,
// 11 and 11 bits), each from a histogram over the cluster, and writes the list of
// the rows that stay.  Weights are ordered as unsigned numbers (sign and magnitude
// made monotone; -0 as +0, NaN above everything).  Up to 16384 positions a CTA stay
// in shared memory from digit to digit.  Bound by latencies: launch, lengths,
// table, weights, and 2 us a digit, of which the largest is counting (the hardware
// adds to one word at a time; neighbouring lanes therefore have counts of their own
// in the first digit, where weights lie in few bins).  4160 positions of 128 heads
// take 12 us, 131072 of 8 in 8 CTAs each 23, of which 2.5 would be reading them.
// Loops are kept rolled and everything twice needed has one place: a launch runs
// each instruction a few times, and fetching them is what it waited for (16 weights
// in registers, each step written out: 16 and 25 us).  A warp writes the rows of two
// units side by side (each lane its own unit's, 128 bytes apart: 2 us more).
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
// wrote; as it is, two chunks ahead, the flags are there when they are asked for.
// How far ahead goes by what a kind of row takes: one chunk (e4m3 rows of 128) to
// five (4 bits of D = 64).  48 sequences cut from 4160 to 4096 tokens of 8 heads, the
// move alone: bf16 264 us (1.62 GB, 91% of the copy rate), 24 in fp32 of D = 64 135 (89%),
// e4m3 148 (0.84 GB, 84%; in chunks of half the rows, four of them ahead, 30 us more), 4 bits
// 105 (0.49 GB, 69%), e4m3 of D = 64 103 (63%) and 4 bits of it 94 (0.26 GB, 41%: as
// many rows, scales and places to look up for a third of the bytes).
// What the ring takes of shared memory, so that two CTAs fit an SM, and with it the
// sequences of a launch, is worked out in evict_ring.h.
#include <atomic>

#include "evict_ring.h"
#include "internal.h"
#include "rows.cuh"
#include "tc_ptx.cuh"

namespace ulysses {

ULYSSES_ERROR_READER(read_error_cache_evict)

namespace {

using namespace rows;
using namespace evict;

constexpr int kUnit = 16;          // positions of one thread at a time
constexpr int kThreads = 512;      // of a selecting CTA
constexpr int kBins = 4096;        // counts of a digit: 1024 of 10 bits by four neighbours, 2048 of 11 by two
constexpr int kMaxCtas = 8;        // of a cluster

// What the selection leaves for the move (workspace).
struct Lists {
  int2* size;      // [B] (tokens before, tokens that stay); equal where nothing moves
  int* ticket;     // chunks taken
  int64_t* src;    // [B][H][positions] rows of the positions that stay, rising (rows: [num_pages][H][page])
  int* before;     // [B][H][chunks] how many of those lie before position chunk * c
  int* read;       // [B][H][chunks] 1: the chunk's rows have been read
  int64_t positions, chunks;
  int chunk;       // rows moved together
};

// A weight as a number whose order is the weights'.
__device__ __forceinline__ uint32_t order_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);             // -0 + 0 = +0
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct Size { int n, m, r, pages; };
// Tokens, those that stay, those of them that stay for their age, pages that hold
// them.  A length that the table cannot hold is reported, and such a sequence is left
// as it is (none of its pages is looked up).
__device__ __forceinline__ Size size_of(const EvictArgs& a, int b) {
  const int n = __ldg(a.lens + b), keep = __ldg(a.keep + b);
  if (n < 0 || n > (int64_t)a.cols * a.page) {
    raise_error(kErrPages);
    return Size{n, n, 0, 0};
  }
  const int m = keep < 0 || keep > n ? n : keep;
  return Size{n, m, min(m, a.recent), (n + a.page - 1) / a.page};
}

__device__ __forceinline__ int ld_cluster(const int* at, int rank) {   // `at` in this CTA's shared memory
  uint32_t p;
  int v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(tc::smem_u32(at)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ int4 ld_cluster4(const int* at, int rank) {
  uint32_t p;
  int4 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(tc::smem_u32(at)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.s32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
  return v;
}

// Of the CTA `rank`, or of the one CTA.
__device__ __forceinline__ int4 ld4(const int* at, int rank, int ctas) {
  return ctas > 1 ? ld_cluster4(at, rank) : *reinterpret_cast<const int4*>(at);
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

// Of 128 counts, four a lane, the one in which the k-th from the top lies (1 <= k
// <= their sum), for all lanes: its number, how many lie above it and in it.
struct Found { int at, above, count; };
__device__ __forceinline__ Found find(int4 n, int k) {
  const int lane = threadIdx.x & 31, own = n.x + n.y + n.z + n.w;
  int upto = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_down_sync(0xffffffffu, upto, o);
    if (lane + o < 32) upto += y;
  }
  Found f{4 * lane + 3, upto - own, n.w};
  if (f.above + f.count < k) { --f.at; f.above += f.count; f.count = n.z; }
  if (f.above + f.count < k) { --f.at; f.above += f.count; f.count = n.y; }
  if (f.above + f.count < k) { --f.at; f.above += f.count; f.count = n.x; }
  const int from = __ffs(__ballot_sync(0xffffffffu, upto >= k && upto - own < k)) - 1;
  f.at = __shfl_sync(0xffffffffu, f.at, from);
  f.above = __shfl_sync(0xffffffffu, f.above, from);
  f.count = __shfl_sync(0xffffffffu, f.count, from);
  return f;
}

// Units of a thread that have a place in shared memory.  A CTA's positions stay
// there from digit to digit where that is enough; else they come again for each
// digit (from L2), one unit ahead.
constexpr int kSlots = 2;
constexpr int kSlotB = kThreads * kUnit * 4;

__global__ void __launch_bounds__(kThreads, 2) evict_select_kernel(const __grid_constant__ EvictArgs a,
                                                                   const __grid_constant__ Lists l, int ctas) {
  extern __shared__ __align__(16) uint4 slots[];           // [slot][thread][4]: weights, then their orders
  __shared__ __align__(16) int hist[kBins];
  __shared__ __align__(16) int part[kBins / 2];            // totals over the cluster, of this CTA's bins
  __shared__ __align__(16) int group[16];                  // and of a 16th of them each
  __shared__ int sums[kThreads / 32];
  __shared__ int mine[2];                                  // of this CTA's positions: above the threshold, at it
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31;
  const int rank = ctas > 1 ? (int)tc::cluster_ctarank() : 0, lg = __ffs(ctas) - 1, item = blockIdx.x >> lg;
  const int b = item / a.H, h = item - b * a.H;
  const int32_t* row = a.table + (int64_t)b * a.cols;
  int page[4];                                             // on their way beside the lengths
#pragma unroll
  for (int i = 0; i < 4; ++i) page[i] = tid + i * kThreads < a.cols ? __ldg(row + tid + i * kThreads) : 0;
  Size z = size_of(a, b);
  if (blockIdx.x == 0 && tid == 0) *l.ticket = 0;
  static_assert(kBins == 8 * kThreads, "");
  reinterpret_cast<int4*>(hist)[2 * tid] = reinterpret_cast<int4*>(hist)[2 * tid + 1] = make_int4(0, 0, 0, 0);
  if (tid < 2) mine[tid] = 0;
  // a page out of range: the sequence is left as it is, all of its heads (each looks at the whole row); where all
  // tokens stay anyway it is reported all the same
  int bad = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) bad |= tid + i * kThreads < z.pages && (unsigned)page[i] >= (unsigned)a.num_pages;
  for (int c = tid + 4 * kThreads; c < z.pages; c += kThreads) bad |= (unsigned)__ldg(row + c) >= (unsigned)a.num_pages;
  if (__syncthreads_or(bad)) {
    if (tid == 0) raise_error(kErrPages);
    z.m = z.n;
  }
  if (h == 0 && rank == 0 && tid == 0) l.size[b] = make_int2(z.n, z.m);
  if (z.m >= z.n) return;                                  // the whole cluster

  int64_t* src = l.src + item * l.positions;
  int* before = l.before + item * l.chunks;
  const int old = z.n - z.r, k = z.m - z.r;                // k of `old` positions stay
  const int units = (old + kUnit - 1) / kUnit, each = (units + ctas - 1) >> lg;
  const int u0 = min(rank * each, units), u1 = min(u0 + each, units);
  const int rounds = (u1 - u0 + kThreads - 1) / kThreads;  // units of a thread, at most
  const bool all = rounds <= kSlots;
  // the thread's `r`-th unit and its place in shared memory, where nobody else looks (16-byte words change places
  // so that no bank is met twice)
  const auto unit_of = [&](int r) { return u0 + r * kThreads + tid; };
  const auto row_of = [&](int p) {                         // of position p
    const int col = p / a.page;
    return ((int64_t)__ldg(row + col) * a.H + h) * a.page + (p - col * a.page);
  };
  const auto place = [&](int i) { return slots + (i * kThreads + tid) * 4; };
  const auto fetch = [&](int r, int i) {
    const int u = unit_of(r);
    if (u < u1) {
      const int64_t at = row_of(u * kUnit);
      const uint32_t to = tc::smem_u32(place(i));
      if (in_bounds(at, a.num_pages * a.H * a.page)) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(to + (j ^ (tid >> 1 & 3)) * 16), "l"(a.w + at + 4 * j) : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // the r-th unit's place, when its weights are there and (round about) the next one's on their way
  int turn = 0;
  const auto arrived = [&](int r) {
    if (all) return place(r);
    fetch(r + 1 < rounds ? r + 1 : 0, (turn + 1) & 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    return place(turn++ & 1);
  };
  // the orders of four of the unit's weights; `raw`: they are weights yet.  Places behind the last get 0, which is no
  // weight's order
  const auto four = [&](const uint4* slot, int j, int u, bool raw) {
    uint4 x = slot[j ^ (tid >> 1 & 3)];
    if (raw) {
      const int live = old - u * kUnit - 4 * j;
      x.x = live > 0 ? order_of(__uint_as_float(x.x)) : 0; x.y = live > 1 ? order_of(__uint_as_float(x.y)) : 0;
      x.z = live > 2 ? order_of(__uint_as_float(x.z)) : 0; x.w = live > 3 ? order_of(__uint_as_float(x.w)) : 0;
    }
    return x;
  };
  if (k > 0) {
#pragma unroll
    for (int r = 0; r < kSlots; ++r)
      if (r < (all ? rounds : 1)) fetch(r, r);
  }
  for (int i = rank * kThreads + tid; i < (z.m + l.chunk - 1) / l.chunk; i += ctas * kThreads) l.read[item * l.chunks + i] = 0;
  for (int i = rank * kThreads + tid; i < z.r; i += ctas * kThreads) src[k + i] = row_of(old + i);
  if (all) asm volatile("cp.async.wait_all;" ::: "memory");

  // the threshold, digit by digit: `prefix` holds the bits found, k_left of the
  // positions that have them are to stay
  uint32_t prefix = 0;
  int k_left = k;
  if (k > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      // bins lie 2^fold apart, and neighbouring lanes count in places of their own
      const int shift = pass == 0 ? 22 : (pass == 1 ? 11 : 0), bits = pass == 0 ? 10 : 11, fold = pass == 0 ? 2 : 1;
      int* const own = hist + (tid & ((1 << fold) - 1));
#pragma unroll 1
      for (int r = 0; r < rounds; ++r) {
        uint4* const slot = arrived(r);
        const int u = unit_of(r);
        if (u >= u1) continue;
#pragma unroll 2
        for (int j = 0; j < 4; ++j) {
          const uint4 x = four(slot, j, u, pass == 0 || !all);
          if (pass == 0 && all) slot[j ^ (tid >> 1 & 3)] = x;
          // those with the digits found so far; four of one bin are counted together: tokens nobody looked at are alike
          const uint32_t top = pass == 0 ? 0 : 0xffffffffu << (shift + bits), want = pass == 0 ? 0 : prefix << (shift + bits);
          const bool in[4] = {(x.x & top) == want, (x.y & top) == want, (x.z & top) == want, (x.w & top) == want};
          if (!(in[0] || in[1] || in[2] || in[3])) continue;
          const uint32_t mask = (1u << bits) - 1, d = x.x >> shift & mask;
          if (x.x >> shift == x.y >> shift && x.x >> shift == x.z >> shift && x.x >> shift == x.w >> shift) {
            atomicAdd(own + (d << fold), 4);
          } else {
            if (in[0]) atomicAdd(own + (d << fold), 1);
            if (in[1]) atomicAdd(own + ((x.y >> shift & mask) << fold), 1);
            if (in[2]) atomicAdd(own + ((x.z >> shift & mask) << fold), 1);
            if (in[3]) atomicAdd(own + ((x.w >> shift & mask) << fold), 1);
          }
        }
      }
      sync_all(ctas);
      // each CTA adds up its share of the counts over the cluster, four of them a thread (eight where it is alone) ..
      const int share = kBins >> lg, wide = ctas == 1 ? 5 : 6 - lg;   // 2^wide threads of a 16th
      int sum = 0;
      const auto add = [&](int i, int4 v) {
        const int lo = v.x + v.y, hi = v.z + v.w;
        if (fold == 2) part[i] = lo + hi;
        else reinterpret_cast<int2*>(part)[i] = make_int2(lo, hi);
        sum += lo + hi;
      };
      if (ctas == 1) {
        add(2 * tid, reinterpret_cast<const int4*>(hist)[2 * tid]);
        add(2 * tid + 1, reinterpret_cast<const int4*>(hist)[2 * tid + 1]);
      } else if (4 * tid < share) {
        int4 v[kMaxCtas];
#pragma unroll
        for (int c = 0; c < kMaxCtas; ++c) v[c] = c < ctas ? ld_cluster4(hist + rank * share + 4 * tid, c) : make_int4(0, 0, 0, 0);
#pragma unroll
        for (int c = 1; c < kMaxCtas; ++c) {
          v[0].x += v[c].x; v[0].y += v[c].y; v[0].z += v[c].z; v[0].w += v[c].w;
        }
        add(tid, v[0]);
      }
      for (int o = 1 << wide >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if ((tid & ((1 << wide) - 1)) == 0 && tid >> wide < 16) group[tid >> wide] = sum;
      sync_all(ctas);
      // .. and every warp finds the 16th of a share that has the digit, and the digit in it
      const Found g = find(lane < 4 * ctas ? ld4(group + lane % 4 * 4, lane / 4, ctas) : make_int4(0, 0, 0, 0), k_left);
      const int bins = (share >> fold) / 16, owner = min(g.at / 16, ctas - 1), first = g.at % 16 * bins;
      const Found f = find(4 * lane < bins ? ld4(part + first + 4 * lane, owner, ctas) : make_int4(0, 0, 0, 0), k_left - g.above);
      const int digit = owner * (share >> fold) + first + f.at;
      k_left -= g.above + f.above;
      prefix = prefix << bits | (uint32_t)digit;
      // this CTA's above it, at last those at it, and the counts cleared for the next digit
      int4* const n = reinterpret_cast<int4*>(hist) + 2 * tid;
      if (ctas > 1) {
        int over = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int lo = n[i].x + n[i].y, hi = n[i].z + n[i].w, at = (8 * tid + 4 * i) >> fold, next = at + (fold == 1);
          over += (at > digit ? lo : 0) + (next > digit ? hi : 0);
          if (pass == 2 && at == digit) mine[1] = lo;
          if (pass == 2 && next == digit) mine[1] = hi;
        }
        over = __reduce_add_sync(0xffffffffu, over);
        if (lane == 0 && over) atomicAdd(mine, over);
      }
      n[0] = n[1] = make_int4(0, 0, 0, 0);
      __syncthreads();
    }
  }
  // positions that stay before this CTA's: those above the threshold and the first k_left at it
  int gt0 = 0, eq0 = 0;
  if (ctas > 1) {
    sync_all(ctas);
    int g = 0, e = 0;
    if (lane < rank) {
      g = ld_cluster(mine, lane);
      e = ld_cluster(mine + 1, lane);
    }
    gt0 = __reduce_add_sync(0xffffffffu, g);
    eq0 = __reduce_add_sync(0xffffffffu, e);
    // no CTA leaves while another reads its shared memory
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }
#pragma unroll 1
  for (int r = 0; r < rounds; ++r) {
    const int u = unit_of(r);
    uint32_t gt = 0, eq = 0;                               // a bit a position
    if (k > 0) {
      const uint4* slot = arrived(r);
      if (u < u1) {
#pragma unroll 2
        for (int j = 0; j < 4; ++j) {
          const uint4 x = four(slot, j, u, !all);
          gt |= ((x.x > prefix) + 2 * (x.y > prefix) + 4 * (x.z > prefix) + 8 * (x.w > prefix)) << 4 * j;
          eq |= ((x.x == prefix) + 2 * (x.y == prefix) + 4 * (x.z == prefix) + 8 * (x.w == prefix)) << 4 * j;
        }
      }
    }
    const int first = gt | eq ? (int)(row_of(u * kUnit) / kUnit) : 0;   // the unit's rows (of 36 bytes or more: 31 bits)
    int total;
    const int counts = __popc(gt) | __popc(eq) << 16;      // at most 8192 of each
    const int upto = block_scan(counts, sums, total) - counts;
    const int g = gt0 + (upto & 0xffff), e = eq0 + (upto >> 16);
    int at = 0;
    uint32_t stay = 0;
    if (u < u1) {
      at = g + min(e, k_left);
      if ((u * kUnit & (l.chunk - 1)) == 0) before[u * kUnit >> (__ffs(l.chunk) - 1)] = at;
      // the first of those at it, as many as are left
      for (int over = __popc(eq) - max(k_left - e, 0); over > 0; --over) eq &= ~(0x80000000u >> __clz(eq));
      stay = gt | eq;
    }
    if (__reduce_max_sync(0xffffffffu, __popc(stay)) <= 4) {
#pragma unroll 1
      for (; stay && at < k; stay &= stay - 1, ++at) src[at] = (int64_t)first * kUnit + __ffs(stay) - 1;
    } else {                                               // many: the rows of two units at a time, side by side
#pragma unroll 4
      for (int i = 0; i < 32; i += 2) {
        const int from = i + (lane >> 4), bit = lane & 15;
        const uint32_t its = __shfl_sync(0xffffffffu, stay, from);
        const int to = __shfl_sync(0xffffffffu, at, from) + __popc(its & ((1u << bit) - 1));
        const int its_first = __shfl_sync(0xffffffffu, first, from);
        if ((its >> bit & 1) && to < k) src[to] = (int64_t)its_first * kUnit + bit;
      }
    }
    gt0 += total & 0xffff;
    eq0 += total >> 16;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (ctas > 1) {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
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
__global__ void __launch_bounds__(kMovers, kCtasAnSm) evict_move_kernel(const __grid_constant__ EvictArgs a,
                                                                const __grid_constant__ Lists l) {
  constexpr int kChunk = chunk_of(kRowB);
  constexpr int kW = kRowB / 16;                           // words of a row
  constexpr int kOwn = own_words(kRowB), kScalars = own_scalars(kRowB, kScales), kBlocks = own_blocks(kRowB, kFour);
  constexpr int kStages = stages_of(kRowB, kFour, kScales), kStageB = stage_bytes(kRowB, kFour, kScales);
  constexpr int kRing = ring_of(kStages);                  // chunks whose places are known
  constexpr int D = kRowB * 2;                             // kFour
  static_assert(kOwn >= 1 && kStages >= 2 && (kChunk & (kChunk - 1)) == 0 && kChunk % kUnit == 0, "");
  static_assert(cta_bytes(kRowB, kFour, kScales, kStages, batch_of(kRowB, kFour, kScales)) * kCtasAnSm <= kSmBytes,
                "two CTAs an SM, as the launch takes for granted");
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

// Clusters of 2^lg selecting CTAs that the current device holds at once (with all
// their slots), asked for once a device.  A GPC's SMs are no multiple of a cluster's:
// with two CTAs an SM 36 clusters of eight, where 304 CTAs would be 38.
int clusters_at_once(int lg) {
  static std::atomic<int> known[64][4];                    // 0: not yet asked
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if ((n = known[dev][lg].load(std::memory_order_relaxed)) != 0) return n;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(1u << lg);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSlots * kSlotB;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1u << lg;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, evict_select_kernel, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    n = 0;
  }
  if (n > 0) known[dev][lg].store(n, std::memory_order_relaxed);
  return n;
}

// CTAs of a cluster for each (sequence, kv head): a unit a thread where two CTAs an
// SM allow it.  (Four and eight an SM: 64 ragged sequences of up to 16384 positions,
// 8 heads, 246 and 265 us where this takes 238, 16 of 40000 207 and 207 where it
// takes 181; a CTA for each head: 1 x 131072 positions 126 where it takes 35.)
// Where the wider clusters would not all run at once, the last of them adding a
// selection's time, the narrower are taken if their CTAs hold the positions from
// digit to digit (38 heads of 40000 in fours 36 us, in eights 45; 76 of 20000 in
// pairs 33, in fours 43), else the wider (38 of 131072 in eights 57, in fours 82).
int cluster_of(const EvictArgs& a, int sms) {
  const int64_t positions = (int64_t)a.cols * a.page, items = (int64_t)a.B * a.H;
  int lg = 0;
  while (lg < 3 && positions > (int64_t)kThreads * kUnit << lg &&
         (items <= clusters_at_once(lg + 1) ||
          (items << (lg + 1) <= 2 * sms && positions > (int64_t)kSlots * kThreads * kUnit << lg)))
    ++lg;
  return 1 << lg;
}

int launch_failed(const char* what, cudaError_t err) {
  (void)cudaGetLastError();
  return set_error(ULYSSES_ERR_CUDA, "%s: launch failed: %s", what, cudaGetErrorString(err));
}

template <int kRowB, bool kFour, bool kScales>
cudaError_t move(const EvictArgs& a, const Lists& l, int sms, cudaStream_t st) {
  constexpr int kStages = stages_of(kRowB, kFour, kScales) * stage_bytes(kRowB, kFour, kScales), kBatch = batch_of(kRowB, kFour, kScales);
  static PerDeviceOnce<> once;
  if (opt_in_smem(once, (const void*)evict_move_kernel<kRowB, kFour, kScales>, kStages + batch_bytes(kBatch), "cache_evict"))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(sms * kCtasAnSm));
  cfg.blockDim = dim3(kMovers);
  cfg.dynamicSmemBytes = kStages + batch_bytes(a.B);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_move_kernel<kRowB, kFour, kScales>, a, l);
}

cudaError_t move_rows(const EvictArgs& a, const Lists& l, int sms, cudaStream_t st) {
  const bool wide = a.D == 128;
  switch (a.cache_dtype) {
    case ULYSSES_E2M1: return wide ? move<64, true, true>(a, l, sms, st) : move<32, true, true>(a, l, sms, st);
    case ULYSSES_E4M3: return wide ? move<128, false, true>(a, l, sms, st) : move<64, false, true>(a, l, sms, st);
    case ULYSSES_BF16: return wide ? move<256, false, false>(a, l, sms, st) : move<128, false, false>(a, l, sms, st);
    default: return wide ? move<512, false, false>(a, l, sms, st) : move<256, false, false>(a, l, sms, st);
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
  const bool four = a.cache_dtype == ULYSSES_E2M1;
  const int most = batch_of(row_bytes, four, four || a.cache_dtype == ULYSSES_E4M3), launches = (a.B + most - 1) / most;
  const int batch = (a.B + launches - 1) / launches;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  for (int b0 = 0; b0 < a.B; b0 += batch) {
    EvictArgs x = a;
    x.B = a.B - b0 < batch ? a.B - b0 : batch;
    x.table = a.table + (int64_t)b0 * a.cols;
    x.lens = a.lens + b0;
    x.keep = a.keep + b0;
    x.out = a.out + b0;
    static PerDeviceOnce<> once;
    if (const int rc = opt_in_smem(once, (const void*)evict_select_kernel, kSlots * kSlotB, "cache_evict")) return rc;
    const int c = cluster_of(x, sms);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((int64_t)x.B * x.H * c));
    cfg.blockDim = dim3(kThreads);
    // places for the units of a full table, as far as there are any
    const int64_t each = ((int64_t)x.cols * x.page / kUnit + c - 1) / c, rounds = (each + kThreads - 1) / kThreads;
    cfg.dynamicSmemBytes = (size_t)(rounds < kSlots ? rounds : kSlots) * kSlotB;
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
    err = move_rows(x, l, sms, st);
    if (err != cudaSuccess) return launch_failed("cache_evict move", err);
    count_launch();
  }
  return ULYSSES_OK;
}

}  // namespace ulysses
