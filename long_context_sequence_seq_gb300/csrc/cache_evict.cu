// Eviction from the paged cache by accumulated attention weight
// (include/ulysses.h, ulysses_cache_evict).
//
// Of a sequence's n tokens m = min(n, keep) stay, for every kv head its own: the
// last r = min(m, recent), and of the n - r before them the m - r of greatest
// weight (the lower position first among equals).  They close up in their order,
// so position i of what is left is the i-th token that stays, and the places from
// m on are left as they were.
//
// Two kernels.  The first selects: a cluster of CTAs for each (sequence, kv
// head) finds the smallest weight that stays by its bits, three digits from the
// top, each from a histogram over the cluster, and writes the list of the
// positions that stay.  Weights are ordered as unsigned numbers (sign and
// magnitude made monotone; -0 as +0, NaN above everything).
//
// The second moves rows, in place: chunks of kChunk rows, K, V, scales and
// weights, are read into registers and written kChunk places together.  A row
// never moves up, so what a chunk overwrites are rows of itself and of at most
// two chunks before it: it waits until those have been read.  CTAs take chunks
// by a counter, in order; a chunk's reading waits for nothing, so the first
// chunk that is not done can always go on.  Every kept row is read and written
// once, which is all the memory traffic there is beside the weights'.
#include "internal.h"
#include "rows.cuh"
#include "tc_ptx.cuh"

namespace ulysses {

ULYSSES_ERROR_READER(read_error_cache_evict)

namespace {

using namespace rows;

constexpr int kUnit = 16;          // positions of one thread at a time
constexpr int kThreads = 512;      // of a selecting CTA
constexpr int kChunk = 64;         // rows moved together
constexpr int kMoveThreads = 256;
constexpr int kMaxBatch = 2048;    // sequences of one launch (their prefix sums sit in shared memory)
constexpr int kBins = 2048;        // of a digit of 11 bits

// What the selection leaves for the move (workspace).
struct Lists {
  int2* size;      // [B] (tokens before, tokens that stay); equal where nothing moves
  int* ticket;     // chunks taken
  int* src;        // [B][H][positions] positions that stay, rising
  int* before;     // [B][H][chunks] how many of those lie before position kChunk * c
  int* read;       // [B][H][chunks] 1: the chunk's rows have been read
  int64_t positions, chunks;
};

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

__global__ void __launch_bounds__(kThreads) evict_select_kernel(const __grid_constant__ EvictArgs a,
                                                                const __grid_constant__ Lists l, int ctas) {
  __shared__ int hist[kBins];
  __shared__ int sums[kThreads / 32];
  __shared__ int found[2];                                 // the digit, and how many of the chosen lie above it
  __shared__ int mine[2];                                  // of this CTA's positions: above the threshold, at it
  const int rank = ctas > 1 ? (int)tc::cluster_ctarank() : 0, item = blockIdx.x / ctas;
  const int b = item / a.H, h = item - b * a.H;
  const int32_t* row = a.table + (int64_t)b * a.cols;
  Size z = size_of(a, b);
  if (blockIdx.x == 0 && threadIdx.x == 0) *l.ticket = 0;
  // a page out of range: the sequence is left as it is, all of its heads (each looks at the whole row)
  int bad = 0;
  if (z.m < z.n)
    for (int c = threadIdx.x; c < (z.n + a.page - 1) / a.page; c += kThreads) bad |= (unsigned)__ldg(row + c) >= (unsigned)a.num_pages;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) raise_error(kErrPages);
    z.m = z.n;
  }
  if (h == 0 && rank == 0 && threadIdx.x == 0) l.size[b] = make_int2(z.n, z.m);
  if (z.m >= z.n) return;                                  // the whole cluster
  int* src = l.src + item * l.positions;
  int* before = l.before + item * l.chunks;
  const int old = z.n - z.r, k = z.m - z.r;                // k of `old` positions stay
  for (int i = rank * kThreads + threadIdx.x; i < (z.m + kChunk - 1) / kChunk; i += ctas * kThreads) l.read[item * l.chunks + i] = 0;
  for (int i = rank * kThreads + threadIdx.x; i < z.r; i += ctas * kThreads) src[k + i] = old + i;
  const int units = (old + kUnit - 1) / kUnit, each = (units + ctas - 1) / ctas;
  const int u0 = min(rank * each, units), u1 = min(u0 + each, units);

  // the threshold, digit by digit: `prefix` holds the bits found, k_left of the
  // positions that have them are to stay
  uint32_t prefix = 0;
  int k_left = k, above = 0, at_it = 0;
  if (k > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
      for (int i = threadIdx.x; i < kBins; i += kThreads) hist[i] = 0;
      __syncthreads();
      for (int u = u0 + threadIdx.x; u < u1; u += kThreads) {
        uint32_t key[kUnit];
        load_unit(a, row, h, u, key);
        const int live = old - u * kUnit;
        // neighbours of one bin are counted together: tokens nobody looked at are alike
        int bin = -1, count = 0;
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
          if (i >= live || (pass > 0 && key[i] >> (shift + bits) != prefix)) continue;
          const int d = (int)(key[i] >> shift) & ((1 << bits) - 1);
          if (d == bin) { ++count; continue; }
          if (count) atomicAdd(hist + bin, count);
          bin = d;
          count = 1;
        }
        if (count) atomicAdd(hist + bin, count);
      }
      __syncthreads();
      if (ctas > 1) tc::cluster_sync();
      // thread t has the bins kBins - 1 - 4t - i: sums from the top
      constexpr int kOwn = kBins / kThreads;
      int n[kOwn], sum = 0;
      const uint32_t hist_at = tc::smem_u32(hist);
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int bin = kBins - 1 - ((int)threadIdx.x * kOwn + i);
        n[i] = 0;
        if (ctas > 1)
          for (int c = 0; c < ctas; ++c) n[i] += ld_cluster(hist_at + bin * 4, c);
        else
          n[i] = hist[bin];
        sum += n[i];
      }
      int total;
      int upto = block_scan(sum, sums, total) - sum;       // positions in the bins above
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        if (upto < k_left && upto + n[i] >= k_left) {      // one thread, once
          found[0] = kBins - 1 - ((int)threadIdx.x * kOwn + i);
          found[1] = upto;
        }
        upto += n[i];
      }
      __syncthreads();
      const int digit = found[0];
      k_left -= found[1];
      prefix = prefix << bits | (uint32_t)digit;
      int own = 0;
      for (int i = threadIdx.x; i < kBins; i += kThreads) own += i > digit ? hist[i] : 0;
      (void)block_scan(own, sums, total);
      above += total;
      at_it = hist[digit];
      __syncthreads();
      if (ctas > 1) tc::cluster_sync();                    // no histogram is cleared while another CTA reads it
    }
  }
  // positions that stay before this CTA's: those above the threshold and the first k_left at it
  int gt0 = 0, eq0 = 0;
  if (ctas > 1) {
    if (threadIdx.x == 0) { mine[0] = above; mine[1] = at_it; }
    __syncthreads();
    tc::cluster_sync();
    const uint32_t mine_at = tc::smem_u32(mine);
    for (int c = 0; c < rank; ++c) {
      gt0 += ld_cluster(mine_at, c);
      eq0 += ld_cluster(mine_at + 4, c);
    }
    tc::cluster_sync();                                    // no CTA leaves while another reads its counts
  }
  for (int t = u0; t < u1; t += kThreads) {
    const int u = t + threadIdx.x;
    uint32_t key[kUnit];
    uint32_t gt = 0, eq = 0;                               // a bit a position
    if (u < u1 && k > 0) {
      load_unit(a, row, h, u, key);
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
    int g = gt0 + (upto & 0xffff), e = eq0 + (upto >> 16);
    if (u < u1) {
      if (u % (kChunk / kUnit) == 0) before[u / (kChunk / kUnit)] = g + min(e, k_left);
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
        const bool is_gt = gt >> i & 1, is_eq = eq >> i & 1;
        if (is_gt || (is_eq && e < k_left)) {
          const int at = g + min(e, k_left);
          if (in_bounds(at, k)) src[at] = u * kUnit + i;
        }
        g += is_gt;
        e += is_eq;
      }
    }
    gt0 += total & 0xffff;
    eq0 += total >> 16;
  }
}

// Moves the rows that stay.  kRowB: bytes of a row's values or codes.
template <int kRowB, bool kFour, bool kScales>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictArgs a,
                                                                  const __grid_constant__ Lists l) {
  constexpr int kW = kRowB / 16;                           // words of a row
  constexpr int kOwn = 2 * kChunk * kW / kMoveThreads;     // words of a thread: K's and V's of a chunk
  constexpr int D = kRowB * 2;                             // kFour
  static_assert(kOwn >= 1, "");
  extern __shared__ int prefix[];                          // chunks of the sequences before, of one head
  __shared__ int64_t from[kChunk], to[kChunk];
  __shared__ int from_slot[kChunk], to_slot[kChunk];
  __shared__ int next_chunk, go;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // each warp adds up a part of the sequences' chunks
  for (int b = threadIdx.x; b < a.B; b += kMoveThreads) {
    const int2 z = l.size[b];
    prefix[b + 1] = z.y < z.x ? (z.y + kChunk - 1) / kChunk : 0;
    if (blockIdx.x == 0) a.out[b] = z.y;
  }
  if (threadIdx.x == 0) {
    prefix[0] = 0;
    next_chunk = atomicAdd(l.ticket, 1);
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int carry = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + threadIdx.x;
      int x = b < a.B ? prefix[b + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if ((int)threadIdx.x >= o) x += y;
      }
      if (b < a.B) prefix[b + 1] = carry + x;
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
  const int64_t total = (int64_t)prefix[a.B] * a.H, rows = a.num_pages * a.H * a.page;
  while (true) {
    const int t = next_chunk;
    __syncthreads();                                       // all have it, and the last chunk's places are done with
    if (t >= total) return;
    if (threadIdx.x == 0) next_chunk = atomicAdd(l.ticket, 1);
    int lo = 0, hi = a.B - 1;                              // the last b with prefix[b] * H <= t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)prefix[mid] * a.H <= t) lo = mid; else hi = mid - 1;
    }
    const int b = lo, chunks = prefix[b + 1] - prefix[b], in_seq = t - prefix[b] * a.H;
    const int h = in_seq / chunks, c = in_seq - h * chunks;
    const int64_t item = (int64_t)b * a.H + h;
    const int2 z = l.size[b];
    const int r0 = c * kChunk, n = min(kChunk, z.y - r0);
    const int* src = l.src + item * l.positions;
    int* read = l.read + item * l.chunks;
    if (__ldg(src + r0 + n - 1) == r0 + n - 1) {           // positions rise and none lies below its rank: none moves
      if (threadIdx.x == 0) asm volatile("st.release.gpu.global.s32 [%0], %1;" :: "l"(read + c), "r"(1) : "memory");
      __syncthreads();                                     // the next chunk's number is there
      continue;
    }
    // threads 0-63 find where the rows are, 64-127 where they go
    if ((int)threadIdx.x < 2 * kChunk) {
      const int i = threadIdx.x % kChunk, side = threadIdx.x / kChunk;
      int64_t place = -1;
      int slot = 0;
      if (i < n) {
        const int s = __ldg(src + r0 + i), p = side ? r0 + i : s;
        const int col = p / a.page;
        slot = p - col * a.page;
        place = ((int64_t)__ldg(a.table + (int64_t)b * a.cols + col) * a.H + h) * a.page + slot;
        if (s == r0 + i || !in_bounds(place, rows)) place = -1;
      }
      (side ? to : from)[i] = place;
      (side ? to_slot : from_slot)[i] = slot;
    }
    __syncthreads();
    // K's words and then V's; word i of the chunk is word i % kW of row i / kW
    uint4 w[kOwn];
#pragma unroll
    for (int x = 0; x < kOwn; ++x) {
      const int i = x * kMoveThreads + threadIdx.x, k = i / kW % kChunk;
      const char* base = static_cast<const char*>(i >= kChunk * kW ? a.vc : a.kc);
      if (from[k] >= 0 && to[k] >= 0)
        w[x] = ld16(base + (kFour ? e2m1_codes(from[k], from_slot[k], D) : from[k] * kRowB) + i % kW * 16);
    }
    float f[3];
    uint32_t blocks[2];
    const int k = threadIdx.x % kChunk, which = threadIdx.x / kChunk;   // threads 0-63 weights, 64-127 K's scales, 128-191 V's
    const bool moves = from[k] >= 0 && to[k] >= 0;
    float* const scalars = which == 0 ? a.w : (kScales ? (which == 1 ? a.ks : (which == 2 ? a.vs : nullptr)) : nullptr);
    if (moves && scalars) f[0] = *reinterpret_cast<const volatile float*>(scalars + from[k]);
    if (kFour && moves && which < 2) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(static_cast<const char*>(which ? a.vc : a.kc) +
                                                            e2m1_blocks(from[k], from_slot[k], a.page, D));
      blocks[0] = ld4(p);
      if (D == 128) blocks[1] = ld4(p + 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      asm volatile("st.release.gpu.global.s32 [%0], %1;" :: "l"(read + c), "r"(1) : "memory");
      // ranks of the rows that lie in the chunk's places
      const int old = z.x - min(z.y, a.recent), k0 = z.y - min(z.y, a.recent);
      const int* before = l.before + item * l.chunks;
      const int first = r0 < old ? __ldg(before + c) : k0 + r0 - old;
      const int end = min(r0 + kChunk, z.x);
      const int last = (end < old ? __ldg(before + c + 1) : k0 + end - old) - 1;
      int ok = 1;
      for (int x = first / kChunk; x <= last / kChunk && x < c; ++x) {
        int v;
        uint64_t begin = 0;
        while (true) {
          asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(read + x) : "memory");
          if (v) break;
          const uint64_t now = global_timer_ns();
          if (begin == 0) begin = now;
          if (now - begin > kWaitLimitNs) break;
        }
        ok &= v;
      }
      if (!ok) raise_error(kErrTimeout);
      go = ok;
    }
    __syncthreads();
    if (!go) continue;
#pragma unroll
    for (int x = 0; x < kOwn; ++x) {
      const int i = x * kMoveThreads + threadIdx.x, k = i / kW % kChunk;
      char* base = static_cast<char*>(i >= kChunk * kW ? a.vc : a.kc);
      if (from[k] >= 0 && to[k] >= 0)
        st16(base + (kFour ? e2m1_codes(to[k], to_slot[k], D) : to[k] * kRowB) + i % kW * 16, w[x]);
    }
    if (moves && scalars) scalars[to[k]] = f[0];
    if (kFour && moves && which < 2) {
      uint32_t* p = reinterpret_cast<uint32_t*>(static_cast<char*>(which ? a.vc : a.kc) + e2m1_blocks(to[k], to_slot[k], a.page, D));
      p[0] = blocks[0];
      if (D == 128) p[1] = blocks[1];
    }
  }
}

// ------------------------------------------------------------------ host

struct WsLayout { size_t size, ticket, before, read, src, total; int64_t positions, chunks; };
WsLayout ws_layout(const EvictArgs& a) {
  WsLayout w{};
  const int64_t b = a.B < kMaxBatch ? a.B : kMaxBatch, items = b * a.H;
  w.positions = (int64_t)a.cols * a.page;
  w.chunks = w.positions / kChunk + 2;
  w.ticket = align256((size_t)b * sizeof(int2));
  w.before = w.ticket + 256;
  w.read = w.before + align256((size_t)(items * w.chunks) * 4);
  w.src = w.read + align256((size_t)(items * w.chunks) * 4);
  w.total = w.src + align256((size_t)(items * w.positions) * 4);
  return w;
}

// CTAs of a cluster for each (sequence, kv head): as many as two an SM allow, and no
// more than there are positions for.
int cluster_of(const EvictArgs& a) {
  int c = 8;
  while (c > 1 && ((int64_t)a.B * a.H * c > 152 * 2 || (int64_t)a.cols * a.page < (int64_t)c * kThreads * 4)) c /= 2;
  return c;
}

int launch_failed(const char* what, cudaError_t err) {
  (void)cudaGetLastError();
  return set_error(ULYSSES_ERR_CUDA, "%s: launch failed: %s", what, cudaGetErrorString(err));
}

template <int kRowB, bool kFour, bool kScales>
cudaError_t move(const EvictArgs& a, const Lists& l, cudaStream_t st) {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(sms * 6));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = (a.B + 1) * sizeof(int);
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
  const Lists l{(int2*)(ws + w.size), (int*)(ws + w.ticket), (int*)(ws + w.src), (int*)(ws + w.before), (int*)(ws + w.read),
                w.positions, w.chunks};
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
