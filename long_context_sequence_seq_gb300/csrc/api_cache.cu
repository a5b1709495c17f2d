// C ABI of the rotary positions, the paged cache and single-token attention:
// argument validation and dispatch (the kernels are in rope.cu, kv_cache.cu
// and attn_decode.cu).
#include <cmath>

#include "common.cuh"
#include "internal.h"

using namespace ulysses;

namespace {

constexpr int64_t kMaxTokens = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxPositions = (int64_t)1 << 30;   // of one sequence: positions and tile counts fit int32

int type_size(int dtype) { return dtype == ULYSSES_E4M3 ? 1 : elt_size(dtype); }

// One dimension of a strided tensor.
struct Dim { int64_t n, stride; };

// Elements from the first to past the last of a strided tensor of rows of D.
int64_t extent(const Dim* d, int nd, int D) {
  int64_t e = D;
  for (int i = 0; i < nd; ++i) e += (d[i].n - 1) * d[i].stride;
  return e;
}

// Strides: not negative, multiples of 16 bytes, extents far from 2^63.
int check_strides(const Dim* d, int nd, int elt, const char* what) {
  for (int i = 0; i < nd; ++i) {
    if (d[i].n > 1 && d[i].stride > ((int64_t)1 << 58) / d[i].n)
      return set_error(ULYSSES_ERR_UNSUPPORTED, "%s: stride %lld too large", what, (long long)d[i].stride);
    if (d[i].n > 1 && (d[i].stride < 0 || (d[i].stride * elt) % 16))
      return set_error(ULYSSES_ERR_UNSUPPORTED, "%s: stride %lld must be a non-negative multiple of 16 bytes", what,
                       (long long)d[i].stride);
  }
  return ULYSSES_OK;
}

// Every element of a tensor that is written has a place of its own: sorted by
// stride, each dimension steps over all of the ones below it.
int check_distinct(Dim* d, int nd, int D, const char* what) {
  for (int i = 0; i < nd; ++i)
    for (int k = i + 1; k < nd; ++k)
      if (d[k].stride < d[i].stride) { const Dim t = d[i]; d[i] = d[k]; d[k] = t; }
  int64_t e = D;
  for (int i = 0; i < nd; ++i) {
    if (d[i].n > 1 && d[i].stride < e)
      return set_error(ULYSSES_ERR_INVALID, "%s: rows overlap (stride %lld below %lld)", what, (long long)d[i].stride,
                       (long long)e);
    e += (d[i].n - 1) * d[i].stride;
  }
  return ULYSSES_OK;
}

// A strided tensor of rows of D in memory, for overlap checks.
struct Span { const char* p; int64_t bytes; int elt; Dim d[3]; };

Span span(const void* p, int elt, int D, const Dim* d, int nd) {
  Span x{(const char*)p, extent(d, nd, D) * elt, elt, {{1, 0}, {1, 0}, {1, 0}}};
  for (int i = 0; i < nd; ++i) x.d[i] = Dim{d[i].n, d[i].n > 1 ? d[i].stride : 0};
  return x;
}

// Whether two strided tensors may share memory.  Slices of one tensor (equal
// strides) are told apart when, inside the period of some dimension that both
// have, their windows lie side by side (Q's heads before K's in a token's row).
bool may_overlap(const Span& x, const Span& y, int D) {
  if (!overlap(x.p, (size_t)x.bytes, y.p, (size_t)y.bytes)) return false;
  if (x.elt != y.elt) return true;
  const Span& lo = x.p <= y.p ? x : y;
  const Span& hi = x.p <= y.p ? y : x;
  const int64_t off = (hi.p - lo.p) / x.elt;
  for (int c = 0; c < 3; ++c) {
    const int64_t pitch = lo.d[c].stride;
    if (pitch == 0 || pitch != hi.d[c].stride || lo.d[c].n != hi.d[c].n) continue;
    int64_t lo_n = D, hi_n = D;
    bool ok = true;
    for (int i = 0; i < 3; ++i) {
      if (i == c) continue;
      const Dim &u = lo.d[i], &v = hi.d[i];
      if (u.stride < pitch && v.stride < pitch) {
        lo_n += (u.n - 1) * u.stride;
        hi_n += (v.n - 1) * v.stride;
      } else if (!(u.stride == v.stride && u.stride >= pitch * lo.d[c].n)) {
        ok = false;
      }
    }
    if (ok && lo_n <= off && off + hi_n <= pitch) return false;
  }
  return true;
}

bool same_place(const Span& x, const Span& y) {
  bool same = x.p == y.p && x.elt == y.elt;
  for (int i = 0; i < 3; ++i) same = same && x.d[i].n == y.d[i].n && x.d[i].stride == y.d[i].stride;
  return same;
}

constexpr double kMaxFreq = 1099511627776.0;   // 2^40

// freq / 2 pi in units of 2^-64 of a turn, whole turns dropped: off by one unit
// at most for |freq| <= 2^40.  A quotient in doubles is off by 2^-53 of itself,
// which at position 2^31 is 2^-22 radians for freq = 1 and 1/4 for 2^20; so
// 1 / 2 pi is held in two doubles and the product's rounding error kept.
uint64_t turn_units(double freq) {
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;   // 1 / 2 pi to 2^-111
  constexpr double kUnits = 18446744073709551616.0;                            // 2^64
  const double f = std::fabs(freq);
  const volatile double whole = f * kHi;                       // rounded here, whatever the compiler contracts
  const double p = whole, rest = std::fma(f, kHi, -p) + f * kLo;
  const double units = (p - std::floor(p)) * kUnits;           // exact, below 2^64
  const uint64_t n = (uint64_t)units;
  const uint64_t u = n + (uint64_t)std::llround(rest * kUnits + (units - (double)n));
  return freq < 0.0 ? 0 - u : u;
}

int rope(const ulysses_rope_item* items, int n_items, const int32_t* positions, int n_axes, const double* inv_freq,
         const int32_t* axes, int rot_dim, int pairs, int64_t S, int B, int D, int dtype, int out_dtype, int inverse,
         void* stream) {
  if (!elt_size(dtype) || !elt_size(out_dtype)) return set_error(ULYSSES_ERR_INVALID, "unknown dtype %d -> %d", dtype, out_dtype);
  if (dtype != out_dtype && !(dtype == ULYSSES_FP32 && out_dtype == ULYSSES_BF16))
    return set_error(ULYSSES_ERR_UNSUPPORTED, "rope: output type must be the input's, or BF16 from FP32");
  if (n_items < 0 || n_items > kMaxRopeItems)
    return set_error(ULYSSES_ERR_INVALID, "n_items=%d must be in [0, %d]", n_items, kMaxRopeItems);
  if (S < 0 || B <= 0) return set_error(ULYSSES_ERR_INVALID, "bad sizes S=%lld B=%d", (long long)S, B);
  if (S > kMaxTokens / B) return set_error(ULYSSES_ERR_UNSUPPORTED, "rope: B*S must fit int32");
  if (D != 64 && D != 128) return set_error(ULYSSES_ERR_UNSUPPORTED, "head dim %d not in {64,128}", D);
  if (rot_dim <= 0 || rot_dim > D || rot_dim % 16)
    return set_error(ULYSSES_ERR_INVALID, "rot_dim=%d must be a multiple of 16 in (0, %d]", rot_dim, D);
  if (pairs != ULYSSES_PAIRS_HALF && pairs != ULYSSES_PAIRS_ADJACENT)
    return set_error(ULYSSES_ERR_INVALID, "unknown pair order %d", pairs);
  if (n_axes < 1 || n_axes > kMaxRopeAxes)
    return set_error(ULYSSES_ERR_INVALID, "n_axes=%d must be in [1, %d]", n_axes, kMaxRopeAxes);
  if (!inv_freq || (n_items > 0 && !items)) return set_error(ULYSSES_ERR_INVALID, "NULL argument");
  RopeArgs a{};
  a.half = rot_dim / 2;
  for (int i = 0; i < a.half; ++i) {
    if (!std::isfinite(inv_freq[i])) return set_error(ULYSSES_ERR_INVALID, "inv_freq[%d] is not finite", i);
    if (std::fabs(inv_freq[i]) > kMaxFreq)
      return set_error(ULYSSES_ERR_UNSUPPORTED, "inv_freq[%d]=%g above 2^40", i, inv_freq[i]);
    a.freq[i] = turn_units(inv_freq[i]);
    const int ax = axes ? axes[i] : 0;
    if (ax < 0 || ax >= n_axes) return set_error(ULYSSES_ERR_INVALID, "axes[%d]=%d outside [0, %d)", i, ax, n_axes);
    a.axis[i] = (uint8_t)ax;
  }
  const int ein = elt_size(dtype), eout = elt_size(out_dtype);
  Span src[kMaxRopeItems], dst[kMaxRopeItems];
  for (int i = 0; i < n_items; ++i) {
    const ulysses_rope_item& it = items[i];
    if (it.H <= 0 || it.H > (1 << 20)) return set_error(ULYSSES_ERR_INVALID, "item %d: bad head count %d", i, it.H);
    if (S == 0) continue;
    if (!it.src || !it.dst) return set_error(ULYSSES_ERR_INVALID, "NULL buffer");
    if (!aligned16(it.src) || !aligned16(it.dst)) return set_error(ULYSSES_ERR_INVALID, "buffers must be 16-byte aligned");
    Dim ds[3] = {{B, it.src_b}, {S, it.src_s}, {it.H, it.src_h}}, dd[3] = {{B, it.dst_b}, {S, it.dst_s}, {it.H, it.dst_h}};
    int rc = check_strides(ds, 3, ein, "rope source");
    if (!rc) rc = check_strides(dd, 3, eout, "rope destination");
    if (rc) return rc;
    a.job[i] = RopeJob{it.src, it.dst, it.H, a.heads, it.src_b, it.src_s, it.src_h, it.dst_b, it.dst_s, it.dst_h,
                       extent(ds, 3, D), extent(dd, 3, D)};
    src[i] = span(it.src, ein, D, ds, 3);
    dst[i] = span(it.dst, eout, D, dd, 3);
    if ((rc = check_distinct(dd, 3, D, "rope destination"))) return rc;
    a.heads += it.H;
  }
  if (S == 0 || n_items == 0) return ULYSSES_OK;
  if (!positions) return set_error(ULYSSES_ERR_INVALID, "NULL positions");
  if (!aligned4(positions)) return set_error(ULYSSES_ERR_INVALID, "positions must be 4-byte aligned");
  if (a.heads > (1 << 20)) return set_error(ULYSSES_ERR_UNSUPPORTED, "rope: %d heads in one call", a.heads);
  for (int i = 0; i < n_items; ++i)
    for (int k = 0; k < n_items; ++k) {
      const bool in_place = i == k && same_place(dst[i], src[i]);
      if ((!in_place && may_overlap(dst[i], src[k], D)) || (i < k && may_overlap(dst[i], dst[k], D)))
        return set_error(ULYSSES_ERR_INVALID, "rope: destination %d overlaps another tensor (in place needs equal strides and types)", i);
    }
  a.njobs = n_items;
  a.pos = positions;
  a.S = S;
  a.N = S * B;
  a.D = D;
  a.pairs = pairs;
  a.inverse = inverse;
  a.heads_fast = items[0].src_h <= items[0].src_s ? 1 : 0;
  a.dtype = dtype;
  a.out_dtype = out_dtype;
  return launch_rope(a, (cudaStream_t)stream);
}

// Shape of the paged cache, shared by every call that touches it.
int check_cache(int64_t num_pages, int page, int H_kv, int D, int B, int cols, int dtype, int cache_dtype,
                const void* kc, const void* vc, const float* ks, const float* vs) {
  if (!elt_size(dtype) || !type_size(cache_dtype))
    return set_error(ULYSSES_ERR_INVALID, "unknown dtype %d (cache %d)", dtype, cache_dtype);
  if (cache_dtype != dtype && cache_dtype != ULYSSES_E4M3)
    return set_error(ULYSSES_ERR_UNSUPPORTED, "cache type %d must be the rows' type %d or E4M3", cache_dtype, dtype);
  if (D != 64 && D != 128) return set_error(ULYSSES_ERR_UNSUPPORTED, "head dim %d not in {64,128}", D);
  if (page <= 0 || page % 16 || page > (1 << 20))
    return set_error(ULYSSES_ERR_UNSUPPORTED, "page_size=%d must be a positive multiple of 16 up to 2^20", page);
  if (num_pages < 0 || num_pages > kMaxTokens || H_kv <= 0 || H_kv > 4096 || B < 0 || cols < 0)
    return set_error(ULYSSES_ERR_INVALID, "bad sizes num_pages=%lld H_kv=%d B=%d table_cols=%d", (long long)num_pages, H_kv, B, cols);
  if ((int64_t)cols * page > kMaxPositions)
    return set_error(ULYSSES_ERR_UNSUPPORTED, "table_cols * page_size = %lld above 2^30 positions", (long long)cols * page);
  if ((double)num_pages * H_kv * (page / 16) > 2147483647.0)
    return set_error(ULYSSES_ERR_UNSUPPORTED, "cache of more than 2^31 blocks of 16 rows");
  if ((cache_dtype == ULYSSES_E4M3) != (ks != nullptr) || (cache_dtype == ULYSSES_E4M3) != (vs != nullptr))
    return set_error(ULYSSES_ERR_INVALID, "scales go with an E4M3 cache, and only with one");
  if (num_pages && (!kc || !vc)) return set_error(ULYSSES_ERR_INVALID, "NULL cache");
  if (!aligned16(kc) || !aligned16(vc) || !aligned4(ks) || !aligned4(vs))
    return set_error(ULYSSES_ERR_INVALID, "caches must be 16-byte aligned, scales 4-byte");
  return ULYSSES_OK;
}

// Shared by cache_write and cache_read; fills a.
int cache_args(CacheArgs& a, const void* k, const void* v, int64_t k_s, int64_t k_h, int64_t v_s, int64_t v_h, int64_t T,
               int B, const int32_t* cu, const int32_t* table, int cols, const int32_t* lens, void* kc, void* vc,
               float* ks, float* vs, int64_t num_pages, int page, int H, int D, int dtype, int cache_dtype, bool written) {
  int rc = check_cache(num_pages, page, H, D, B, cols, dtype, cache_dtype, kc, vc, ks, vs);
  if (rc) return rc;
  if (T < 0 || T > kMaxTokens) return set_error(ULYSSES_ERR_INVALID, "bad token count %lld", (long long)T);
  if (T == 0 || B == 0) return ULYSSES_OK;
  if (!k || !v || !table) return set_error(ULYSSES_ERR_INVALID, "NULL buffer");
  if (!aligned4(table) || !aligned4(lens) || !aligned4(cu))
    return set_error(ULYSSES_ERR_INVALID, "tables, lengths and offsets must be 4-byte aligned");
  if (!aligned16(k) || !aligned16(v)) return set_error(ULYSSES_ERR_INVALID, "buffers must be 16-byte aligned");
  Dim dk[2] = {{T, k_s}, {H, k_h}}, dv[2] = {{T, v_s}, {H, v_h}};
  const int e = elt_size(dtype);
  if ((rc = check_strides(dk, 2, e, "k")) || (rc = check_strides(dv, 2, e, "v"))) return rc;
  const Span sk = span(k, e, D, dk, 2), sv = span(v, e, D, dv, 2);
  if (written) {
    if ((rc = check_distinct(dk, 2, D, "k")) || (rc = check_distinct(dv, 2, D, "v"))) return rc;
    if (may_overlap(sk, sv, D)) return set_error(ULYSSES_ERR_INVALID, "k overlaps v");
  }
  const size_t rows = (size_t)num_pages * H * page, cb = rows * D * type_size(cache_dtype);
  const Span* both[2] = {&sk, &sv};
  for (const Span* s : both)
    if (overlap(s->p, (size_t)s->bytes, (const char*)kc, cb) || overlap(s->p, (size_t)s->bytes, (const char*)vc, cb))
      return set_error(ULYSSES_ERR_INVALID, "k and v must not overlap the caches");
  if (!written && overlap((const char*)kc, cb, (const char*)vc, cb))
    return set_error(ULYSSES_ERR_INVALID, "k_cache overlaps v_cache");
  a = CacheArgs{kc, vc, ks, vs, const_cast<void*>(k), const_cast<void*>(v), k_s, k_h, v_s, v_h, cu, lens, table,
                T, num_pages, B, cols, page, H, D, dtype, cache_dtype};
  return ULYSSES_OK;
}

int decode_args(DecodeArgs& a, int B, int H_q, int H_kv, int D, int cols, int page, int dtype, int cache_dtype) {
  if (H_q <= 0 || H_kv <= 0 || H_q % H_kv)
    return set_error(ULYSSES_ERR_INVALID, "H_q=%d must be a multiple of H_kv=%d", H_q, H_kv);
  if ((int64_t)B * H_q > (1 << 24)) return set_error(ULYSSES_ERR_UNSUPPORTED, "B*H_q=%lld above 2^24", (long long)B * H_q);
  a = DecodeArgs{};
  a.B = B; a.H_q = H_q; a.H_kv = H_kv; a.G = H_q / H_kv; a.D = D;
  a.cols = cols; a.page = page; a.dtype = dtype; a.cache_dtype = cache_dtype;
  return ULYSSES_OK;
}

}  // namespace

extern "C" {

int ulysses_rope_fwd(const ulysses_rope_item* items, int n_items, const int32_t* positions, int n_axes,
                     const double* inv_freq, const int32_t* axes, int rot_dim, int pairs, int64_t S, int B,
                     int D, int dtype, int out_dtype, void* stream) {
  return rope(items, n_items, positions, n_axes, inv_freq, axes, rot_dim, pairs, S, B, D, dtype, out_dtype, 0, stream);
}

int ulysses_rope_bwd(const ulysses_rope_item* items, int n_items, const int32_t* positions, int n_axes,
                     const double* inv_freq, const int32_t* axes, int rot_dim, int pairs, int64_t S, int B,
                     int D, int dtype, int out_dtype, void* stream) {
  return rope(items, n_items, positions, n_axes, inv_freq, axes, rot_dim, pairs, S, B, D, dtype, out_dtype, 1, stream);
}

int ulysses_cache_write(const void* k, const void* v, int64_t k_s, int64_t k_h, int64_t v_s, int64_t v_h,
                        int64_t T, int B, const int32_t* cu_new, const int32_t* page_table, int table_cols,
                        const int32_t* seq_lens, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                        int64_t num_pages, int page_size, int H_kv, int D, int dtype, int cache_dtype,
                        void* stream) {
  CacheArgs a{};
  int rc = cache_args(a, k, v, k_s, k_h, v_s, v_h, T, B, cu_new, page_table, table_cols, seq_lens, k_cache, v_cache,
                      k_scale, v_scale, num_pages, page_size, H_kv, D, dtype, cache_dtype, false);
  if (rc) return rc;
  if (!cu_new && T != B)
    return set_error(ULYSSES_ERR_INVALID, "without cu_new there is one token per sequence: T=%lld, B=%d", (long long)T, B);
  if (T == 0 || B == 0) return ULYSSES_OK;
  if (!seq_lens) return set_error(ULYSSES_ERR_INVALID, "NULL seq_lens");
  return launch_cache_write(a, (cudaStream_t)stream);
}

int ulysses_cache_read(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                       const int32_t* page_table, int table_cols, const int32_t* cu, const int32_t* first,
                       void* k, void* v, int64_t k_s, int64_t k_h, int64_t v_s, int64_t v_h, int64_t T, int B,
                       int64_t num_pages, int page_size, int H_kv, int D, int dtype, int cache_dtype,
                       void* stream) {
  CacheArgs a{};
  int rc = cache_args(a, k, v, k_s, k_h, v_s, v_h, T, B, cu, page_table, table_cols, first, const_cast<void*>(k_cache),
                      const_cast<void*>(v_cache), const_cast<float*>(k_scale), const_cast<float*>(v_scale), num_pages,
                      page_size, H_kv, D, dtype, cache_dtype, true);
  if (rc) return rc;
  if (T == 0 || B == 0) return ULYSSES_OK;
  if (!cu) return set_error(ULYSSES_ERR_INVALID, "NULL cu");
  return launch_cache_read(a, (cudaStream_t)stream);
}

size_t ulysses_attn_decode_workspace(int B, int H_q, int H_kv, int D, int table_cols, int page_size, int dtype,
                                     int cache_dtype) {
  DecodeArgs a;
  if (B < 0 || decode_args(a, B, H_q, H_kv, D, table_cols, page_size, dtype, cache_dtype)) return 0;
  return decode_workspace(a);
}

int ulysses_attn_decode(const void* q, int64_t q_b, int64_t q_h, const void* k_cache, const void* v_cache,
                        const float* k_scale, const float* v_scale, const int32_t* page_table, int table_cols,
                        const int32_t* seq_lens, void* o, int64_t o_b, int64_t o_h, float* lse, int B, int H_q,
                        int H_kv, int D, int64_t num_pages, int page_size, float scale, int dtype,
                        int cache_dtype, void* workspace, size_t ws_bytes, void* stream) {
  int rc = check_cache(num_pages, page_size, H_kv, D, B, table_cols, dtype, cache_dtype, k_cache, v_cache, k_scale, v_scale);
  if (rc) return rc;
  DecodeArgs a;
  if ((rc = decode_args(a, B, H_q, H_kv, D, table_cols, page_size, dtype, cache_dtype))) return rc;
  if (B == 0) return ULYSSES_OK;
  if (!q || !o || !seq_lens || (table_cols && !page_table)) return set_error(ULYSSES_ERR_INVALID, "NULL buffer");
  if (!aligned16(q) || !aligned16(o)) return set_error(ULYSSES_ERR_INVALID, "buffers must be 16-byte aligned");
  if (!aligned4(page_table) || !aligned4(seq_lens) || !aligned4(lse))
    return set_error(ULYSSES_ERR_INVALID, "table, lengths and LSE must be 4-byte aligned");
  Dim dq[2] = {{B, q_b}, {H_q, q_h}}, dout[2] = {{B, o_b}, {H_q, o_h}};
  const int e = elt_size(dtype);
  if ((rc = check_strides(dq, 2, e, "q")) || (rc = check_strides(dout, 2, e, "o"))) return rc;
  const int64_t qn = extent(dq, 2, D) * e, on = extent(dout, 2, D) * e;
  if ((rc = check_distinct(dout, 2, D, "o"))) return rc;
  if (overlap((const char*)o, (size_t)on, (const char*)q, (size_t)qn))
    return set_error(ULYSSES_ERR_INVALID, "o overlaps q");
  const size_t need = decode_workspace(a);
  if (ws_bytes < need || (need && !workspace))
    return set_error(ULYSSES_ERR_INVALID, "workspace too small: %zu < %zu", ws_bytes, need);
  if (((uintptr_t)workspace & 255u) != 0) return set_error(ULYSSES_ERR_INVALID, "workspace must be 256-byte aligned");
  a.q = q; a.q_b = q_b; a.q_h = q_h;
  a.o = o; a.o_b = o_b; a.o_h = o_h; a.lse = lse;
  a.kc = k_cache; a.vc = v_cache; a.ks = k_scale; a.vs = v_scale;
  a.table = page_table; a.lens = seq_lens; a.num_pages = num_pages;
  a.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)D)) * 1.4426950408889634f;
  a.ws = workspace;
  return launch_decode(a, simt_chosen(), (cudaStream_t)stream);
}

}  // extern "C"
