// Internal launcher interfaces shared by the CUDA translation units.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "device_once.h"
#include "ulysses.h"

namespace ulysses {

// Argument helpers of the C entry points.
inline int elt_size(int dtype) { return dtype == ULYSSES_BF16 ? 2 : (dtype == ULYSSES_FP32 ? 4 : 0); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline bool overlap(const char* a, size_t la, const char* b, size_t lb) { return a < b + lb && b < a + la; }

// Arguments of one attention launch on head-layout buffers (batch folded into
// the head index: buffer q head n in [0, n_q) reads kv head n / G).
struct AttnArgs {
  const void* q; const void* k; const void* v; const void* o; const void* dO;
  void* o_out;          // forward output O (input dtype)
  float* lse;           // forward output LSE
  const float* lse_in;  // backward input LSE
  float* dq; float* dk; float* dv;
  float* delta;         // backward scratch D_i, [n_q][S]
  int64_t S;
  int n_q;              // q heads in the buffer across the batch (B * nq)
  int nq;               // q heads per batch entry in the buffer
  int G; int D;
  int64_t lse_bstride;  // LSE element stride between batch entries
  const int32_t* cu; int nd; int causal; float scale; int dtype;
  // seq != 0: q/k/v/o/dO and dq/dk/dv point at the stage's first head inside
  // sequence-layout tensors [S][hq_tot or hkv_tot][D] (B == 1) instead of
  // head-layout buffers: the re-layout is folded into the kernels' addressing
  int seq; int hq_tot; int hkv_tot;
};

// Opts `func` in to `bytes` of dynamic shared memory on the current device,
// once per device (the runtime records the attribute per device); reports
// ULYSSES_ERR_CUDA with a message when the runtime refuses.  api.cu.
int opt_in_smem(PerDeviceOnce<>& once, const void* func, int bytes, const char* what);

// One tensor of a batched re-layout launch (relayout.cu): moves n heads
// starting at h0 of a sequence-layout tensor with H heads to or from a
// head-layout buffer; `add` (scatter, fp32 only) adds instead of writing.
// x0 is filled in by the launcher.
constexpr int kMaxRelayoutJobs = 6;
struct RelayoutJob {
  const void* src; void* dst;
  int H, n, h0, add;
  int x0;
};
// Tensors of one launch share S, B and the row size V (16-byte words per
// D-vector).
struct RelayoutBatch {
  RelayoutJob job[kMaxRelayoutJobs];
  int njobs;
  int B;
  int V;
  int64_t S;
};
int launch_relayout_batch(bool to_head, RelayoutBatch& bt, cudaStream_t stream);
int launch_relayout(bool to_head, const void* src, void* dst, int64_t S, int B, int H, int D,
                    int n, int h0, int elt, cudaStream_t stream, bool add = false);
int launch_simt_fwd(const AttnArgs& a, cudaStream_t st);
int launch_simt_bwd(const AttnArgs& a, cudaStream_t st);
int launch_delta(const AttnArgs& a, cudaStream_t st);
int launch_check_seqlens(const int32_t* cu, int nd, int64_t S, cudaStream_t st);
int launch_lse_merge(float* o_acc, float* lse_acc, const void* o_part, const float* lse_part, int64_t rows,
                     int D, int dtype, int first, cudaStream_t st);                       // ring.cu
int launch_cast_f32(void* dst, const float* src, int64_t n, int dtype, cudaStream_t st);  // ring.cu
int launch_add_f32(float* dst, const float* src, int64_t n, cudaStream_t st);             // ring.cu
int launch_pad_seq(const void* x, void* x_pad, int64_t S, int64_t S_pad, int B, int64_t row_bytes,
                   cudaStream_t st);                                                      // pad.cu
int launch_pad_cu(const int32_t* cu, int nd, int32_t* out, int64_t S, int64_t S_pad, cudaStream_t st);  // pad.cu
int launch_qkv_proj(const void* x, const void* w, void* qkv_head, int64_t S, int hidden, int n_heads, int D,
                    cudaStream_t st);                                                     // proj_gemm.cu
int launch_out_proj(const void* o_head, const void* w, void* y, int64_t S, int H_q, int D, int hidden,
                    cudaStream_t st);                                                     // proj_gemm.cu


// One tensor of a rotary launch (rope.cu), element strides; head0 is the first
// of its heads in the launch's numbering, src_n / dst_n the elements spanned.
constexpr int kMaxRopeItems = 4, kMaxRopeAxes = 4, kMaxRopePairs = 64;
struct RopeJob {
  const void* src; void* dst;
  int H, head0;
  int64_t src_b, src_s, src_h, dst_b, dst_s, dst_h;
  int64_t src_n, dst_n;
};
struct RopeArgs {
  RopeJob job[kMaxRopeItems];
  int njobs, heads;            // tensors, heads of all of them
  const int32_t* pos;          // [n_axes][N]
  int64_t S, N;                // tokens per batch entry, tokens in all
  int D, half, pairs, inverse;
  int heads_fast;              // rows of one token lie closer than rows of one head
  int dtype, out_dtype;
  uint64_t freq[kMaxRopePairs];   // turns per position, in units of 2^-64
  uint8_t axis[kMaxRopePairs];
};
int launch_rope(const RopeArgs& a, cudaStream_t st);

// The paged cache and the tokens of one write or read (kv_cache.cu).
struct CacheArgs {
  void* kc; void* vc; float* ks; float* vs;       // caches and scales
  void* k; void* v;                               // tokens' rows
  int64_t k_s, k_h, v_s, v_h;
  const int32_t* cu; const int32_t* lens;         // write: lens; read: first (in lens)
  const int32_t* table;
  int64_t T, num_pages;
  int B, cols, page, H, D, dtype, cache_dtype;
};
int launch_cache_write(const CacheArgs& a, cudaStream_t st);
int launch_cache_read(const CacheArgs& a, cudaStream_t st);

// Attention of one new token per sequence over the paged cache (attn_decode.cu).
struct DecodeArgs {
  const void* q; int64_t q_b, q_h;
  void* o; int64_t o_b, o_h;
  float* lse;
  const void* kc; const void* vc; const float* ks; const float* vs;
  const int32_t* table; const int32_t* lens;
  int64_t num_pages;
  int B, H_q, H_kv, G, D, cols, page, dtype, cache_dtype;
  float scale_log2;            // score scale * log2(e)
  void* ws;
};
size_t decode_workspace(const DecodeArgs& a);
int launch_decode(const DecodeArgs& a, bool simt, cudaStream_t st);
bool simt_chosen();                                                       // api.cu
bool multicast_allowed();                                                 // api.cu

}  // namespace ulysses
