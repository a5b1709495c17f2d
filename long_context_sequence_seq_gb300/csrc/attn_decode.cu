// Attention of one new token per sequence over the paged cache: caches as they
// are and in e4m3, and the choice between the units that hold the kernels
// (attn_decode.cuh).
#include "attn_decode.cuh"

namespace ulysses {

ULYSSES_ERROR_READER(read_error_attn_decode)

size_t decode_workspace(const DecodeArgs& a) {
  if (a.B == 0) return 0;
  // both engines', whichever the process has chosen when the call is made
  size_t most = 0;
  for (const bool simt : {false, true}) {
    const int heads = heads_of(a, simt);
    const size_t n = cluster_of(a, heads) ? 0 : ws_layout(a, heads).total;
    if (n > most) most = n;
  }
  return most;
}

int launch_decode(const DecodeArgs& a, bool simt, cudaStream_t st) {
  if (a.cache_dtype == ULYSSES_E2M1) return launch_decode_4bit(a, simt, st);
  if (a.seen) return launch_decode_seen(a, simt, st);
  return a.cache_dtype == ULYSSES_E4M3 ? run_decode<true, false>(a, simt, st) : run_decode<false, false>(a, simt, st);
}

}  // namespace ulysses
