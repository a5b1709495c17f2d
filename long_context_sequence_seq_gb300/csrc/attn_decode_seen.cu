// Attention of one new token per sequence over the paged cache, adding each
// cached token's attention weight to what it has gathered: caches as they are
// and in e4m3 (attn_decode.cuh).
#include "attn_decode.cuh"

namespace ulysses {

ULYSSES_ERROR_READER(read_error_attn_decode_seen)

int launch_decode_seen(const DecodeArgs& a, bool simt, cudaStream_t st) {
  return a.cache_dtype == ULYSSES_E4M3 ? run_decode<true, true>(a, simt, st) : run_decode<false, true>(a, simt, st);
}

}  // namespace ulysses
