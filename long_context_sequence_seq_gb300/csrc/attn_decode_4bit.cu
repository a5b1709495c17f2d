// Attention of one new token per sequence over the paged cache: 4-bit caches
// (attn_decode.cuh).
#include "attn_decode.cuh"

namespace ulysses {

ULYSSES_ERROR_READER(read_error_attn_decode_4bit)

int launch_decode_4bit(const DecodeArgs& a, bool simt, cudaStream_t st) {
  return a.seen ? run_decode<kE2m1, true>(a, simt, st) : run_decode<kE2m1, false>(a, simt, st);
}

}  // namespace ulysses
