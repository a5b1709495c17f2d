// How an eviction's move (cache_evict.cu) uses shared memory: rows of a chunk,
// chunks on their way, and what a CTA takes, so that two of them fit an SM.  Plain
// host C++ (no CUDA types), so the sums can be checked on a machine without a GPU.
#pragma once

#include <cstdint>

namespace ulysses {
namespace evict {

constexpr int kMoveThreads = 256;  // that move rows, of a CTA
constexpr int kMaxBatch = 2048;    // sequences of one launch, at most
constexpr int kMinBatch = 256;     // that every kind of row has room for (lengths and prefix sums, in shared memory)
constexpr int kMostStages = 6;

// Of an SM: 228 KB of shared memory, of which each CTA has 1 KB for the system.
constexpr int kSmBytes = 228 * 1024, kReservedBytes = 1024, kCtasAnSm = 2;

// Rows moved together: 16 KB of K and of V, at most 128.  (8 KB of rows of 128 bytes,
// for more chunks on their way: 48 sequences cut from 4160 to 4096 tokens of 8 heads
// in e4m3 209 us, this way 178; in bf16 of D = 64 208 and 162.)
constexpr int chunk_of(int row_bytes) { return row_bytes >= 128 ? 16384 / row_bytes : 128; }

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

// Chunks whose places are known: those on their way, one that is looked up and one more.
constexpr int ring_of(int stages) { return stages + 2; }
// What is not a stage: places, four barriers each and the flag that ends the CTA;
// lengths and prefix sums.
constexpr int fixed_bytes(int row_bytes, int stages) {
  return ring_of(stages) * (2 * 8 * chunk_of(row_bytes) + 24 + 4 * 8) + 16;
}
constexpr int batch_bytes(int sequences) { return sequences * 12 + 4; }
constexpr int cta_bytes(int row_bytes, bool four, bool scales, int stages, int sequences) {
  return stages * stage_bytes(row_bytes, four, scales) + fixed_bytes(row_bytes, stages) + batch_bytes(sequences) + kReservedBytes;
}

// Chunks on their way through shared memory: as many as leave room for the other CTA.
// (One more in 4 bits of D = 128, with one CTA an SM: 48 sequences cut from 4160 to
// 4096 tokens of 8 heads 182 us, this way 129.)
constexpr int stages_of(int row_bytes, bool four, bool scales) {
  int n = kMostStages;
  while (n > 1 && cta_bytes(row_bytes, four, scales, n, kMinBatch) * kCtasAnSm > kSmBytes) --n;
  return n;
}
// Sequences of a launch: as many as leave it too.  (2048 sequences cut from 300 to 256
// bf16 tokens of 8 heads of 128 in one launch, one CTA an SM: 1552 us; in three 1267.)
constexpr int batch_of(int row_bytes, bool four, bool scales) {
  const int room = kSmBytes / kCtasAnSm - cta_bytes(row_bytes, four, scales, stages_of(row_bytes, four, scales), 0);
  return room / 12 < kMaxBatch ? room / 12 : kMaxBatch;
}

static_assert(sizeof(Places<64>) == 2 * 8 * 64 + 24, "");

}  // namespace evict
}  // namespace ulysses
