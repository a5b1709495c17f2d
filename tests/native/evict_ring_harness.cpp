// Host test of the shared memory that an eviction's move takes (csrc/evict_ring.h):
// prints, for every kind of row, its chunks, stages and launches.
#include <cstdio>

#include "evict_ring.h"

using namespace ulysses::evict;

template <int kRowB, bool kFour, bool kScales>
void tell(const char* held, int D) {
  constexpr int chunk = chunk_of(kRowB), stages = stages_of(kRowB, kFour, kScales);
  // what the kernel declares itself: the ring of places, four barriers each, a flag
  struct Declared {
    Places<chunk> places[ring_of(stages)];
    uint64_t barriers[4 * ring_of(stages)];
    int stop;
  };
  constexpr int batch = batch_of(kRowB, kFour, kScales);
  std::printf("%s %d chunk %d row_bytes %d stages %d stage %d batch %d declared %d counted %d\n", held, D, chunk,
              kRowB + (kScales ? 4 : 0) + (kFour ? kRowB / 8 : 0), stages, stage_bytes(kRowB, kFour, kScales), batch,
              (int)sizeof(Declared), fixed_bytes(kRowB, stages));
}

int main() {
  tell<64, true, true>("e2m1", 128);
  tell<32, true, true>("e2m1", 64);
  tell<128, false, true>("e4m3", 128);
  tell<64, false, true>("e4m3", 64);
  tell<256, false, false>("bf16", 128);
  tell<128, false, false>("bf16", 64);
  tell<512, false, false>("fp32", 128);
  tell<256, false, false>("fp32", 64);
  return 0;
}
