// What is still under way in a ring of copies when its reader gives up.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define NVFP4_RING_FN __device__ __forceinline__
#else
#define NVFP4_RING_FN inline
#endif

namespace nvfp4 {

// The fills that were asked for and not read, in their order: wait(stage, parity) for each, until one says
// false.  reads_left, loads_left: tiles that the reader has yet to read, and the loader yet to ask for;
// stage and parity: of the reader's next tile.
template <typename Wait>
NVFP4_RING_FN void await_fills(uint32_t reads_left, uint32_t loads_left, uint32_t stage, uint32_t parity,
                               uint32_t stages, Wait wait) {
  for (uint32_t n = reads_left - loads_left; n > 0 && wait(stage, parity); --n)
    if (++stage == stages) stage = 0, parity ^= 1u;
}

}  // namespace nvfp4
