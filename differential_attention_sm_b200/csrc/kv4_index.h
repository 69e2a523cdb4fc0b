// kv4_index.h — the rules by which the decode over the 4-bit cache turns what
// it reads on the device into addresses.  Plain C++ beside CUDA, so that the
// host tests compile and try them without a device.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define DA_INDEX_FN __host__ __device__ __forceinline__
#else
#define DA_INDEX_FN inline
#endif

namespace da {

// What stands in for the index of a tile in the cache.
constexpr uint32_t kNoTile = 0xFFFFFFFFu;   // of no use to the segment
constexpr uint32_t kBadTile = 0xFFFFFFFEu;  // on a page out of range

// Whether tile `next` lies right behind tile `mine` in memory.  Both have to be
// tiles: kNoTile + 1 is 0, the index of the cache's first tile.
DA_INDEX_FN bool tiles_joined(uint32_t mine, uint32_t next) {
  return mine < kBadTile && next < kBadTile && next == mine + 1u;
}

// Runs [first, first + count) of a unit, as they were written down, cut to the
// runs that there are.  A warp whose wait timed out leaves without writing its
// units' spans: what lies there then is whatever the scratch held, and the
// second kernel, which still runs, must not read outside the scratch for it.
DA_INDEX_FN void bound_span(int& first, int& count, int runs) {
  first = first < 0 ? 0 : (first > runs ? runs : first);
  count = count < 0 ? 0 : (count > runs - first ? runs - first : count);
}

}  // namespace da
