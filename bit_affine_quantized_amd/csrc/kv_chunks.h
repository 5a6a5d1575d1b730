// The size of the chunks that lengths are cut into, as a plain function (host
// and device).
#pragma once

#include <stdint.h>

namespace qmvd {

constexpr uint32_t kChunkLine = 64;            // slots; lengths are counted in lines, so that their sum fits 32 bits
constexpr uint32_t kChunkUnit = 128;           // chunks are multiples of it

// Slots a chunk at most, for about `share` chunks of `lines` lines in all (at most
// 2^30), and at most most_chunk slots, a multiple of kChunkUnit.  Compared in
// lines: in slots an equal share can pass 32 bits.
constexpr uint32_t chunk_slots(uint32_t lines, uint32_t share, uint32_t most_chunk) {
  constexpr uint32_t unit = kChunkUnit / kChunkLine;
  const uint32_t even = (lines + share - 1) / share, most = most_chunk / kChunkLine;
  const uint32_t size = even < 1 ? unit : (even + unit - 1) / unit * unit;
  return (size < most ? size : most) * kChunkLine;
}

}  // namespace qmvd
