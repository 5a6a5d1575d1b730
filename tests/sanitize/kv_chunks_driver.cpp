// The cutting of lengths into chunks (csrc/kv_chunks.h) on the host, with the
// room that qmv_kv_attend's launch and workspace leave: max(share, full) + B
// chunks, full = all slots over most_chunk.  Prints "ok".
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <random>
#include <vector>

#include "kv_chunks.h"

using namespace qmvd;

static int check(const std::vector<uint32_t> &lens, uint32_t longest, uint32_t share, uint32_t most_chunk) {
  uint64_t lines = 0, chunks = 0;
  for (uint32_t n : lens) lines += (uint64_t(n) + kChunkLine - 1) / kChunkLine;
  if (lines > (1u << 30)) return 0;
  const uint32_t most = chunk_slots(static_cast<uint32_t>(lines), share, most_chunk);
  bool bad = most < kChunkUnit || most > most_chunk || most % kChunkUnit != 0;
  for (uint32_t n : lens)
    if (!bad) {
      const uint64_t k = (uint64_t(n) + most - 1) / most, even = k ? (n + k - 1) / k : 1;
      const uint64_t size = (even + kChunkUnit - 1) / kChunkUnit * kChunkUnit;
      bad = k * size < n || size > most;
      chunks += k;
    }
  const uint64_t full = (uint64_t(lens.size()) * longest + most_chunk - 1) / most_chunk;
  bad = bad || chunks > std::max<uint64_t>(full, share) + lens.size();
  if (bad) std::printf("%zu sequences, longest %u, share %u, most_chunk %u: chunk %u, %llu chunks\n", lens.size(), longest, share, most_chunk, most, (unsigned long long)chunks);
  return bad;
}

int main() {
  std::mt19937 rng(1);
  // up to 2^35 slots in all, the most that is accepted
  for (uint32_t share : {1u, 2u, 3u, 7u, 64u, 1024u})
    for (uint32_t B : {1u, 2u, 63u, 64u, 65u, 200u, 4096u, 65536u})
      for (uint32_t longest : {1u, 64u, 65u, 1025u, 16384u, 131071u, 1u << 20, 1u << 28, 0x7FFF0000u}) {
        if (uint64_t(B) * longest > uint64_t(1) << 35) continue;
        const uint64_t even = (uint64_t(B) * longest + 8 * share - 1) / (8 * share);
        const uint64_t whole = (uint64_t(longest) + kChunkUnit - 1) / kChunkUnit * kChunkUnit;
        const uint32_t most = static_cast<uint32_t>(std::min(whole, std::max<uint64_t>(2048, (even + kChunkUnit - 1) / kChunkUnit * kChunkUnit)));
        for (int kind = 0; kind < 4; ++kind) {
          std::vector<uint32_t> lens(B, longest);
          if (kind == 1) for (auto &n : lens) n = rng() % (longest + 1);
          if (kind == 2) for (auto &n : lens) n = rng() % 4 ? 0 : longest;
          if (kind == 3) std::fill(lens.begin(), lens.end(), 0);
          if (check(lens, longest, share, most)) return 1;
        }
      }
  std::printf("ok\n");
  return 0;
}
