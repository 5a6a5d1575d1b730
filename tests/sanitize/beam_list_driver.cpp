// The scan's list of hits (csrc/beam_list.h), run thread by thread on the host
// in many orders of their atomics: no place is read back that was not written.
// Arguments: the threads' hits, run lengths as "count x hits" pairs.  Prints "ok".
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "beam_list.h"

using namespace qmvd;

static bool clean(const std::vector<int> &mine, const std::vector<int> &order) {
  std::vector<char> written(kScanList, 0);     // bounds checked by .at()
  int count = 0;
  for (int t : order) {
    int i = count;
    count += mine[t];
    if (list_fits(i, mine[t]))
      for (int j = 0; j < mine[t]; ++j) written.at(i++) = 1;
  }
  for (int i = 0; i < list_readable(count); ++i)
    if (!written.at(i)) return false;
  return count > kScanList || list_readable(count) == count;
}

int main(int argc, char **argv) {
  std::vector<int> mine;
  for (int i = 1; i + 1 < argc; i += 2) mine.insert(mine.end(), std::atoi(argv[i]), std::atoi(argv[i + 1]));
  const int n = static_cast<int>(mine.size());
  std::vector<int> order(n);
  for (int i = 0; i < n; ++i) order[i] = i;
  // the four waves in each of their orders, then threads in any order
  int waves[] = {0, 1, 2, 3};
  do {
    std::vector<int> by_wave;
    for (int w : waves)
      for (int i = w * n / 4; i < (w + 1) * n / 4; ++i) by_wave.push_back(i);
    if (!clean(mine, by_wave)) return std::printf("a gap is read, waves %d %d %d %d\n", waves[0], waves[1], waves[2], waves[3]), 1;
  } while (std::next_permutation(waves, waves + 4));
  std::mt19937 rng(1);
  for (int k = 0; k < 5000; ++k) {
    std::shuffle(order.begin(), order.end(), rng);
    if (!clean(mine, order)) return std::printf("a gap is read, shuffle %d\n", k), 1;
  }
  std::printf("ok\n");
  return 0;
}
