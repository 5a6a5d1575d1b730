// The scan's list of hits in LDS, as plain functions (host and device): which
// places a thread writes, and which may be read back.
#pragma once

namespace qmvd {

constexpr int kScanList = 1024;                // logits of a chunk that are ranked

// A thread reserves `mine` places from `first` on with one atomic and writes
// all of them, or none if they do not all fit.
constexpr bool list_fits(int first, int mine) { return first + mine <= kScanList; }

// How many places hold an entry once `hits` have been reserved in all.  Past
// the list's end it is none: the thread that crosses the end wrote nothing, so
// a gap of whatever LDS held before lies somewhere below it.
constexpr int list_readable(int hits) { return hits <= kScanList ? hits : 0; }

}  // namespace qmvd
