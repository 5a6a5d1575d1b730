// The appended codes' short cut around a division, as plain functions (host
// and device, built without contraction).
//
// A code is min(round((x - z) / s), top), each operation rounded to fp32.  The
// difference is taken as the definition takes it; the quotient then comes from
// the reciprocal of s, itself off by one unit of 2^-23 at most.  With the
// roundings of the product and of the true quotient that is off by at most two
// units of 2^-23 of the quotient, which lies between 0 and top + 1 (s is the range
// over top, moved by at most half a step in the edge's code).  Where it is
// further from a half than four units of 2^-23 of 2^BITS, it rounds to the same
// code; elsewhere (one lane in 500 at 8 bits) the divisions are done.  x / s - z / s
// would save an operation, but not do: in a group without a value at or below
// zero |z / s| is not bounded by top.
#pragma once

namespace qmvd {

constexpr float quick_quotient(float x, float z, float inverse) { return (x - z) * inverse; }

// How close to a half a quotient has to be for the divisions.
constexpr float quick_near(int bits) { return static_cast<float>(1 << bits) / (1 << 21); }

}  // namespace qmvd
