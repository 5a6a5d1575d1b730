// The appended codes' short cut (csrc/append_quick.h) against the divisions:
// every (largest, smallest, value) of the groups of bf16 values above zero with
// the largest in [1, 2) and the smallest from 1/2 on, and a grid of groups with
// values far apart or on both sides; with the reciprocal exact and one unit off
// either way.  Prints the number of values compared, then "ok".
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "append_quick.h"

static float bf16(int bits) {
  const uint32_t u = static_cast<uint32_t>(bits) << 16;
  float f;
  std::memcpy(&f, &u, 4);
  return f;
}

static long compared = 0, taken = 0;

// One group's scale and bias by the quantizer's steps, then one of its values.
struct Group {
  float s, z, top;
  int bits;
  Group(float lo, float hi, int b) : top(static_cast<float>((1 << b) - 1)), bits(b) {
    s = (hi - lo) / top;
    s = s < 1e-7f ? 1e-7f : s;
    const bool side = std::fabs(lo) > std::fabs(hi);
    s = side ? s : -s;
    const float edge = side ? lo : hi;
    const float q0 = std::round(edge / s);
    z = 0.0f;
    if (q0 != 0.0f) {
      s = edge / q0;
      z = edge;
    }
  }
  bool agrees(float x) const {
    const float want = std::fmin(std::round((x - z) / s), top);
    const float exact = 1.0f / s;
    const float inverse[3] = {exact, std::nextafter(exact, 0.0f), std::nextafter(exact, std::copysign(INFINITY, exact))};
    for (float inv : inverse) {
      ++compared;
      const float r = qmvd::quick_quotient(x, z, inv);
      if (!(std::fabs(r - std::nearbyint(r)) < 0.5f - qmvd::quick_near(bits))) continue;   // the divisions are done
      ++taken;
      const float got = std::fmin(std::nearbyint(r), top);
      if (got != want) {
        std::printf("bits %d s %.9g z %.9g x %.9g: %g by the reciprocal, %g by division\n", bits, s, z, x, got, want);
        return false;
      }
    }
    return true;
  }
};

int main() {
  constexpr int kOne = 0x3F80;                 // bf16 1.0; 128 values a binade
  for (int bits : {4, 8}) {
    // all values above zero (one of the loops' binades covers all: scaling by a power of two changes no step)
    for (int hi = kOne; hi < kOne + 128; ++hi)
      for (int lo = hi - 1; lo >= kOne - 128; --lo) {
        const Group g(bf16(lo), bf16(hi), bits);
        for (int x = lo; x <= hi; ++x)
          if (!g.agrees(bf16(x))) return 1;
      }
    // far apart, and on both sides of zero
    for (int hi = kOne; hi < kOne + 128; hi += 3)
      for (int lo = kOne - 1024; lo < kOne + 256; lo += 11)
        for (int sign : {0, 1}) {
          const float l = sign ? -bf16(lo) : bf16(lo), h = bf16(hi);
          if (l > h) continue;
          const Group g(l, h, bits);
          for (int x = kOne - 1024; x < kOne + 256; x += 5)
            for (int neg : {0, 1}) {
              const float v = neg ? -bf16(x) : bf16(x);
              if (v >= l && v <= h && !g.agrees(v)) return 1;
            }
        }
  }
  if (taken * 10 < compared * 9) return std::printf("the short cut is hardly taken: %ld of %ld\n", taken, compared), 1;
  std::printf("%ld values\nok\n", compared);
  return 0;
}
