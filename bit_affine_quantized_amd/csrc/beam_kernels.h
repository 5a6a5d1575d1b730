// Beam search's selection: the best `num` of W beams x V tokens.
//
//   lse_w = ln sum_v exp(x[w, v])
//   c[w, v] = score_w + (x[w, v] - lse_w)      (fp32, each operation rounded)
//
// in descending c, ties to the lowest w*V + v; a NaN c counts as -infinity.
//
// The logits are read once.  beam_scan_kernel takes a chunk of one row:
// its maximum, its sum of exponentials and its `num` best logits.  c does not
// fall where x rises, so these hold every winner, with one exception: logits
// a rounding apart can share one c, and then the index decides, so a logit
// just below a chunk's list could still win.  Each chunk reports the best
// logit it left out; beam_join_kernel, which joins the sums, ranks the lists
// and sees the threshold, goes through the logits for the entries that tie with
// it where one left out could do so ahead of a listed one.  Everything above the
// threshold is listed, so one sweep in index order is enough, and it ends with the
// last entry found: at once for a finished item, whose beams' scores are all
// -infinity.
//
// On MI355X, 16 items x 8 beams x 131072 tokens, bf16 (33.6 MB): 15.9 us for the
// scan, of which the loads take about 4 and vector instructions the rest: all
// waves come to them at once, and the bound and the list are paid once a thread
// (so 64 logits a thread where the machine is full with that, 17.8 us with 32).
// A bound first and a list of the few logits above it (about 1.5 times `num` a
// chunk) take the place of sorting; with the bound found bit by bit over whole
// 64-bit keys, and a list entry at a time under a branch, the scan took 58.
// The join takes 4 to 7 us, a launch and a chain of barriers.  One call among others
// takes 23 us; with 100 tokens of each row open and the rest at -infinity 34, with all
// logits equal 36; with one item of nothing but NaN, whose chunks have no bound and
// are taken logit by logit, 229.

#pragma once

#include <float.h>

#include "beam_list.h"
#include "kv_device.h"

namespace qmvd {

constexpr int kBeamMost = 32;                  // `num` at most (fewer than a wave's lanes)
constexpr int kScanThreads = 256;
constexpr int kScanWaves = kScanThreads / 64;

struct BeamArgs {
  const void *logits;                          // [B, W, V] bf16 or fp32, row stride logits_ld
  const float *scores;                         // [B, W]
  int64_t logits_ld;
  float *m, *l, *left_out;                     // [B*W*chunks]
  u32x2 *list;                                 // [B*W*chunks][num]: logit, token; token -1 past a short list
  float *out_scores;
  int32_t *out_parents, *out_tokens;           // [B, num]
  int B, W, num, chunks, f32;
  int V;
  Divider per_row, per_chunk;                  // by chunks * num, by chunks
};

__device__ __forceinline__ float logit_at(const BeamArgs &a, int64_t row, int v) {
  return a.f32 ? static_cast<const float *>(a.logits)[row * a.logits_ld + v]
               : qmvk::bf16_to_f32(static_cast<const uint16_t *>(a.logits)[row * a.logits_ld + v]);
}

// Keys that no two entries share: the order of the value, then the lower
// index first.  NaN ranks lowest here.
__device__ __forceinline__ uint64_t rank_key(float x, uint32_t index) {
  const uint32_t o = x != x ? 0u : ordered(x);
  return (static_cast<uint64_t>(o) << 32) | (0xFFFFFFFFu - index);
}

__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t o = static_cast<uint32_t>(key >> 32);
  return o == 0u ? __uint_as_float(0x7FC00000u)
                 : __uint_as_float((o & 0x80000000u) ? (o ^ 0x80000000u) : ~o);
}

__device__ __forceinline__ uint32_t key_index(uint64_t key) { return 0xFFFFFFFFu - static_cast<uint32_t>(key); }

// A bound that at least `need` of a wave's 64 keys reach (0 if there are not
// that many; keys are unique but for zeros, which mean "none") and hardly more:
// half as many more at most.  Bit by bit on the values, from the largest
// one's exponent or the one below it if enough lanes reach that, which leaves
// a handful of steps on logits; only where values tie do the indexes decide.
// `index` gives the lane's index part, asked for only then.
template <typename I>
__device__ __forceinline__ uint64_t wave_bound(uint32_t value, int need, I index) {
  const int most = need + need / 2;
  if (__popcll(__ballot(value != 0)) < need) return 0;
  const uint32_t top = wave_max(value) & 0xFF800000u;
  uint32_t t = top;
  int bit = 22;
  int n = __popcll(__ballot(value >= t));
  if (n < need && top >= 0x01000000u) {
    t = top - 0x00800000u;
    n = __popcll(__ballot(value >= t));
  }
  if (n < need) {
    t = 0;
    n = 64;
    bit = 31;
  }
  for (; bit >= 0; --bit) {
    if (n <= most) return static_cast<uint64_t>(t) << 32;
    const uint32_t c = t | (1u << bit);
    const int k = __popcll(__ballot(value >= c));
    t = k >= need ? c : t;
    n = k >= need ? k : n;
  }
  if (n <= most) return static_cast<uint64_t>(t) << 32;
  const int more = need - __popcll(__ballot(value > t));   // of those equal to t
  const uint32_t mine = index();
  uint32_t u = 0;
  for (bit = 31; bit >= 0; --bit) {
    const uint32_t c = u | (1u << bit);
    u = __popcll(__ballot(value == t && mine >= c)) >= more ? c : u;
  }
  return (static_cast<uint64_t>(t) << 32) | u;
}

__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint64_t o = __shfl_xor(v, off, 64);
    v = o > v ? o : v;
  }
  return v;
}

// Eight logits from v0 on, 16-byte loads of any alignment.
__device__ __forceinline__ void load8(const BeamArgs &a, int64_t at, float *x) {
  if (a.f32) {
    float r[8];
    __builtin_memcpy(r, static_cast<const float *>(a.logits) + at, 32);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = r[e];
  } else {
    uint32_t r[4];
    __builtin_memcpy(r, static_cast<const uint16_t *>(a.logits) + at, 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(r[e] << 16);
      x[2 * e + 1] = __uint_as_float(r[e] & 0xFFFF0000u);
    }
  }
}

// PER logits a thread, in pieces of eight: piece p of thread t starts at
// (p * kScanThreads + t) * 8 of the chunk.
template <int PER>
__global__ __launch_bounds__(kScanThreads) void beam_scan_kernel(BeamArgs a) {
  constexpr int kChunk = kScanThreads * PER;
  __shared__ uint64_t list[kScanList];
  __shared__ uint32_t found[kScanList];
  __shared__ uint64_t slots[kScanWaves];
  __shared__ float wave_m[kScanWaves], wave_l[kScanWaves];
  __shared__ int count;
  const int64_t row = div_by(blockIdx.x, a.per_chunk);
  const int chunk = blockIdx.x - static_cast<int>(row) * a.chunks;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int v0 = chunk * kChunk;
  const int len = min(kChunk, a.V - v0);
  const int64_t base = row * a.logits_ld + v0;
  if (tid == 0) count = 0;

  float x[PER];
  if (len == kChunk) {
#pragma unroll
    for (int p = 0; p < PER / 8; ++p) load8(a, base + (p * kScanThreads + tid) * 8, x + 8 * p);
  } else {
#pragma unroll
    for (int p = 0; p < PER / 8; ++p) {
      const int at = (p * kScanThreads + tid) * 8;
      if (at + 8 <= len) {
        load8(a, base + at, x + 8 * p);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[8 * p + e] = at + e < len ? logit_at(a, row, v0 + at + e) : -INFINITY;
      }
    }
  }
  // Sum of exponentials against the wave's own maximum; a NaN or +infinity
  // makes it NaN.
  float top = -INFINITY;
#pragma unroll
  for (int e = 0; e < PER; e += 2)             // fmaxf would first quiet each operand
    asm("v_max3_f32 %0, %0, %1, %2" : "+v"(top) : "v"(x[e]), "v"(x[e + 1]));
  const float m = wave_max(top);
  const float mm = m == -INFINITY ? 0.0f : m;
  float l = 0.0f;
#pragma unroll
  for (int e = 0; e < PER; ++e) l += __expf(x[e] - mm);
  l = wave_sum(l);

  // The list: `num` logits and the best one left out.  At least that many of
  // a wave's lanes hold a logit at or above `cut`.
  auto offset = [&](int e) { return ((e >> 3) * kScanThreads + tid) * 8 + (e & 7); };
  bool none = top != top;                      // NaN alone: no logit of the lane's equals `top`
  if (__builtin_expect(__ballot(top == -INFINITY) != 0, 0)) {
    uint32_t own = 0;
#pragma unroll
    for (int e = 0; e < PER; ++e) own |= x[e] == top && offset(e) < len ? 1u : 0u;
    none = own == 0;
  }
  const uint32_t best = tid * 8 < len && !none ? ordered(top) : 0u;
  const uint64_t cut_w = wave_bound(best, a.num + 1, [&] {
    int first = 0;                             // the lane's first logit that equals `top`
#pragma unroll
    for (int e = PER - 1; e >= 0; --e) first = x[e] == top ? e : first;
    return 0xFFFFFFFFu - static_cast<uint32_t>(v0 + offset(first));
  });
  if (lane == 0) {
    wave_m[wave] = m;
    wave_l[wave] = l;
    slots[wave] = cut_w;
  }
  __syncthreads();
  uint64_t cut = 0;
#pragma unroll
  for (int j = 0; j < kScanWaves; ++j) cut = slots[j] > cut ? slots[j] : cut;
  const float cut_x = cut == 0 ? -INFINITY : key_value(cut);
  if (!(top < cut_x)) {
    uint32_t hits[PER / 16];                   // NaN too: it ranks lowest, but has a rank
#pragma unroll
    for (int p = 0; p < PER / 16; ++p) {
      hits[p] = 0;
#pragma unroll
      for (int e = 15; e >= 0; --e) hits[p] = hits[p] + hits[p] + (x[16 * p + e] < cut_x ? 0u : 1u);
    }
    // Where lanes tie at the bound it has an index, or there is no bound: of the
    // logits at its value only those up to that index (or the chunk's end) are
    // hits, else the -infinities of a masked vocabulary would overflow the list.
    if (__builtin_expect(cut == 0 || static_cast<uint32_t>(cut) != 0, 0)) {
      const uint32_t reach = key_index(cut) - static_cast<uint32_t>(v0);
      const int last = reach < static_cast<uint32_t>(len) ? static_cast<int>(reach) : len - 1;
#pragma unroll
      for (int p = 0; p < PER / 16; ++p) {
        uint32_t over = 0;
#pragma unroll
        for (int e = 15; e >= 0; --e) over = over + over + (x[16 * p + e] > cut_x ? 1u : 0u);
        const int k0 = min(max(last + 1 - offset(16 * p), 0), 8), k1 = min(max(last + 1 - offset(16 * p + 8), 0), 8);
        hits[p] &= over | ((1u << k0) - 1) | (((1u << k1) - 1) << 8);
      }
    }
    int mine = 0;
#pragma unroll
    for (int p = 0; p < PER / 16; ++p) mine += __popc(hits[p]);
    int i = atomicAdd(&count, mine);
    if (list_fits(i, mine)) {
#pragma unroll
      for (int p = 0; p < PER / 16; ++p) {
        for (uint32_t bits = hits[p]; bits != 0; bits &= bits - 1) {   // one or two in all
          const int e = 16 * p + __ffs(static_cast<int>(bits)) - 1;
          found[i++] = static_cast<uint32_t>(offset(e));
        }
      }
    }
  }
  __syncthreads();
  const int n = count;
  // as keys, the logits read again (they are in the cache); zeros among them
  // are no entries
  for (int i = tid; i < list_readable(n); i += kScanThreads) {
    const uint32_t f = found[i];
    const uint64_t key = f < static_cast<uint32_t>(len) ? rank_key(logit_at(a, row, v0 + f), v0 + f) : 0;
    list[i] = key >= cut ? key : 0;
  }
  __syncthreads();
  const int64_t at = row * a.chunks + chunk;
  if (tid == 0) {
    float all = wave_m[0];
#pragma unroll
    for (int j = 1; j < kScanWaves; ++j) all = fmaxf(all, wave_m[j]);
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < kScanWaves; ++j) sum += wave_m[j] == -INFINITY ? wave_l[j] : wave_l[j] * __expf(wave_m[j] - all);
    a.m[at] = all;
    a.l[at] = sum;
    if (len <= a.num) a.left_out[at] = -INFINITY;
  }
  auto emit = [&](int rank, uint64_t key) {
    if (rank < a.num) a.list[at * a.num + rank] = u32x2{__float_as_uint(key_value(key)), key_index(key)};
    else a.left_out[at] = key_value(key);
  };
  if (n <= kScanList) {
    for (int i = tid; i < n; i += kScanThreads) {
      const uint64_t key = list[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += list[j] > key;
      if (rank <= a.num && key != 0) emit(rank, key);
    }
    for (int i = len + tid; i < a.num; i += kScanThreads) a.list[at * a.num + i] = u32x2{0u, ~0u};
    return;
  }
  // more logits above the bound than fit (all in few threads): one by one
  uint64_t last = ~uint64_t(0);
  for (int r = 0; r <= a.num; ++r) {
    uint64_t best = 0;
    for (int i = tid; i < len; i += kScanThreads) {
      const uint64_t key = rank_key(logit_at(a, row, v0 + i), v0 + i);
      best = key < last && key > best ? key : best;
    }
    best = wave_max(best);
    __syncthreads();
    if (lane == 0) slots[wave] = best;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kScanWaves; ++j) best = slots[j] > best ? slots[j] : best;
    if (tid == 0) emit(r, best);
    last = best;
  }
}

constexpr int kJoinThreads = 1024;
constexpr int kJoinWaves = kJoinThreads / 64;
constexpr int kJoinList = 2048;                // candidates ranked at once
constexpr int kJoinHeld = 4;                   // list entries a thread holds in registers

__device__ __forceinline__ float candidate(float score, float x, float lse) {
  const float c = score + (x - lse);
  return c != c ? -INFINITY : c;
}

__device__ __forceinline__ uint64_t block_max(uint64_t v, uint64_t *slots) {
  v = wave_max(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
  __syncthreads();
  for (int j = 0; j < kJoinWaves; ++j) v = slots[j] > v ? slots[j] : v;
  return v;
}

// The next logit below a finite x that the logits' type can hold.
__device__ __forceinline__ float just_below(float x, bool f32) {
  const uint32_t u = __float_as_uint(x), step = f32 ? 1u : 0x10000u;
  return __uint_as_float(x > 0.0f ? u - step : x < 0.0f ? u + step : 0x80000000u + step);
}

// Whether a chunk that left `next` out, as the best of what its full list does
// not hold, may hold a logit below `next` with next's score c.  c does not fall
// where x rises, so the one just below decides.  In a row whose lse is NaN every
// logit's c is -infinity.  Nothing ranks below NaN, and in a row with a number
// for lse, so without NaN, nothing below -infinity.
__device__ __forceinline__ bool lower_ties(float score, float next, float lse, bool f32) {
  if (next != next) return false;
  if (lse != lse) return true;
  return next != -INFINITY &&
         ordered(candidate(score, just_below(next, f32), lse)) == ordered(candidate(score, next, lse));
}

// One workgroup per batch item.
__global__ __launch_bounds__(kJoinThreads) void beam_join_kernel(BeamArgs a) {
  extern __shared__ float lse[];               // [W], then the scores [W]
  float *score = lse + a.W;
  __shared__ uint64_t list[kJoinList];
  __shared__ uint64_t slots[kJoinWaves];
  __shared__ uint64_t winner_min;
  __shared__ uint32_t sums[kJoinWaves];
  __shared__ int count, tie, above;
  const int b = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row0 = static_cast<int64_t>(b) * a.W;
  if (tid == 0) count = tie = above = 0;
  // the entries of the lists that a thread holds itself, on their way early
  const int total = a.W * a.chunks * a.num;
  const u32x2 *entries = a.list + row0 * a.chunks * a.num;
  u32x2 held[kJoinHeld];
#pragma unroll
  for (int j = 0; j < kJoinHeld; ++j) {
    const int i = tid + j * kJoinThreads;
    held[j] = entries[min(i, total - 1)];
    if (i >= total) held[j][1] = ~0u;
  }
  for (int w = wave; w < a.W; w += kJoinWaves) {
    float m = -INFINITY, l = 0.0f;
    for (int c = lane; c < a.chunks; c += 64) {
      const float mc = a.m[(row0 + w) * a.chunks + c], lc = a.l[(row0 + w) * a.chunks + c];
      const float hi = fmaxf(m, mc), base = hi == -INFINITY ? 0.0f : hi;
      l = l * __expf(m - base) + lc * __expf(mc - base);
      m = hi;
    }
    const float all = wave_max(m);
    l = wave_sum(l * __expf(m - (all == -INFINITY ? 0.0f : all)));
    if (lane == 0) {
      lse[w] = all + logf(l);
      score[w] = a.scores[row0 + w];
    }
  }
  __syncthreads();
  auto key_of = [&](int i, u32x2 e) -> uint64_t {
    const uint32_t w = div_by(static_cast<uint32_t>(i), a.per_row);
    if (e[1] == ~0u) return 0;
    return rank_key(candidate(score[w], __uint_as_float(e[0]), lse[w]), w * static_cast<uint32_t>(a.V) + e[1]);
  };
  auto each = [&](auto &&f) {
#pragma unroll
    for (int j = 0; j < kJoinHeld; ++j) f(key_of(tid + j * kJoinThreads, held[j]));
    for (int i = tid + kJoinHeld * kJoinThreads; i < total; i += kJoinThreads) f(key_of(i, entries[i]));
  };
  uint64_t best = 0;
  each([&](uint64_t k) { best = k > best ? k : best; });
  const uint64_t cut_w = wave_bound(static_cast<uint32_t>(best >> 32), a.num, [&] { return static_cast<uint32_t>(best); });
  if (lane == 0) slots[wave] = cut_w;
  __syncthreads();
  uint64_t cut = 0;
#pragma unroll
  for (int j = 0; j < kJoinWaves; ++j) cut = slots[j] > cut ? slots[j] : cut;
  if (best >= cut) {
    each([&](uint64_t k) {
      if (k != 0 && k >= cut) {
        const int p = atomicAdd(&count, 1);
        if (p < kJoinList) list[p] = k;
      }
    });
  }
  __syncthreads();
  int n = count;
  if (__builtin_expect(n > kJoinList, 0)) {    // a few threads hold most of the entries: the winners one by one
    uint64_t last = ~uint64_t(0);
    for (int r = 0; r < a.num; ++r) {
      uint64_t top = 0;
#pragma nounroll
      for (int i = tid; i < total; i += kJoinThreads) {
        const uint64_t k = key_of(i, entries[i]);
        top = k < last && k > top ? k : top;
      }
      top = block_max(top, slots);
      if (tid == 0) list[r] = top;
      last = top;
    }
    n = a.num;
    __syncthreads();
  }
  const int64_t out = static_cast<int64_t>(b) * a.num;
  auto write = [&](int rank, uint64_t key) {
    const uint32_t i = key_index(key), w = i / static_cast<uint32_t>(a.V);
    a.out_scores[out + rank] = key_value(key);
    a.out_parents[out + rank] = static_cast<int32_t>(w);
    a.out_tokens[out + rank] = static_cast<int32_t>(i - w * static_cast<uint32_t>(a.V));
  };
  for (int i = tid; i < n; i += kJoinThreads) {
    const uint64_t key = list[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += list[j] > key;
    if (rank < a.num) write(rank, key);
    if (rank == a.num - 1) winner_min = key;
  }
  __syncthreads();
  // a logit that no list holds, yet ties with the threshold ahead of a
  // listed one: it lies in a chunk whose list is full, at or below the best
  // logit left out there.  Where it equals that one, the listed logits equal to
  // it come first, and only a larger listed one with the same c may not.
  const uint32_t t = static_cast<uint32_t>(winner_min >> 32);
  for (int i = tid; i < a.W * a.chunks; i += kJoinThreads) {
    const int w = static_cast<int>(div_by(static_cast<uint32_t>(i), a.per_chunk));
    const u32x2 *mine = a.list + (row0 * a.chunks + i) * a.num;
    const float next = a.left_out[row0 * a.chunks + i];
    if (mine[a.num - 1][1] == ~0u) continue;
    if (ordered(candidate(score[w], next, lse[w])) != t) continue;
    if (lower_ties(score[w], next, lse[w], a.f32)) tie = 1;
    for (int j = 0; j < a.num; ++j) {
      const float x = __uint_as_float(mine[j][0]);
      if (!(x == next) && ordered(candidate(score[w], x, lse[w])) == t) tie = 1;
    }
  }
  __syncthreads();
  if (__builtin_expect(!tie, 1)) return;
  for (int i = tid; i < n; i += kJoinThreads)
    if (static_cast<uint32_t>(list[i] >> 32) > t) atomicAdd(&above, 1);
  __syncthreads();
  // in the ranks below those, the lowest indices that tie, eight logits a thread
  // at a time
  int filled = above;
  for (int w = 0; w < a.W && filled < a.num; ++w) {
    const float of = score[w], by = lse[w];
    for (int64_t v0 = 0; v0 < a.V && filled < a.num; v0 += 8 * kJoinThreads) {
      const int64_t v = v0 + 8 * tid;
      float x[8];
      if (v + 8 <= a.V) {
        load8(a, (row0 + w) * a.logits_ld + v, x);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = v + e < a.V ? logit_at(a, row0 + w, static_cast<int>(v) + e) : 0.0f;
      }
      uint32_t hits = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) hits |= (v + e < a.V && ordered(candidate(of, x[e], by)) == t ? 1u : 0u) << e;
      const uint32_t mine = __popc(hits), upto = wave_scan(mine);
      if (lane == 63) sums[wave] = upto;
      __syncthreads();
      int at = filled + static_cast<int>(upto - mine);
#pragma unroll
      for (int j = 0; j < kJoinWaves; ++j) {
        at += j < wave ? static_cast<int>(sums[j]) : 0;
        filled += static_cast<int>(sums[j]);
      }
      for (; hits != 0 && at < a.num; hits &= hits - 1, ++at) {
        const uint32_t i = static_cast<uint32_t>(w) * static_cast<uint32_t>(a.V) + static_cast<uint32_t>(v) +
                           static_cast<uint32_t>(__ffs(static_cast<int>(hits)) - 1);
        write(at, (static_cast<uint64_t>(t) << 32) | (0xFFFFFFFFu - i));
      }
      __syncthreads();                         // sums have been read
    }
  }
}

}  // namespace qmvd
