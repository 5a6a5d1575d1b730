// Kernels that write or move rows of the paged cache: appending new tokens,
// eviction by accumulated attention weight, and the reordering of beams.
#pragma once

#include <float.h>

#include "append_quick.h"
#include "kv_device.h"

namespace qmvd {

// ---------------------------------------------------------------------------
// Append: token t's key and value heads go to slot slots[t] of sequence
// rows[t] (t itself without `rows`).  A negative slot, a sequence or a page
// that does not exist writes nothing.  A decode step's append (64 tokens, 8
// heads of 128, bf16) takes 3.1 us, a launch and one chain of three loads.
// Four prompts of 2047 tokens into 8-bit rows, 51 MB in all: 21 us (2.4 TB/s),
// bound by the vector instructions of the rounding and by two rounds of that
// chain; with 64-bit divisions in the indexing and true ones in the rounding
// it took 27.
// ---------------------------------------------------------------------------
struct AppendArgs {
  const uint16_t *k, *v;                       // bf16 [T, heads, D]
  int64_t k_t, k_h, v_t, v_h;                  // strides in values
  Pools pool;
  Tables tab;
  const int32_t *rows, *slots, *token_positions;
  float *weights;                              // [B, heads, S], zero for the new slot
  int32_t *positions;                          // [B, heads, S]
  int64_t meta_b, meta_h;
  int64_t B, S;
  Divider per_token;                           // rows to tokens: by heads
  int T, heads, D, piece_bits, line_bits;      // 2^piece_bits pieces of 8 values a row
};

__device__ __forceinline__ void append_meta(const AppendArgs &a, int64_t b, int h, int slot, int64_t t) {
  if (slot >= a.S) return;
  const int64_t at = b * a.meta_b + h * a.meta_h + slot;
  if (a.weights) a.weights[at] = 0.0f;
  if (a.positions) a.positions[at] = a.token_positions ? a.token_positions[t] : slot;
}

constexpr int kAppendThreads = 256;

// bf16: one thread per 16 bytes of a key row and the same 16 of the value row.
__global__ __launch_bounds__(kAppendThreads) void append_bf16_kernel(AppendArgs a) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kAppendThreads + threadIdx.x;
  const int piece = static_cast<int>(i) & ((1 << a.piece_bits) - 1);
  const uint32_t r = static_cast<uint32_t>(i >> a.piece_bits);
  const int t = static_cast<int>(div_by(r, a.per_token)), h = static_cast<int>(r) - t * a.heads;
  if (t >= a.T) return;
  const int slot = a.slots[t];
  const int64_t b = a.rows ? a.rows[t] : t;
  if (slot < 0 || b < 0 || b >= a.B) return;
  if (piece == 0) append_meta(a, b, h, slot, t);
  const int64_t row = row_at(a.pool, a.tab, b, h, slot);
  if (row < 0) return;
  const u32x4 kk = *reinterpret_cast<const u32x4 *>(a.k + t * a.k_t + h * a.k_h + piece * 8);
  const u32x4 vv = *reinterpret_cast<const u32x4 *>(a.v + t * a.v_t + h * a.v_h + piece * 8);
  const int64_t at = row * (2 * a.D) + piece * 16;
  *reinterpret_cast<u32x4 *>(const_cast<uint8_t *>(a.pool.k) + at) = kk;
  *reinterpret_cast<u32x4 *>(const_cast<uint8_t *>(a.pool.v) + at) = vv;
}

// Codes: the steps of qmv_pack's quantizer on the bf16 values, eight values a
// lane (GS/8 lanes per group), so the eight codes are one or two whole words.
// Each step is one IEEE fp32 operation (no contraction), as in qmv_pack.
template <int BITS, int GS>
struct Quantized {
  uint32_t word[BITS / 4];
  float scale, bias;

  __device__ __forceinline__ explicit Quantized(u32x4 raw) {
    constexpr int LPG = GS / 8;
    float x[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // a signalling NaN would not be passed over by min and max, but end them
      x[2 * e] = __builtin_canonicalizef(__uint_as_float(raw[e] << 16));
      x[2 * e + 1] = __builtin_canonicalizef(__uint_as_float(raw[e] & 0xFFFF0000u));
    }
    float lo = FLT_MAX, hi = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {           // fminf would quiet each operand once more
      asm("v_min3_f32 %0, %0, %1, %2" : "+v"(lo) : "v"(x[e]), "v"(x[e + 1]));
      asm("v_max3_f32 %0, %0, %1, %2" : "+v"(hi) : "v"(x[e]), "v"(x[e + 1]));
    }
    // over the group's lanes, which are neighbours (mirrors stand for the
    // wider exchanges: by then the mirrored quads hold one value each)
    auto join = [&](auto ctrl) {
      constexpr int kCtrl = decltype(ctrl)::value;
      lo = fminf(lo, __uint_as_float(dpp<kCtrl>(__float_as_uint(lo))));
      hi = fmaxf(hi, __uint_as_float(dpp<kCtrl>(__float_as_uint(hi))));
    };
    join(std::integral_constant<int, 0xB1>{});
    join(std::integral_constant<int, 0x4E>{});
    if constexpr (LPG >= 8) join(std::integral_constant<int, 0x141>{});
    if constexpr (LPG >= 16) join(std::integral_constant<int, 0x140>{});
    const float top = static_cast<float>((1 << BITS) - 1);
    float s = (hi - lo) / top;
    s = s < 1e-7f ? 1e-7f : s;
    const bool side = fabsf(lo) > fabsf(hi);
    s = side ? s : -s;
    const float edge = side ? lo : hi;
    const float q0 = roundf(edge / s);
    float z = 0.0f;
    if (q0 != 0.0f) {
      s = edge / q0;
      z = edge;
    }
    // q = min(round((x - z) / s), top), by the reciprocal of s where that is sure
    // to give the same code (append_quick.h)
    constexpr float kNear = quick_near(BITS);
    const float inverse = __builtin_amdgcn_rcpf(s);
    uint32_t byte[2] = {0u, 0u};
    float far = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float r = quick_quotient(x[e], z, inverse);
      far = fmaxf(far, fabsf(r - __builtin_rintf(r)));
      // 0 to 255, NaN as 0; the median of NaN and two numbers is the smaller one
      byte[e / 4] = __builtin_amdgcn_cvt_pk_u8_f32(BITS == 8 ? r : __builtin_amdgcn_fmed3f(r, 0.0f, top), e % 4, byte[e / 4]);
    }
    if (!(far < 0.5f - kNear)) {
      byte[0] = byte[1] = 0u;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float r = roundf((x[e] - z) / s);
        byte[e / 4] |= static_cast<uint32_t>(static_cast<int>(r > top ? top : r)) << (8 * (e % 4));
      }
    }
    if constexpr (BITS == 8) {
      word[0] = byte[0];
      word[1] = byte[1];
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {            // nibbles of bytes 0 1 and 2 3 side by side
        const uint32_t pair = byte[i] | (byte[i] >> 4);
        byte[i] = (pair & 0xFFu) | ((pair >> 8) & 0xFF00u);
      }
      word[0] = byte[0] | (byte[1] << 16);
    }
    scale = s;
    bias = z;
  }

  __device__ __forceinline__ void store(const uint8_t *pool, const uint16_t *scales, const uint16_t *biases, int64_t row,
                                        int D, int piece) const {
    uint8_t *to = const_cast<uint8_t *>(pool) + row * (D * BITS / 8) + piece * BITS;
    if constexpr (BITS == 8) *reinterpret_cast<u32x2 *>(to) = u32x2{word[0], word[1]};
    else *reinterpret_cast<uint32_t *>(to) = word[0];
    if (piece % (GS / 8) == 0) {
      const int64_t g = row * (D / GS) + piece / (GS / 8);
      const_cast<uint16_t *>(scales)[g] = qmvk::f32_to_bf16(scale);
      const_cast<uint16_t *>(biases)[g] = qmvk::f32_to_bf16(bias);
    }
  }
};

// A thread takes eight values of a key row and the same of the value row, so
// that finding the row is paid once for both.  In prompts 16 tokens in line
// are next to each other before the next head is, as their rows are.
template <int BITS, int GS>
__global__ __launch_bounds__(kAppendThreads) void append_codes_kernel(AppendArgs a) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kAppendThreads + threadIdx.x;
  const int piece = static_cast<int>(i) & ((1 << a.piece_bits) - 1);
  const uint32_t r = static_cast<uint32_t>(i >> a.piece_bits), line = r >> a.line_bits;
  const int lines = static_cast<int>(div_by(line, a.per_token)), h = static_cast<int>(line) - lines * a.heads;
  const int t = (lines << a.line_bits) + static_cast<int>(r & ((1u << a.line_bits) - 1));
  const bool in = t < a.T;
  u32x4 key = {0u, 0u, 0u, 0u}, value = {0u, 0u, 0u, 0u};
  int64_t b = -1, row = -1;
  int slot = -1;
  if (in) {
    slot = a.slots[t];
    b = a.rows ? a.rows[t] : t;
    key = *reinterpret_cast<const u32x4 *>(a.k + t * a.k_t + h * a.k_h + piece * 8);
    value = *reinterpret_cast<const u32x4 *>(a.v + t * a.v_t + h * a.v_h + piece * 8);
  }
  if (slot >= 0 && b >= 0 && b < a.B) {
    if (piece == 0) append_meta(a, b, h, slot, t);
    row = row_at(a.pool, a.tab, b, h, slot);
  }
  const Quantized<BITS, GS> k(key), v(value);  // lanes of a group work together
  if (row < 0) return;
  k.store(a.pool.k, a.pool.ks, a.pool.kb, row, a.D, piece);
  v.store(a.pool.v, a.pool.vs, a.pool.vb, row, a.D, piece);
}

// ---------------------------------------------------------------------------
// Eviction.  Per (sequence, head) the entries are ranked: the protected ones
// (position >= next - recent) first, then by weight, ties to the lowest slot;
// the first `budget` stay.  Attention does not look at the order of slots, so
// nothing is compacted: a survivor at or past the budget moves into a hole
// below it, the i-th into the i-th hole.  Sources lie at or past the budget and
// destinations below it, so moves never overlap.
//
// Ranking is a radix selection of the budget-th key (three histograms in LDS)
// by one workgroup a head: it wants barriers, not bandwidth.  Moving rows is
// bandwidth, and a kernel of its own over the whole machine.  On MI355X, 4
// prompts of 32768 entries, 8 heads of 128, bf16, to 4096: 23 us for the ranks
// (256 KB a workgroup) and 33 us for 117 MB of rows (3.6 TB/s: 256-byte rows, half of them scattered); with
// keys read again at each of four 8-bit digits and one thread looking for each
// digit the ranks took 132.  32 sequences of 2112 to 2048: 10.4 + 5.0 us, eight
// barriers and two chains of loads.
// ---------------------------------------------------------------------------
struct EvictArgs {
  Pools pool;
  Tables tab;
  const int32_t *lengths, *next;
  const float *weights;
  const int32_t *positions;                    // [B, heads, S], strides shared with weights
  int64_t meta_b, meta_h;
  float *weights_out;
  int32_t *positions_out, *lengths_out;        // [B, heads, S] contiguous, [B]
  int32_t *moves;                              // [B*heads][2][most]: holes, sources
  int32_t *counts;                             // [B*heads]
  uint64_t *stay;                              // [B*heads][mask_words]: a bit per slot below the budget, 4 words for 256
  int mask_words;
  int heads, S, budget, recent, most;
  int row_bytes, groups;                       // groups: scales a row (0 for bf16)
};

constexpr int kEvictThreads = 1024;
constexpr int kEvictWaves = kEvictThreads / 64;
constexpr int kEvictBins = 2048;

__device__ __forceinline__ uint32_t evict_key(float w, int pos, int64_t first_safe) {
  return pos >= first_safe ? 0xFFFFFFFFu : ordered(w);
}

// Where the rank `left` (1-based, from the largest digit down) falls in a
// histogram of kEvictBins digits: {digit, rank inside it, count of it}.  Two
// bins a thread.
__device__ __forceinline__ void rank_in_histogram(const int *hist, int left, int *wave_sum, int *pick) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int hi = kEvictBins - 1 - 2 * tid;     // this thread's bins: hi, hi - 1
  const int a = hist[hi], c = hist[hi - 1];
  int sum = a + c;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(sum, off, 64);
    if (lane >= off) sum += o;
  }
  if (lane == 63) wave_sum[wave] = sum;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kEvictWaves; ++j) sum += j < wave ? wave_sum[j] : 0;
  const int before = sum - a - c;
  if (left > before && left <= sum) {
    const bool first = left <= before + a;
    pick[0] = first ? hi : hi - 1;
    pick[1] = left - before - (first ? 0 : a);
    pick[2] = first ? a : c;
  }
  __syncthreads();
}

// One workgroup per (sequence, head).  Every wave owns a contiguous run of
// slots, so ranks in slot order need one total a wave and no barrier inside a
// run; a lane takes four slots in line at a time (a step: 256 slots a wave).
// RESIDENT: the entries are read once and their keys stay in LDS (4 bytes
// each, up to kEvictResident); otherwise they are read again from the cache at
// each of the passes.
constexpr int kEvictResident = 32768;
constexpr int kEvictStep = 256;

template <bool RESIDENT>
__global__ __launch_bounds__(kEvictThreads) void evict_select_kernel(EvictArgs a) {
  extern __shared__ u32x4 keys[];              // RESIDENT: [run * kEvictWaves / 4]
  __shared__ int hist[3][kEvictBins];
  __shared__ int wave_sum[5][kEvictWaves];
  __shared__ int pick[3][3];
  const int bh = blockIdx.x, b = bh / a.heads, h = bh % a.heads;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t cap = static_cast<int64_t>(a.tab.cols) * a.pool.page_size;
  const int n = clamp_length(a.lengths[b], cap < a.S ? cap : a.S);
  const int keep = n < a.budget ? n : a.budget;
  const float *w = a.weights + b * a.meta_b + h * a.meta_h;
  const int32_t *pos = a.positions + b * a.meta_b + h * a.meta_h;
  const int64_t first_safe = static_cast<int64_t>(a.next[b]) - a.recent;
  if (h == 0 && tid == 0) a.lengths_out[b] = keep;
  if (n <= a.budget) {
    if (tid == 0) a.counts[bh] = 0;
    return;
  }

  const int steps = (n + kEvictWaves * kEvictStep - 1) / (kEvictWaves * kEvictStep), first = wave * steps * kEvictStep;
#pragma unroll
  for (int i = 0; i < 3 * kEvictBins / kEvictThreads; ++i) (&hist[0][0])[tid + i * kEvictThreads] = 0;
  __syncthreads();
  // f(step, the lane's first slot, its four keys), in slot order; slots at or
  // past n have no meaning
  auto each = [&](auto &&f) {
#pragma unroll 2
    for (int j = 0; j < steps; ++j) {
      const int i = first + j * kEvictStep + 4 * lane;
      u32x4 key;
      if constexpr (RESIDENT) {
        key = keys[i >> 2];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int at = min(i + e, n - 1);
          key[e] = evict_key(w[at], pos[at], first_safe);
        }
      }
      f(j, i, key);
    }
  };
  // the keep-th largest key, eleven, eleven and ten bits from the top; the
  // loads of eight entries a lane in flight together, sixteen bytes each where
  // the rows allow it
  auto take = [&](int i, float wi, int pi) {
    const uint32_t key = evict_key(wi, pi, first_safe);
    if constexpr (RESIDENT) reinterpret_cast<uint32_t *>(keys)[i] = key;
    if (i < n) atomicAdd(&hist[0][key >> 21], 1);
  };
  if (((reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(pos)) & 15) == 0) {
    const int whole = n & ~3;
    for (int i0 = 4 * tid; i0 < whole; i0 += 8 * 4 * kEvictThreads) {
      f32x4 wv[8];
      u32x4 pv[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = min(i0 + j * 4 * kEvictThreads, whole - 4);
        wv[j] = *reinterpret_cast<const f32x4 *>(w + at);
        pv[j] = *reinterpret_cast<const u32x4 *>(pos + at);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = i0 + j * 4 * kEvictThreads;
        if (i < whole) {
#pragma unroll
          for (int e = 0; e < 4; ++e) take(i + e, wv[j][e], static_cast<int>(pv[j][e]));
        }
      }
    }
    if (whole + tid < n) take(whole + tid, w[whole + tid], pos[whole + tid]);
  } else {
#pragma unroll 8
    for (int i = tid; i < n; i += kEvictThreads) take(i, w[i], pos[i]);
  }
  __syncthreads();
  rank_in_histogram(hist[0], keep, wave_sum[0], pick[0]);
  uint32_t prefix = static_cast<uint32_t>(pick[0][0]) << 21;
  each([&](int, int i, u32x4 key) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < n && ((key[e] ^ prefix) >> 21) == 0) atomicAdd(&hist[1][(key[e] >> 10) & 2047], 1);
  });
  __syncthreads();
  rank_in_histogram(hist[1], pick[0][1], wave_sum[1], pick[1]);
  prefix |= static_cast<uint32_t>(pick[1][0]) << 10;
  each([&](int, int i, u32x4 key) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < n && ((key[e] ^ prefix) >> 10) == 0) atomicAdd(&hist[2][key[e] & 1023], 1);
  });
  __syncthreads();
  rank_in_histogram(hist[2], pick[1][1], wave_sum[2], pick[2]);
  prefix |= static_cast<uint32_t>(pick[2][0]);

  // `left` of the entries equal to the threshold stay, the lowest slots
  // first; only where some of them go do their ranks matter
  const int left = pick[2][1];
  const bool ties = left < pick[2][2];
  const uint64_t below = (uint64_t(1) << lane) - 1;
  // four flags a lane, in slot order: how many lie in lower lanes, how many in all
  struct Flags {
    uint64_t mask[4];
    int before, all;
  };
  auto count = [&](bool f0, bool f1, bool f2, bool f3) {
    Flags r{{__ballot(f0), __ballot(f1), __ballot(f2), __ballot(f3)}, 0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      r.before += __popcll(r.mask[e] & below);
      r.all += __popcll(r.mask[e]);
    }
    return r;
  };
  int eq = 0;                                  // equal entries in lower runs, then in this run so far
  if (ties) {
    int mine = 0;
    each([&](int, int i, u32x4 key) {
#pragma unroll
      for (int e = 0; e < 4; ++e) mine += __popcll(__ballot(i + e < n && key[e] == prefix));
    });
    if (lane == 0) wave_sum[0][wave] = mine;
    __syncthreads();
    for (int j = 0; j < wave; ++j) eq += wave_sum[0][j];
  }
  const int eq0 = eq;
  // the lane's entries that stay, as four bits
  auto stays = [&](int i, u32x4 key) {
    uint32_t bits = 0;
    if (!ties) {
#pragma unroll
      for (int e = 0; e < 4; ++e) bits |= (i + e < n && key[e] >= prefix ? 1u : 0u) << e;
      return bits;
    }
    bool same[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) same[e] = i + e < n && key[e] == prefix;
    const Flags f = count(same[0], same[1], same[2], same[3]);
    int rank = eq + f.before;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      bits |= (i + e < n && (key[e] > prefix || (same[e] && rank < left)) ? 1u : 0u) << e;
      rank += same[e];
    }
    eq += f.all;
    return bits;
  };
  // RESIDENT: a run is at most eight steps, and its bits fit a register
  uint32_t stay_bits = 0;
  int holes_here = 0, sources_here = 0;
  each([&](int j, int i, u32x4 key) {
    const uint32_t bits = stays(i, key);
    if constexpr (RESIDENT) stay_bits |= bits << (4 * j);
    const int base = first + j * kEvictStep;
    if (base < keep) {
#pragma unroll
      for (int e = 0; e < 4; ++e) holes_here += __popcll(__ballot(i + e < keep && !((bits >> e) & 1)));
    }
    if (base + kEvictStep > keep) {
#pragma unroll
      for (int e = 0; e < 4; ++e) sources_here += __popcll(__ballot(i + e >= keep && ((bits >> e) & 1)));
    }
  });
  if (lane == 0) {
    wave_sum[3][wave] = holes_here;
    wave_sum[4][wave] = sources_here;
  }
  __syncthreads();
  int hole0 = 0, source0 = 0, moves = 0;
#pragma unroll
  for (int j = 0; j < kEvictWaves; ++j) {
    hole0 += j < wave ? wave_sum[3][j] : 0;
    source0 += j < wave ? wave_sum[4][j] : 0;
    moves += wave_sum[3][j];
  }
  int32_t *holes = a.moves + static_cast<int64_t>(bh) * 2 * a.most, *sources = holes + a.most;
  uint64_t *stay = a.stay + static_cast<int64_t>(bh) * a.mask_words;
  eq = eq0;
  auto list = [&](int j, int i, uint32_t bits) {
    const int base = first + j * kEvictStep;
    if (base < keep) {                         // keep <= n: all these slots exist
      bool hole[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) hole[e] = i + e < keep && !((bits >> e) & 1);
      const Flags f = count(hole[0], hole[1], hole[2], hole[3]);
      int at = hole0 + f.before;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (hole[e]) holes[at++] = i + e;
      hole0 += f.all;
      // word e of a step: a bit for slot 4 lane + e
      if (lane < 4) {
        const uint64_t m01 = lane == 0 ? f.mask[0] : f.mask[1], m23 = lane == 2 ? f.mask[2] : f.mask[3];
        stay[(base >> 8) * 4 + lane] = ~(lane < 2 ? m01 : m23);
      }
    }
    if (base + kEvictStep > keep) {
      bool source[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) source[e] = i + e >= keep && ((bits >> e) & 1);
      const Flags f = count(source[0], source[1], source[2], source[3]);
      int at = source0 + f.before;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (source[e]) sources[at++] = i + e;
      source0 += f.all;
    }
  };
  if constexpr (RESIDENT) {
    for (int j = 0; j < steps; ++j) list(j, first + j * kEvictStep + 4 * lane, stay_bits >> (4 * j));
  } else {
    each([&](int j, int i, u32x4 key) { list(j, i, stays(i, key)); });
  }
  if (tid == 0) a.counts[bh] = moves;
}

// One move per 16 lanes: 16-byte pieces of the key and the value row by
// consecutive lanes, the few bytes of scales and biases, and the entry's
// weight and position, by the first ones.
constexpr int kMoveThreads = 256;

__device__ __forceinline__ void copy_row(const Pools &p, int64_t to, int64_t from, int row_bytes, int groups,
                                         int lane, int lanes) {
  for (int c = lane * 16; c < row_bytes; c += lanes * 16) {
    const u32x4 x = *reinterpret_cast<const u32x4 *>(p.k + from * row_bytes + c);
    const u32x4 y = *reinterpret_cast<const u32x4 *>(p.v + from * row_bytes + c);
    *reinterpret_cast<u32x4 *>(const_cast<uint8_t *>(p.k) + to * row_bytes + c) = x;
    *reinterpret_cast<u32x4 *>(const_cast<uint8_t *>(p.v) + to * row_bytes + c) = y;
  }
  for (int g = lane; g < groups; g += lanes) {
    const_cast<uint16_t *>(p.ks)[to * groups + g] = p.ks[from * groups + g];
    const_cast<uint16_t *>(p.kb)[to * groups + g] = p.kb[from * groups + g];
    const_cast<uint16_t *>(p.vs)[to * groups + g] = p.vs[from * groups + g];
    const_cast<uint16_t *>(p.vb)[to * groups + g] = p.vb[from * groups + g];
  }
}

// The bookkeeping of slots that no move writes: entries that stay, nothing
// past the new length.
__device__ __forceinline__ void evict_meta(const EvictArgs &a, int bh, int b, int h, int count, int part, int parts) {
  const int64_t cap = static_cast<int64_t>(a.tab.cols) * a.pool.page_size;
  const int n = clamp_length(a.lengths[b], cap < a.S ? cap : a.S);
  const int keep = n < a.budget ? n : a.budget;
  const int64_t in = b * a.meta_b + h * a.meta_h, out = static_cast<int64_t>(bh) * a.S;
  const uint64_t *stay = a.stay + static_cast<int64_t>(bh) * a.mask_words;
  // unsigned: the step past the last slot can pass 2^31
  for (uint32_t i = part * kMoveThreads + threadIdx.x; i < static_cast<uint32_t>(a.S); i += parts * kMoveThreads) {
    if (i >= static_cast<uint32_t>(keep)) {
      a.weights_out[out + i] = 0.0f;
      a.positions_out[out + i] = -1;
    } else if (count == 0 || ((stay[(i >> 8) * 4 + (i & 3)] >> ((i >> 2) & 63)) & 1)) {
      a.weights_out[out + i] = a.weights[in + i];
      a.positions_out[out + i] = a.positions[in + i];
    }
  }
}

// `move_parts` workgroups of each (sequence, head) move rows, `meta_parts`
// more bring the bookkeeping over.
__global__ __launch_bounds__(kMoveThreads) void evict_move_kernel(EvictArgs a, int move_parts, int meta_parts) {
  const int parts = move_parts + meta_parts, part = blockIdx.x % parts;
  const int bh = blockIdx.x / parts, b = bh / a.heads, h = bh % a.heads;
  const int count = a.counts[bh];
  if (part >= move_parts) {
    evict_meta(a, bh, b, h, count, part - move_parts, meta_parts);
    return;
  }
  const int32_t *holes = a.moves + static_cast<int64_t>(bh) * 2 * a.most, *sources = holes + a.most;
  constexpr int kLanes = 16, kRows = kMoveThreads / kLanes;
  const int sub = threadIdx.x % kLanes;
  for (int i = part * kRows + threadIdx.x / kLanes; i < count; i += move_parts * kRows) {
    const int d = holes[i], s = sources[i];
    if (sub == 0) {
      const int64_t in = b * a.meta_b + h * a.meta_h + s, out = static_cast<int64_t>(bh) * a.S + d;
      a.weights_out[out] = a.weights[in];
      a.positions_out[out] = a.positions[in];
    }
    const int64_t to = row_at(a.pool, a.tab, b, h, d), from = row_at(a.pool, a.tab, b, h, s);
    if (to >= 0 && from >= 0) copy_row(a.pool, to, from, a.row_bytes, a.groups, sub, kLanes);
  }
}

// ---------------------------------------------------------------------------
// Reordering of beams.  New beam i of batch item b continues old beam
// parents[b, i]: it takes over the parent's full pages by number, and gets a
// copy of the parent's last, partly filled page in the free page given for it
// (an empty page where the parent's last one is full).  Launch bound: 3.4 us for
// 4 beams, 5 for 128 beams' tables and 8 MB of last pages.
// ---------------------------------------------------------------------------
struct ReorderArgs {
  Pools pool;
  const int32_t *tables, *lengths;             // [B, W, cols], [B, W], contiguous
  const int32_t *parents;                      // [B, M], row stride parents_ld
  const int32_t *spare;                        // [B, M]
  int32_t *tables_out, *lengths_out;           // [B, M, cols], [B, M]
  int64_t parents_ld;
  Divider per_page;
  int W, M, cols, heads, row_bytes, groups, parts;
};

constexpr int kReorderThreads = 256;

__global__ __launch_bounds__(kReorderThreads) void reorder_kernel(ReorderArgs a) {
  const int row = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
  const int b = row / a.M, i = row % a.M;
  const int parent = a.parents[b * a.parents_ld + i];
  const bool live = parent >= 0 && parent < a.W;
  const int64_t from_row = static_cast<int64_t>(b) * a.W + (live ? parent : 0);
  const int n = live ? clamp_length(a.lengths[from_row], static_cast<int64_t>(a.cols) * a.pool.page_size) : 0;
  const int full = static_cast<int>(div_by(static_cast<uint32_t>(n), a.per_page));
  const int tail = n - full * a.pool.page_size;
  const int32_t *src = a.tables + from_row * a.cols;
  const int spare = a.spare[row];
  if (part == 0) {
    for (int c = threadIdx.x; c < a.cols; c += kReorderThreads)
      a.tables_out[static_cast<int64_t>(row) * a.cols + c] = c < full ? src[c] : (c == full ? spare : -1);
    if (threadIdx.x == 0) a.lengths_out[row] = n;
    return;
  }
  if (tail == 0) return;                       // then full < cols: n <= cols * page_size
  const int old = src[full];
  if (old < 0 || old >= a.pool.pages || spare < 0 || spare >= a.pool.pages || old == spare) return;
  constexpr int kLanes = 16, kRows = kReorderThreads / kLanes;
  const int sub = threadIdx.x % kLanes;
  for (int r = (part - 1) * kRows + threadIdx.x / kLanes; r < a.heads * tail; r += (a.parts - 1) * kRows) {
    const int h = r / tail, s = r - h * tail;
    copy_row(a.pool, row_of(a.pool, spare, h, s), row_of(a.pool, old, h, s), a.row_bytes, a.groups, sub, kLanes);
  }
}

}  // namespace qmvd
