// Attention of one new token per sequence over its paged keys and values.
//
//   s_t = scale * q . k_t + mask_t,   m = max_t s_t,   p_t = exp(s_t - m)
//   y = sum_t p_t v_t / sum_t p_t,    lse = m + ln sum_t p_t
//
// for t below the sequence's length, per query head; `group` query heads share
// one key-value head.  Every key and value row is read once for the whole
// group, so memory bounds it: 4 flop a byte for each query head of the group
// on bf16 rows.  A length is cut into chunks that workgroups take in parallel
// (struct Chunks), a chunk into tiles of 32 tokens that its waves take in turn,
// each wave with its own running maximum, sum and weighted values; a workgroup
// joins its waves in LDS, attend_finish_kernel joins the chunks.
//
// Both products run on the matrix cores with the tokens on rows, so that no
// value ever changes lanes: scores S^T = K Q^T (16 keys x 16 heads a step) leave
// head n of keys 4 g + r in lane 16 g + n, which is just where P^T has to be for
// out^T += V^T P^T; only the choice of tokens for V's lanes follows from that.
// What 16 columns cost beyond the group's heads is matrix-core time, of which
// memory leaves plenty (8-bit rows: busy 256 of about 6000 cycles a tile).
//
// Why this shape, on MI355X: tiles in registers with one tile of loads in
// flight behind the one at work, 2 (bf16 rows, D = 128) to 4 waves a SIMD.  32
// sequences of 12000 to 16384 tokens, 8 heads of 128, 4 queries each, bf16: 320
// to 329 us, 5.7 to 5.8 TB/s (without the tile ahead: 343); three waves a SIMD
// spill (336 -> 343 in a graph).  131071 tokens, 8-bit rows, 8 queries each: 68
// us (4.2 TB/s; without the tile ahead 118); 40 us of it are its loop, 5 to 16
// the wait for lengths, then pages, then rows, while other workgroups' loads
// already queue.  24 sequences of 16 heads of 64, 4-bit rows: 25 us, bound by
// vector instructions (about 300 a tile of 2.5 KB: unpacking, softmax, splits).

#pragma once

#include "kv_chunks.h"
#include "kv_device.h"

namespace qmvd {

struct AttendArgs {
  const uint16_t *q;                           // bf16, strides in values
  int64_t q_b, q_h;
  Pools pool;
  Tables tab;
  const int32_t *lengths;
  const float *mask;                           // [B|1, Hq|1, >= max_len] or null
  int64_t mask_b, mask_h;
  void *y;                                     // [B, Hq, D] bf16 or fp32
  float *lse;                                  // [B, Hq] or null
  float *part;                                 // [chunk of any sequence][Hq][D]
  float *part_ml;                              // [chunk of any sequence][Hq][2]
  float *scores;                               // [B*Hq][scores_ld] or null
  int64_t scores_ld;
  int heads, group, head_blocks;               // key-value heads; query heads each; blocks of HB of them
  int max_len, waves;                          // waves a workgroup
  int whole;                                   // one workgroup per sequence and head, no chunks
  int share, most_chunk;                       // see Chunks
  float scale;                                 // of q . k into the units of the scores
  float unit, natural;                         // exp2((s - m) * unit); s * natural is in powers of e
  int f32;
};

// Weights, the accumulated attention of each cache entry.
struct WeightArgs {
  const float *in;
  float *out;                                  // [B, heads, S], strides shared
  int64_t out_b, out_h;
  int S;
};
constexpr int kWeightSlots = 512;              // slots a workgroup

constexpr int kTile = 32;                      // tokens a wave takes at a time
constexpr int kChunkWaves = 4;                 // waves a workgroup that takes a chunk
static_assert(kChunkUnit == kChunkWaves * kTile, "a tile for every wave");

// Waves a SIMD that an instance's registers are shared out for: as many as fit
// with hardly a spill (bf16 rows are held in registers, codes go through LDS;
// bf16 and 4-bit rows spill none, 8-bit rows up to 9 registers at D = 128 and, in
// groups of 32, 83 at D = 256).
constexpr int attend_waves(int D, int bits) {
  return D == 64 ? 4 : D == 128 ? (bits == 16 ? 2 : 3) : (bits == 16 ? 1 : 2);
}
// Waves a workgroup at most.
constexpr int attend_most_waves(int D) { return D == 256 ? 4 : 8; }
// Floats of LDS a wave: its rows, its scales and a tile's codes, and after the
// loop, in the same place, what it hands to the join.
constexpr int attend_wave_lds(int D, int bits, int groups, int hb) {
  const int loop = 4 * kTile + (bits == 16 ? 0 : 4 * kTile * groups + kTile * (D * bits / 8 + 16) / 4);
  const int join = hb * (D + 6);
  return loop > join ? loop : join;
}

// How lengths are cut into chunks, found on the device since that is where the
// lengths are: about `share` chunks in all (what the machine holds at once, by
// key-value head), of at least one tile a wave and at most `most_chunk` slots,
// and equal ones within a sequence.  The chunks of all sequences in line are
// numbered j = 0, 1, ...; all kernels agree on them.
struct Chunks {
  int b;                                       // the sequence
  int len, size, count;                        // its length, slots a chunk, chunks
  int first;                                   // its first chunk's j
};

// Of the sequence that chunk j belongs to (BY_J), or of sequence `want`.
// Every lane of the wave calls and gets it; b = -1: there is no chunk j.
template <bool BY_J>
__device__ __forceinline__ Chunks chunks_of(const AttendArgs &a, int want) {
  const int lane = threadIdx.x & 63, B = static_cast<int>(a.tab.B);
  Chunks c{-1, 0, 0, 0, 0};
  if (a.whole) {
    c.b = want < B ? want : -1;
    c.len = clamp_length(a.lengths[min(want, B - 1)], a.max_len);
    c.size = a.max_len;
    c.count = c.len > 0;
    c.first = want;
    return c;
  }
  // the host keeps all lengths' lines within 2^30
  auto length = [&](int i) { return i < B ? clamp_length(a.lengths[i], a.max_len) : 0; };
  const int own = length(lane);                // of the first 64 sequences
  uint32_t total = 0;
  for (int i = 0; i < B; i += 64) {
    const uint32_t lines = ((i == 0 ? own : length(i + lane)) + kChunkLine - 1) / kChunkLine;
    total += wave_all(lines, [](uint32_t x, uint32_t y) { return x + y; });
  }
  const uint32_t most = chunk_slots(total, static_cast<uint32_t>(a.share), static_cast<uint32_t>(a.most_chunk));
  uint32_t before = 0;
  for (int i = 0; i < B; i += 64) {
    const uint32_t len = i == 0 ? own : length(i + lane);
    const uint32_t count = (len + most - 1) / most, sum = before + wave_scan(count);
    const uint64_t hit = __ballot(BY_J ? static_cast<uint32_t>(want) >= sum - count && static_cast<uint32_t>(want) < sum
                                       : i + lane == want);
    if (hit != 0) {
      const int at = __ffsll(static_cast<unsigned long long>(hit)) - 1;
      const uint32_t n = __builtin_amdgcn_readlane(len, at), k = __builtin_amdgcn_readlane(count, at);
      const uint32_t even = k > 0 ? (n + k - 1) / k : 1;
      c.b = i + at;
      c.len = static_cast<int>(n);
      c.count = static_cast<int>(k);
      c.first = static_cast<int>(__builtin_amdgcn_readlane(sum, at) - k);
      c.size = static_cast<int>((even + kChunkUnit - 1) / kChunkUnit * kChunkUnit);
      return c;
    }
    before = __builtin_amdgcn_readlane(sum, 63);
  }
  return c;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// {bf16(a), bf16(b)} to nearest even, a in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  bf16x2 r = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(uint32_t, r);
}
// c minus both bf16 values of a pair times the middle of what holds a code:
// 127.5 (8 bits), 128 + 8 * 7.5 (4 bits).
template <int BITS>
__device__ __forceinline__ float take_mid(uint32_t pair, float c) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  constexpr uint32_t kMinusMid = BITS == 4 ? 0xC33CC33Cu : 0xC2FFC2FFu;
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), __builtin_bit_cast(bf16x2, kMinusMid), c, false);
}
// The high halves of a and b, a's in the low half.
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x05040100u);
}

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                 0, 0);
}

// The shapes of one instance: BITS 16 (bf16 rows, one "group" of D), 8 or 4;
// HB query heads at a time; PAGED16: the page size is a multiple of 16, so 16
// tokens in line share a page and their addresses one scalar base.
template <int BITS_, int D_, int GS_, int HB_, bool PAGED16_>
struct AttendShape {
  static constexpr int BITS = BITS_, D = D_, GS = BITS_ == 16 ? D_ : GS_, HB = HB_;
  static constexpr bool PAGED16 = PAGED16_;
  static constexpr int NG = D / GS;            // groups a row
  static constexpr int KS = D / 32;            // matrix steps over D
  static constexpr int VPL = GS / 16;          // values of a group a lane holds
  static constexpr int OT = D / 16;            // output tiles
  static constexpr int ROW = BITS == 16 ? 2 * D : D * BITS / 8;
};

// One wave's loads of VPL * BITS / 8 bytes: at most 16 at a time.
template <int BYTES>
struct Piece {
  uint32_t w[(BYTES + 3) / 4];
  __device__ __forceinline__ void load(const uint8_t *p) {
    if constexpr (BYTES == 1) w[0] = *p;
    else if constexpr (BYTES == 2) w[0] = *reinterpret_cast<const uint16_t *>(p);
    else if constexpr (BYTES == 4) w[0] = *reinterpret_cast<const uint32_t *>(p);
    else if constexpr (BYTES == 8) {
      const u32x2 v = *reinterpret_cast<const u32x2 *>(p);
      w[0] = v[0];
      w[1] = v[1];
    } else {
#pragma unroll
      for (int i = 0; i < BYTES / 16; ++i) {
        const u32x4 v = reinterpret_cast<const u32x4 *>(p)[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * i + j] = v[j];
      }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (BYTES + 3) / 4; ++i) w[i] = 0u;
  }
};

// Values j of two rows' pieces as a pair of bf16.  Codes come out exactly:
// 8-bit ones as 0..255, 4-bit ones as 128 + 8 q (the code in the top bits of
// a bf16 mantissa); the scales undo the latter.
template <int BITS, int J, int BYTES>
__device__ __forceinline__ uint32_t value_pair(const Piece<BYTES> &a, const Piece<BYTES> &b) {
  if constexpr (BITS == 16) {
    return J % 2 == 0 ? low_halves(a.w[J / 2], b.w[J / 2]) : high_halves(a.w[J / 2], b.w[J / 2]);
  } else if constexpr (BITS == 8) {
    const float x = static_cast<float>((a.w[J / 4] >> (8 * (J % 4))) & 255u);
    const float y = static_cast<float>((b.w[J / 4] >> (8 * (J % 4))) & 255u);
    return high_halves(__float_as_uint(x), __float_as_uint(y));
  } else {
    constexpr int P = J % 8, SH = 4 * (P % 4);
    const uint32_t both = P < 4 ? low_halves(a.w[J / 8], b.w[J / 8]) : high_halves(a.w[J / 8], b.w[J / 8]);
    const uint32_t at3 = SH >= 3 ? both >> (SH - 3) : both << (3 - SH);
    return (at3 & 0x00780078u) | 0x43004300u;
  }
}

// Where a wave's tile of 32 tokens lies.  Missing rows (past the chunk's end,
// or in a page that does not exist) are read from page 0, always there, and
// take no part.  The page numbers are fetched ahead, so that no tile's loads
// wait for them.
template <bool PAGED16>
struct TileRows;

// 16 tokens in line share a page: two scalar row numbers.
template <>
struct TileRows<true> {
  int64_t row[2];
  int live[2];                                 // tokens of each half that exist
  // The pages of a wave's next 32 tiles, two a tile, one a lane.
  struct Ahead {
    int page, used;
    __device__ __forceinline__ void fetch(const AttendArgs &a, int64_t b, int tile, int t1, int lane) {
      const int t = tile + (lane >> 1) * a.waves * kTile + 16 * (lane & 1);
      page = t >= tile && t < t1 ? page_of(a.tab, b, div_by(static_cast<uint32_t>(t), a.tab.per_page), a.pool.pages) : -1;
      used = 0;
    }
  };
  __device__ __forceinline__ void find(const AttendArgs &a, Ahead &pages, int64_t *, int64_t b, int h, int tile, int t1,
                                       int lane) {
    if (pages.used == 32) pages.fetch(a, b, tile, t1, lane);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = tile + 16 * u;
      const int id = __builtin_amdgcn_readlane(pages.page, 2 * pages.used + u);
      const int col = static_cast<int>(div_by(static_cast<uint32_t>(t), a.tab.per_page));
      row[u] = id < 0 ? h * a.pool.head_rows : row_of(a.pool, id, h, t - col * a.pool.page_size);
      live[u] = id < 0 ? 0 : min(16, t1 - t);
    }
    ++pages.used;
  }
  __device__ __forceinline__ bool whole() const { return live[0] + live[1] == kTile; }
  __device__ __forceinline__ bool exists(int at) const {
    return at < 16 ? at < live[0] : at - 16 < live[1];
  }
  template <int UNIT>
  __device__ __forceinline__ const uint8_t *at(const uint8_t *pool, const AttendArgs &a, int u, int in,
                                               int bytes) const {
    // a scalar base and a 32-bit lane offset that no tile changes (16 slots
    // are far below 4 GiB: attend_paged16)
    const uint8_t *base = pool + row[u] * UNIT;
    return base + static_cast<uint32_t>(in * static_cast<int>(a.pool.slot_rows) * UNIT + bytes);
  }
};

// Any page size: each lane finds one token's row, all read them from LDS.
template <>
struct TileRows<false> {
  const int64_t *rows;                         // of this tile: they alternate between two places
  bool all;
  // The page of this lane's token in the next tile.
  struct Ahead {
    int page;
    __device__ __forceinline__ void fetch(const AttendArgs &a, int64_t b, int tile, int t1, int lane) {
      const int t = tile + (lane & 31);
      const int col = static_cast<int>(div_by(static_cast<uint32_t>(min(t, t1 - 1)), a.tab.per_page));
      page = a.tab.ids[b * a.tab.ld + col];    // a slot below the length, so in the table
    }
  };
  __device__ __forceinline__ void find(const AttendArgs &a, Ahead &pages, int64_t *place, int64_t b, int h, int tile,
                                       int t1, int lane) {
    int64_t r = -1;
    const int t = tile + (lane & 31), id = pages.page;
    if (t < t1 && id >= 0 && id < a.pool.pages) {
      const int col = static_cast<int>(div_by(static_cast<uint32_t>(t), a.tab.per_page));
      r = row_of(a.pool, id, h, t - col * a.pool.page_size);
    }
    all = __ballot(r < 0) == 0;
    rows = place;
    wave_lds_fence();                          // the readers of the tile before the last are done
    if (lane < kTile) place[lane] = r < 0 ? ~(h * a.pool.head_rows) : r;   // missing: page 0's row, inverted
    wave_lds_fence();
    pages.fetch(a, b, tile + a.waves * kTile, t1, lane);
  }
  __device__ __forceinline__ bool whole() const { return all; }
  __device__ __forceinline__ bool exists(int at) const { return rows[at] >= 0; }
  template <int UNIT>
  __device__ __forceinline__ const uint8_t *at(const uint8_t *pool, const AttendArgs &, int u, int in, int bytes) const {
    const int64_t r = rows[16 * u + in];
    return pool + (r < 0 ? ~r : r) * UNIT + bytes;
  }
};

template <typename S>
__global__ __launch_bounds__(64 * attend_most_waves(S::D), attend_waves(S::D, S::BITS)) void attend_kernel(AttendArgs a) {
  constexpr int BITS = S::BITS, D = S::D, HB = S::HB, NG = S::NG, KS = S::KS, VPL = S::VPL, OT = S::OT;
  constexpr int ROW = S::ROW;
  constexpr bool CODES = BITS != 16;
  constexpr int KB = 8 * BITS / 8;             // bytes of 8 key values
  constexpr int VB = VPL * BITS / 8;           // bytes of a lane's values of one group
  // by wave: see attend_wave_lds
  extern __shared__ int64_t lds[];
  constexpr int kWaveLds = attend_wave_lds(D, BITS, NG, HB), kOut = D + 4;
  const int waves = blockDim.x >> 6;
  float *region = reinterpret_cast<float *>(lds);
  auto join_o = [&](int w, int hh) { return region + w * kWaveLds + hh * kOut; };
  auto join_m = [&](int w, int hh) -> float & { return region[w * kWaveLds + HB * kOut + hh]; };
  auto join_l = [&](int w, int hh) -> float & { return region[w * kWaveLds + HB * (kOut + 1) + hh]; };

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, kg = lane >> 4;
  const int streams = a.heads * a.head_blocks;
  const int j = blockIdx.x / streams, stream = blockIdx.x % streams;
  const int hb = stream % a.head_blocks, h = stream / a.head_blocks;
  const Chunks part = chunks_of<true>(a, j);
  if (part.b < 0) return;
  const int64_t b = part.b;
  const int t0 = (j - part.first) * part.size, t1 = min(part.len, t0 + part.size);
  int tile = t0 + wave * kTile;
  using Rows = TileRows<S::PAGED16>;
  typename Rows::Ahead pages;

  // The query heads of this block; with at most 8 of them, columns 8..15
  // repeat columns 0..7 (see the values' product below).
  const int first = hb * HB, here = min(HB, a.group - first);
  const int hl = HB == 8 ? (n & 7) : n;
  const bool head_live = hl < here;
  const int64_t hq = static_cast<int64_t>(h) * a.group + first + (head_live ? hl : 0);
  const uint16_t *qp = a.q + b * a.q_b + hq * a.q_h;
  u32x4 qf[KS];
  float q_sum[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) q_sum[g] = 0.0f;
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    qf[s] = u32x4{0u, 0u, 0u, 0u};
    if (head_live) qf[s] = *reinterpret_cast<const u32x4 *>(qp + 32 * s + 8 * kg);
  }
  if (tile < t1) pages.fetch(a, b, tile, t1, lane);   // behind the queries, which need not arrive yet
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    if constexpr (CODES) {
#pragma unroll
      for (int i = 0; i < 4; ++i) q_sum[s * 32 / S::GS] += bf16_lo(qf[s][i]) + bf16_hi(qf[s][i]);
    }
    if constexpr (BITS == 4) {                 // pairs of codes 16 bits apart: 0 4, 1 5, 2 6, 3 7
      const u32x4 r = qf[s];
      qf[s] = u32x4{low_halves(r[0], r[2]), high_halves(r[0], r[2]), low_halves(r[1], r[3]), high_halves(r[1], r[3])};
    }
  }
  auto add = [](float x, float y) { return x + y; };
  auto larger = [](float x, float y) { return fmaxf(x, y); };
  if constexpr (CODES) {
#pragma unroll
    for (int g = 0; g < NG; ++g) q_sum[g] = across_rows(q_sum[g], add);
  }

  f32x4 o[OT];
  // A probability enters the values' product as the sum of its two terms T, off
  // by 2^-16 of itself, and a code as what holds it.  That error must not grow
  // by how far the held codes are from zero, so with their middle and the value
  // v_mid there
  //   sum p v = sum T held + sum (p v_mid - T middle),
  // the second sum in fp32, in mid_sum.  Where columns 8..15 carry the second
  // terms, the columns n and n + 8 are added in the end: each takes half of p v_mid.
  constexpr float kHalf = HB == 8 ? 0.5f : 1.0f;
  float mid_sum[NG];
#pragma unroll
  for (int j = 0; j < OT; ++j) o[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int g = 0; g < NG; ++g) mid_sum[g] = 0.0f;
  float m = -INFINITY, l = 0.0f;
  const float lazy = 8.0f * (a.natural == 1.0f ? 0.69314718055994531f : 1.0f);   // a factor of 2^8
  const float *mask = a.mask ? a.mask + b * a.mask_b + hq * a.mask_h : nullptr;
  float *scores = a.scores ? a.scores + (b * a.heads * a.group + hq) * a.scores_ld : nullptr;
  int64_t *rows = reinterpret_cast<int64_t *>(region + wave * kWaveLds);
  f32x4 *affine = reinterpret_cast<f32x4 *>(rows + 2 * kTile);   // 4 arrays, by group, then token
  constexpr int kArr = kTile * NG / 4;
  uint8_t *stage = reinterpret_cast<uint8_t *>(affine + 4 * kArr);   // 32 rows of codes
  constexpr int kStageRow = ROW + 16;          // spreads the rows over the banks

  // What a tile needs, in the order it is needed, is loaded one tile ahead:
  // its keys (and scales) as soon as the last tile's have left their
  // registers, its values likewise.  The memory counter retires loads in
  // order, so each wait covers just what it has to.
  // Codes are loaded as they lie, 16 bytes a lane and whole rows a load, and
  // are rearranged through LDS.
  constexpr int kRowLanes = ROW / 16, kLoadRows = 64 / kRowLanes, kLoads = kTile / kLoadRows;   // codes
  Piece<KB> key[CODES ? 1 : 2][KS];
  Piece<VB> val[8][NG];
  u32x4 key_codes[CODES ? kLoads : 1], value_codes[CODES ? kLoads : 1];
  Piece<2 * NG> affine_k, affine_v;            // scales by lanes 0..31, biases by 32..63
  float open[8];                               // the mask
  auto load_codes = [&](const Rows &from, const uint8_t *pool, u32x4 *out) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int in = lane / kRowLanes, bytes = (lane % kRowLanes) * 16;
      const uint8_t *p;
      if constexpr (kLoadRows <= 16) {
        constexpr int per_half = 16 / kLoadRows;
        p = from.template at<ROW>(pool, a, i / per_half, (i % per_half) * kLoadRows + in, bytes);
      } else {
        const uint8_t *p0 = from.template at<ROW>(pool, a, 0, in & 15, bytes);
        const uint8_t *p1 = from.template at<ROW>(pool, a, 1, in & 15, bytes);
        p = in < 16 ? p0 : p1;
      }
      out[i] = *reinterpret_cast<const u32x4 *>(p);
    }
  };
  auto stage_codes = [&](const u32x4 *in) {
    wave_lds_fence();                          // what lay there has been read
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      *reinterpret_cast<u32x4 *>(stage + (i * kLoadRows + lane / kRowLanes) * kStageRow + (lane % kRowLanes) * 16) = in[i];
    wave_lds_fence();
  };
  auto load_keys = [&](const Rows &from) {
    if constexpr (!CODES) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint8_t *kp = from.template at<ROW>(a.pool.k, a, u, n, kg * KB);
#pragma unroll
        for (int st = 0; st < KS; ++st) key[u][st].load(kp + 32 * st * BITS / 8);
      }
    } else {
      load_codes(from, a.pool.k, key_codes);
      // lanes 0..31 take the scales of the tile's 32 rows, lanes 32..63 the biases
      const uint8_t *of[4] = {reinterpret_cast<const uint8_t *>(a.pool.ks), reinterpret_cast<const uint8_t *>(a.pool.kb),
                              reinterpret_cast<const uint8_t *>(a.pool.vs), reinterpret_cast<const uint8_t *>(a.pool.vb)};
      const uint8_t *at[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t *p0 = from.template at<2 * NG>(of[i], a, 0, n, 0);
        const uint8_t *p1 = from.template at<2 * NG>(of[i], a, 1, n, 0);
        at[i] = (lane & 16) ? p1 : p0;
      }
      affine_k.load(lane < 32 ? at[0] : at[1]);
      affine_v.load(lane < 32 ? at[2] : at[3]);
    }
  };
  auto load_mask = [&](int tile) {
    if (mask) {
      if (tile + kTile <= t1) {
        __builtin_memcpy(open, mask + tile + 4 * kg, 16);
        __builtin_memcpy(open + 4, mask + tile + 16 + 4 * kg, 16);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int t = tile + 16 * (e / 4) + 4 * kg + e % 4;
          open[e] = t < t1 ? mask[t] : -INFINITY;
        }
      }
    }
  };
  auto load_values = [&](const Rows &from) {
    if constexpr (CODES) {
      load_codes(from, a.pool.v, value_codes);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        val[e][0].load(from.template at<ROW>(a.pool.v, a, e / 4, 4 * kg + e % 4, VB * n));
    }
  };

  Rows where, ahead;
  int place = 0;
  if (tile < t1) {
    where.find(a, pages, rows, b, h, tile, t1, lane);
    load_keys(where);
    load_mask(tile);
    load_values(where);
  }
  // One tile.  The last one is a call of its own: loads under a condition
  // inside the loop would make every wait assume that they were not issued.
  auto step = [&](auto is_last) {
    constexpr bool kLast = decltype(is_last)::value;
    const int next = tile + waves * kTile;
    ahead = where;
    if constexpr (!kLast) {
      place ^= kTile;
      ahead.find(a, pages, rows + place, b, h, next, t1, lane);
    }
    const bool whole = where.whole();
    if constexpr (CODES) {
      // 4-bit codes enter the products as 128 + 8 q: scale / 8, and for the keys
      // bias - 16 scale; the values' bias is taken at the middle code
      float ak[NG], av[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        ak[g] = __uint_as_float(g % 2 == 0 ? affine_k.w[g / 2] << 16 : affine_k.w[g / 2] & 0xFFFF0000u);
        av[g] = __uint_as_float(g % 2 == 0 ? affine_v.w[g / 2] << 16 : affine_v.w[g / 2] & 0xFFFF0000u);
        const float sv = across_halves(av[g]); // lanes 32..63 get the scales
        if constexpr (BITS == 4) {
          const float sk = across_halves(ak[g]);
          ak[g] = lane < 32 ? ak[g] * 0.125f : fmaf(-16.0f, sk, ak[g]);
          av[g] = lane < 32 ? av[g] * 0.125f : kHalf * fmaf(7.5f, sv, av[g]);
        } else {
          av[g] = lane < 32 ? av[g] : kHalf * fmaf(127.5f, sv, av[g]);
        }
        float *ka = reinterpret_cast<float *>(affine + (lane < 32 ? 0 : 1) * kArr);
        float *va = reinterpret_cast<float *>(affine + (lane < 32 ? 2 : 3) * kArr);
        ka[32 * g + (lane & 31)] = ak[g];
        va[32 * g + (lane & 31)] = av[g];
      }
      stage_codes(key_codes);
      if constexpr (!kLast) load_keys(ahead);
    }

    // scores, keys x heads: this lane gets head n of the keys 16 u + 4 kg + r
    float s[8];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if constexpr (CODES) {
        __builtin_amdgcn_sched_barrier(0);     // one half's codes in registers at a time
#pragma unroll
        for (int st = 0; st < KS; ++st)
          key[0][st].load(stage + (16 * u + n) * kStageRow + (32 * st + 8 * kg) * BITS / 8);
      }
      f32x4 total = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int st = g * KS / NG; st < (g + 1) * KS / NG; ++st) {
          const Piece<KB> &piece = key[CODES ? 0 : u][st];
          u32x4 kf;
          if constexpr (BITS == 16) {
            kf = u32x4{piece.w[0], piece.w[1], piece.w[2], piece.w[3]};
          } else if constexpr (BITS == 8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t w = piece.w[i / 2];
              const float x = static_cast<float>((w >> (16 * (i & 1))) & 255u);
              const float y = static_cast<float>((w >> (16 * (i & 1) + 8)) & 255u);
              kf[i] = high_halves(__float_as_uint(x), __float_as_uint(y));
            }
          } else {
            const uint32_t w = piece.w[0];
            kf = u32x4{((w << 3) & 0x00780078u) | 0x43004300u, ((w >> 1) & 0x00780078u) | 0x43004300u,
                       ((w >> 5) & 0x00780078u) | 0x43004300u, ((w >> 9) & 0x00780078u) | 0x43004300u};
          }
          d = mfma(kf, qf[st], d);
        }
        if constexpr (!CODES) {
          total = d;
        } else {                               // of this lane's four keys
          const f32x4 ks = affine[0 * kArr + 8 * g + 4 * u + kg], kb = affine[1 * kArr + 8 * g + 4 * u + kg];
#pragma unroll
          for (int r = 0; r < 4; ++r) total[r] = fmaf(ks[r], d[r], fmaf(kb[r], q_sum[g], total[r]));
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) s[4 * u + r] = total[r] * a.scale;
    }

    // what most tiles do not need
    if (!whole || mask || scores) {
      bool dead[8];                            // takes no part, for any head of the block
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool missing = !whole && !where.exists(16 * (e / 4) + 4 * kg + e % 4);
        const bool shut = missing || (mask && open[e] == -INFINITY);
        s[e] = shut ? -INFINITY : (mask ? s[e] + open[e] : s[e]);
        dead[e] = missing || (mask && ((__ballot(!shut && head_live) >> (16 * kg)) & 0xFFFFu) == 0);
      }
      if (scores && head_live && (HB == 16 || n < 8)) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int t = tile + 16 * u + 4 * kg;
          if (t + 4 <= t1) {
            *reinterpret_cast<f32x4 *>(scores + t) = f32x4{s[4 * u], s[4 * u + 1], s[4 * u + 2], s[4 * u + 3]};
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (t + r < t1) scores[t + r] = s[4 * u + r];
          }
        }
      }
      // whatever a dead entry's memory holds: 0 * NaN would spread
      if (!whole || mask) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (dead[e]) {
            if constexpr (!CODES) {
              val[e][0].clear();
            } else {                           // codes are numbers, scales may be anything
#pragma unroll
              for (int g = 0; g < NG; ++g) {
                const int at = 32 * g + 16 * (e / 4) + 4 * kg + e % 4;
                reinterpret_cast<float *>(affine + 2 * kArr)[at] = 0.0f;
                reinterpret_cast<float *>(affine + 3 * kArr)[at] = 0.0f;
              }
            }
          }
        }
        if constexpr (CODES) wave_lds_fence();
      }
    }

    if constexpr (!kLast) {
      if constexpr (!CODES) load_keys(ahead);
      load_mask(next);
    }

    // Running maximum, moved only when a score passes it by a factor of 2^8:
    // the probabilities and their sum then stay within fp32's range and the
    // usual tile needs no exchange between lanes.
    float mx = s[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) mx = fmaxf(mx, s[e]);
    if (__ballot(mx > m + lazy) != 0) {
      const float m_new = fmaxf(m, across_rows(mx, larger));
      const float alpha = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m - m_new) * a.unit);
      m = m_new;
      l *= alpha;
#pragma unroll
      for (int j = 0; j < OT; ++j) o[j] *= alpha;
#pragma unroll
      for (int g = 0; g < NG; ++g) mid_sum[g] *= alpha;
    }
    const float base = m == -INFINITY ? 0.0f : m;
    float p[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      p[e] = __builtin_amdgcn_exp2f((s[e] - base) * a.unit);
      l += p[e];
    }

    // Values: out^T += V^T P^T, the probabilities as two bf16 terms (high and
    // low), which keeps 16 bits of them: outputs are off by 3e-6 to 4e-6 of their
    // size (root mean square, all row types), a few thousandths of a bf16 output's
    // rounding.  A third term would take a product more a tile.  With at most 8
    // heads the columns 8..15 carry the low terms, so one product does both.
    if constexpr (CODES) {
      stage_codes(value_codes);
      if constexpr (!kLast) load_values(ahead);
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      if constexpr (CODES) {
        __builtin_amdgcn_sched_barrier(0);     // one group's codes in registers at a time
#pragma unroll
        for (int e = 0; e < 8; ++e)
          val[e][g].load(stage + (16 * (e / 4) + 4 * kg + e % 4) * kStageRow + (g * S::GS + VPL * n) * BITS / 8);
      }
      u32x4 ph, pl;
      float pg[8], hi[8], lo[8];
      f32x4 vs[2], vb[2];
      if constexpr (CODES) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          vs[u] = affine[2 * kArr + 8 * g + 4 * u + kg];
          vb[u] = affine[3 * kArr + 8 * g + 4 * u + kg];
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (CODES) {
          pg[e] = p[e] * vs[e / 4][e % 4];
          mid_sum[g] = fmaf(p[e], vb[e / 4][e % 4], mid_sum[g]);
        } else {
          pg[e] = p[e];
        }
        hi[e] = __uint_as_float(__float_as_uint(pg[e]) & 0xFFFF0000u);
        lo[e] = pg[e] - hi[e];
        if (HB == 8 && n >= 8) hi[e] = lo[e];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ph[i] = pack_bf16(hi[2 * i], hi[2 * i + 1]);
        if constexpr (HB == 16) pl[i] = pack_bf16(lo[2 * i], lo[2 * i + 1]);
        if constexpr (CODES) {
          mid_sum[g] = take_mid<BITS>(ph[i], mid_sum[g]);
          if constexpr (HB == 16) mid_sum[g] = take_mid<BITS>(pl[i], mid_sum[g]);
        }
      }
      qmvk::static_for<0, VPL>([&](auto J) {
        constexpr int j = decltype(J)::value;
        u32x4 vf;
#pragma unroll
        for (int i = 0; i < 4; ++i) vf[i] = value_pair<BITS, j>(val[2 * i][g], val[2 * i + 1][g]);
        o[g * VPL + j] = mfma(vf, ph, o[g * VPL + j]);
        if constexpr (HB == 16) o[g * VPL + j] = mfma(vf, pl, o[g * VPL + j]);
      });
    }
    if constexpr (CODES) wave_lds_fence();     // the next tile's scales replace these
    else if constexpr (!kLast) load_values(ahead);
    tile = next;
    where = ahead;
  };
  while (tile + waves * kTile < t1) step(std::false_type{});
  if (tile < t1) step(std::true_type{});

  // join the waves
  wave_lds_fence();                            // a wave's results replace its tiles
  l = across_rows(l, add);
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    mid_sum[g] = across_rows(mid_sum[g], add);
    if constexpr (HB == 8) mid_sum[g] += __builtin_bit_cast(float, dpp<0x128>(__builtin_bit_cast(uint32_t, mid_sum[g])));   // lane ^ 8
  }
  if (kg == 0 && n < HB) {
    join_m(wave, n) = m;
    join_l(wave, n) = l;
  }
  qmvk::static_for<0, OT>([&](auto J) {
    constexpr int j = decltype(J)::value;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float x = o[j][r];
      if constexpr (HB == 8) x += __builtin_bit_cast(float, dpp<0x128>(__builtin_bit_cast(uint32_t, x)));   // lane ^ 8
      if constexpr (CODES) x += mid_sum[j / VPL];
      if (n < HB) join_o(wave, n)[(j / VPL) * S::GS + VPL * (4 * kg + r) + j % VPL] = x;
    }
  });
  __syncthreads();
  const int64_t hq0 = b * a.heads * a.group + static_cast<int64_t>(h) * a.group + first;
  for (int i = tid; i < here * D; i += blockDim.x) {
    const int hh = i / D, d = i % D;
    float top = join_m(0, hh);
    for (int w = 1; w < waves; ++w) top = fmaxf(top, join_m(w, hh));
    const float base = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f, x = 0.0f;
    for (int w = 0; w < waves; ++w) {
      const float f = __builtin_amdgcn_exp2f((join_m(w, hh) - base) * a.unit);
      sum = fmaf(join_l(w, hh), f, sum);
      x = fmaf(join_o(w, hh)[d], f, x);
    }
    if (a.part) {
      const int64_t at = static_cast<int64_t>(j) * a.heads * a.group + h * a.group + first + hh;
      a.part[at * D + d] = x;
      if (d == 0) {
        a.part_ml[at * 2] = top;
        a.part_ml[at * 2 + 1] = sum;
      }
    } else {
      const int64_t head = hq0 + hh;
      const float y = sum == 0.0f ? 0.0f : x / sum;
      if (a.f32) static_cast<float *>(a.y)[head * D + d] = y;
      else static_cast<uint16_t *>(a.y)[head * D + d] = qmvk::f32_to_bf16(y);
      if (d == 0 && a.lse) a.lse[head] = top * a.natural + logf(sum);
    }
  }
}

// What is left once every chunk is done, in one launch: the join of the chunks
// (one workgroup per sequence and query head), and the attention that each
// slot got (`weight_parts` workgroups per sequence and key-value head), from
// the scores that the first kernel left behind: 4 bytes written and read per
// slot and query head, against 512 of rows per slot and key-value head (bf16,
// D = 128).  Launch and latency bound: 4 to 6 us at all sizes measured (a join
// and a weights kernel apart, the join serial over the chunks: 9 to 13).
constexpr int kFinishThreads = 256;
constexpr int kFinishWaves = kFinishThreads / 64;

// Maximum and sum over a head's chunks, by one wave; every lane has them.
__device__ __forceinline__ void join_chunks(const float *ml, int64_t stride, int used, float unit, int lane, float &base,
                                            float &top, float &sum) {
  float m = -INFINITY, l = 0.0f;
  for (int i = lane; i < used; i += 64) {
    const float mi = ml[i * stride], li = ml[i * stride + 1], hi = fmaxf(m, mi), z = hi == -INFINITY ? 0.0f : hi;
    l = fmaf(l, __builtin_amdgcn_exp2f((m - z) * unit), li * __builtin_amdgcn_exp2f((mi - z) * unit));
    m = hi;
  }
  top = wave_max(m);
  base = top == -INFINITY ? 0.0f : top;
  sum = wave_sum(l * __builtin_amdgcn_exp2f((m - base) * unit));
}

template <int D>
__device__ __forceinline__ void finish_head(const AttendArgs &a, int64_t head) {
  constexpr int kLanes = D / 4, kGroups = kFinishThreads / kLanes;
  __shared__ f32x4 parts[kGroups][kLanes];
  const int Hq = a.heads * a.group;
  const int b = static_cast<int>(head / Hq), hq = static_cast<int>(head - static_cast<int64_t>(b) * Hq);
  const int tid = threadIdx.x, lane = tid & 63;
  const Chunks part = chunks_of<false>(a, b);
  const int64_t at0 = static_cast<int64_t>(part.first) * Hq + hq;
  const float *ml = a.part_ml + at0 * 2;
  const f32x4 *values = reinterpret_cast<const f32x4 *>(a.part + at0 * D);
  const int d4 = tid % kLanes, g = tid / kLanes;
  float base, top, sum;
  join_chunks(ml, 2 * Hq, part.count, a.unit, lane, base, top, sum);
  f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int i = g; i < part.count; i += kGroups)
    x += values[static_cast<int64_t>(i) * Hq * kLanes + d4] *
         __builtin_amdgcn_exp2f((ml[static_cast<int64_t>(i) * 2 * Hq] - base) * a.unit);
  parts[g][d4] = x;
  __syncthreads();
  if (g == 0) {
#pragma unroll
    for (int j = 1; j < kGroups; ++j) x += parts[j][d4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float y = sum == 0.0f ? 0.0f : x[e] / sum;
      if (a.f32) static_cast<float *>(a.y)[head * D + 4 * d4 + e] = y;
      else static_cast<uint16_t *>(a.y)[head * D + 4 * d4 + e] = qmvk::f32_to_bf16(y);
    }
  }
  if (tid == 0 && a.lse) a.lse[head] = top * a.natural + logf(sum);
}

// weights_out[t] = weights_in[t] + sum over the group's query heads of p_t / sum p
__device__ __forceinline__ void finish_weights(const AttendArgs &a, const WeightArgs &w, int64_t bh, int part,
                                               float *norm) {
  const int64_t b = bh / a.heads;
  const int h = static_cast<int>(bh % a.heads);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const Chunks chunks = chunks_of<false>(a, static_cast<int>(b));
  const int len = chunks.len, Hq = a.heads * a.group;
  const float *ml = a.part_ml + (static_cast<int64_t>(chunks.first) * Hq + h * a.group) * 2;
  for (int g = wave; g < a.group; g += kFinishWaves) {
    float base, top, sum;
    join_chunks(ml + 2 * g, 2 * Hq, chunks.count, a.unit, lane, base, top, sum);
    if (lane == 0) {
      norm[2 * g] = base;
      norm[2 * g + 1] = sum == 0.0f ? 0.0f : 1.0f / sum;
    }
  }
  __syncthreads();
  const float *in = w.in + b * w.out_b + h * w.out_h;
  float *out = w.out + b * w.out_b + h * w.out_h;
  for (int t = part * kWeightSlots + tid; t < min(w.S, (part + 1) * kWeightSlots); t += kFinishThreads) {
    float x = in[t];
    if (t < len) {
      const float *s = a.scores + bh * a.group * a.scores_ld + t;
#pragma unroll 4
      for (int g = 0; g < a.group; ++g)
        x = fmaf(__builtin_amdgcn_exp2f((s[g * a.scores_ld] - norm[2 * g]) * a.unit), norm[2 * g + 1], x);
    }
    out[t] = x;
  }
}

template <int D>
static __global__ __launch_bounds__(kFinishThreads) void attend_finish_kernel(AttendArgs a, WeightArgs w,
                                                                              unsigned join_blocks, int weight_parts) {
  extern __shared__ float norm[];              // [group][2]
  if (blockIdx.x < join_blocks) {
    finish_head<D>(a, blockIdx.x);
  } else {
    const unsigned i = blockIdx.x - join_blocks;
    finish_weights(a, w, i / weight_parts, i % weight_parts, norm);
  }
}

}  // namespace qmvd
