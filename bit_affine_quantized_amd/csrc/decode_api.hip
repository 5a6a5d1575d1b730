// C ABI of the decode operators around a paged key-value cache (declared in
// include/qmv.h): validation before any HIP call, sizing, launch.
#include <utility>

#include "host_error.h"
#include "beam_kernels.h"
#include "kv_attend_launch.h"
#include "kv_move_kernels.h"

namespace qmvd {
namespace {

constexpr int64_t kMaxSlots = 0x7FFFFFFF - 65536;   // slot numbers are 32-bit

int64_t round_up(int64_t v, int64_t unit) { return (v + unit - 1) / unit * unit; }

bool misaligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

int check_cache(const char *fn, const qmv_kv_cache *c) {
  if (!c) return fail(QMV_EINVAL, "%s: null cache", fn);
  if (!c->k || !c->v) return fail(QMV_EINVAL, "%s: null k or v in the cache", fn);
  if (misaligned(c->k, 16) || misaligned(c->v, 16))
    return fail(QMV_EINVAL, "%s: the cache's k and v must be 16-byte aligned", fn);
  if (c->bits != 16 && c->bits != 8 && c->bits != 4)
    return fail(QMV_EINVAL, "%s: cache bits=%d not in {16,8,4}", fn, c->bits);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(QMV_EUNSUPPORTED, "%s: head_dim=%d not in {64,128,256}", fn, c->head_dim);
  if (c->bits != 16) {
    if (c->group_size != 32 && c->group_size != 64 && c->group_size != 128)
      return fail(QMV_EINVAL, "%s: group_size=%d not in {32,64,128}", fn, c->group_size);
    if (c->head_dim % c->group_size != 0)
      return fail(QMV_EINVAL, "%s: head_dim=%d is not a multiple of group_size=%d", fn, c->head_dim, c->group_size);
    if (!c->k_scales || !c->k_biases || !c->v_scales || !c->v_biases)
      return fail(QMV_EINVAL, "%s: null scales or biases in the cache", fn);
    const uintptr_t row = 2 * (c->head_dim / c->group_size);   // a row's are loaded at once
    if (misaligned(c->k_scales, row) || misaligned(c->k_biases, row) || misaligned(c->v_scales, row) ||
        misaligned(c->v_biases, row))
      return fail(QMV_EINVAL, "%s: the cache's scales and biases must be aligned to a row's %d bytes", fn, static_cast<int>(row));
  }
  if (c->pages < 1 || c->pages > 0x7FFFFFFF || c->heads < 1 || c->page_size < 1)
    return fail(QMV_EINVAL, "%s: pages=%lld, heads=%d and page_size=%d must be positive", fn, (long long)c->pages,
                c->heads, c->page_size);
  if (c->page_size > (1 << 20)) return fail(QMV_EINVAL, "%s: page_size=%d too large", fn, c->page_size);
  const int64_t far = int64_t(1) << 40;
  if (c->page_rows < 1 || c->head_rows < 1 || c->slot_rows < 1 || c->page_rows > far || c->head_rows > far ||
      c->slot_rows > far)
    return fail(QMV_EINVAL, "%s: cache strides must be positive", fn);
  return QMV_OK;
}

Pools pools_of(const qmv_kv_cache &c) {
  return Pools{static_cast<const uint8_t *>(c.k), static_cast<const uint8_t *>(c.v),
               c.bits == 16 ? nullptr : c.k_scales, c.bits == 16 ? nullptr : c.k_biases,
               c.bits == 16 ? nullptr : c.v_scales, c.bits == 16 ? nullptr : c.v_biases,
               c.page_rows, c.head_rows, c.slot_rows, static_cast<int>(c.pages), c.page_size};
}

int row_bytes(const qmv_kv_cache &c) { return c.bits == 16 ? 2 * c.head_dim : c.head_dim * c.bits / 8; }
int groups(const qmv_kv_cache &c) { return c.bits == 16 ? 0 : c.head_dim / c.group_size; }

int check_tables(const char *fn, const qmv_kv_cache *c, const int32_t *tables, int64_t B, int64_t cols, int64_t ld) {
  if (!tables) return fail(QMV_EINVAL, "%s: null block_tables", fn);
  if (B < 1 || cols < 1) return fail(QMV_EINVAL, "%s: B=%lld and cols=%lld must be positive", fn, (long long)B, (long long)cols);
  if (B > (1 << 24)) return fail(QMV_EINVAL, "%s: B=%lld too large", fn, (long long)B);
  if (ld < cols) return fail(QMV_EINVAL, "%s: table stride %lld below cols=%lld", fn, (long long)ld, (long long)cols);
  if (cols > kMaxSlots / c->page_size) return fail(QMV_EINVAL, "%s: cols * page_size too large", fn);
  return QMV_OK;
}

Tables tables_of(const qmv_kv_cache &c, const int32_t *tables, int64_t B, int64_t cols, int64_t ld) {
  return Tables{B, tables, ld, static_cast<int>(cols), divider(static_cast<uint32_t>(c.page_size))};
}

// ------------------------------------------------------------------ attend
struct AttendPlan {
  int max_len, hb, head_blocks, waves, whole, share, most_chunk;
  int64_t chunks;                              // at most, of all sequences
  int64_t scores_ld;
  size_t part, ml, scores, bytes;              // byte offsets in the workspace, and its size
};

// Whole: a sequence's head is one workgroup of eight waves (four at D = 256)
// and, without weights to add, the only launch: up to 640 slots, or up to 1024
// if that makes 128 workgroups or more.  (bf16, 8 heads of 128, graph replays
// on MI355X, chunks -> whole: one sequence of 128 / 512 / 640 / 1024 slots 10.1
// -> 6.3, 10.1 -> 9.8, 10.2 -> 10.6, 10.3 -> 13.8 us, and 3 us less of launching
// from the host, so from 513 to 640 slots of few heads the one launch gains for a
// caller that launches and loses 0.4 us in a graph; 16 sequences of 512 / 1024 /
// 2048: 12.3 -> 10.9, 20.1 -> 16.2, 28.2 -> 25.9 us, but long batches of ragged
// lengths need the sharing out that chunks give.)  Others are cut into chunks for workgroups of
// four waves, about as many as the machine holds at once if that makes chunks
// of kMostChunk slots at most, else so many of that size (1024 to 4096 measure
// within 2% of each other).  The lengths are on the device, and so is the
// cutting (struct Chunks); the launch has room for whatever lengths the tables
// allow, but no more than kRounds machines full of chunks beside one a
// sequence.
AttendPlan attend_plan(const qmv_kv_cache &c, int64_t B, int64_t cols, int group, bool weights, int64_t max_length) {
  constexpr int64_t kWholeFew = 640, kWholeMany = 1024, kMany = 128, kMostChunk = 2048, kRounds = 8, kCus = 256;
  AttendPlan p{};
  const int64_t cap = cols * c.page_size;
  p.max_len = static_cast<int>(max_length > 0 && max_length < cap ? max_length : cap);
  p.hb = group <= 8 ? 8 : 16;
  p.head_blocks = (group + p.hb - 1) / p.hb;
  const int64_t unit = kChunkUnit, streams = static_cast<int64_t>(c.heads) * p.head_blocks;
  p.whole = p.max_len <= (B * streams >= kMany ? kWholeMany : kWholeFew);
  p.waves = p.whole ? attend_most_waves(c.head_dim) : kChunkWaves;
  int64_t share = kCus * attend_waves(c.head_dim, c.bits) / streams;
  if (share < 1) share = 1;
  int64_t most = round_up((B * p.max_len + kRounds * share - 1) / (kRounds * share), unit);
  if (most < kMostChunk) most = kMostChunk;
  if (most > round_up(p.max_len, unit)) most = round_up(p.max_len, unit);
  p.most_chunk = static_cast<int>(most);
  const int64_t full = (B * p.max_len + most - 1) / most;
  p.chunks = p.whole ? B : (full > share ? full : share) + B;
  // every sequence's last chunk is on average half empty
  p.share = static_cast<int>(share - B / 2 > (share + 1) / 2 ? share - B / 2 : (share + 1) / 2);
  const int64_t hq = static_cast<int64_t>(c.heads) * group;
  const bool finish = !p.whole || weights;
  size_t at = 0;
  p.part = at;
  if (finish) at += static_cast<size_t>(p.chunks) * hq * c.head_dim * 4;
  p.ml = at;
  if (finish) at += round_up(p.chunks * hq * 8, 16);
  p.scores = at;
  p.scores_ld = round_up(p.max_len, 4);
  if (weights) at += static_cast<size_t>(B) * hq * p.scores_ld * 4;
  p.bytes = at;
  return p;
}

int check_attend(const char *fn, const qmv_kv_cache *c, int64_t B, int64_t cols, int group, int64_t max_length) {
  if (int rc = check_cache(fn, c)) return rc;
  if (B < 1 || B > (1 << 24)) return fail(QMV_EINVAL, "%s: B=%lld out of range", fn, (long long)B);
  if (cols < 1 || cols > kMaxSlots / c->page_size) return fail(QMV_EINVAL, "%s: cols=%lld out of range", fn, (long long)cols);
  const int64_t cap = cols * c->page_size, longest = max_length > 0 && max_length < cap ? max_length : cap;
  if (B * longest > int64_t(1) << 35)
    return fail(QMV_EUNSUPPORTED, "%s: %lld sequences of up to %lld slots are too many", fn, (long long)B, (long long)longest);
  if (group < 1 || group > 1024) return fail(QMV_EINVAL, "%s: group=%d not in [1,1024]", fn, group);
  if (max_length < 0) return fail(QMV_EINVAL, "%s: max_length=%lld is negative", fn, (long long)max_length);
  return QMV_OK;
}

// Whether slots of a [B, heads, S] array with these strides share memory.
bool overlapping(int64_t B, int64_t heads, int64_t S, int64_t stride_b, int64_t stride_h) {
  struct Axis {
    int64_t size, stride;
  } axes[2] = {{B, stride_b < 0 ? -stride_b : stride_b}, {heads, stride_h < 0 ? -stride_h : stride_h}};
  if (axes[0].stride < axes[1].stride) std::swap(axes[0], axes[1]);
  int64_t run = S;                             // what the inner axes span
  for (int i = 1; i >= 0; --i) {
    if (axes[i].size == 1) continue;
    if (axes[i].stride < run) return true;
    run = axes[i].stride > INT64_MAX / axes[i].size ? INT64_MAX : (axes[i].size - 1) * axes[i].stride + run;
  }
  return false;
}

int attend(const uint16_t *q, int64_t q_b, int64_t q_h, const qmv_kv_cache *c, const int32_t *tables, int64_t ld,
           int64_t cols, const int32_t *lengths, int64_t B, int group, float scale, const float *mask, int64_t mask_b,
           int64_t mask_h, int64_t mask_cols, const float *weights_in, float *weights_out, int64_t w_b, int64_t w_h,
           int64_t S, void *y, float *lse, int64_t max_length, int out_dtype, void *workspace, size_t workspace_bytes,
           hipStream_t st) {
  const char *fn = "qmv_kv_attend";
  if (int rc = check_attend(fn, c, B, cols, group, max_length)) return rc;
  if (int rc = check_tables(fn, c, tables, B, cols, ld)) return rc;
  if (!q || !lengths || !y) return fail(QMV_EINVAL, "%s: null q, lengths or y", fn);
  if (misaligned(q, 16) || q_b % 8 != 0 || q_h % 8 != 0)
    return fail(QMV_EINVAL, "%s: q must be 16-byte aligned in every row", fn);
  if (out_dtype != QMV_OUT_BF16 && out_dtype != QMV_OUT_F32) return fail(QMV_EINVAL, "%s: out_dtype=%d", fn, out_dtype);
  if ((weights_in == nullptr) != (weights_out == nullptr))
    return fail(QMV_EINVAL, "%s: weights_in and weights_out go together", fn);
  const bool weights = weights_out != nullptr;
  if (weights && (S < 1 || S > kMaxSlots)) return fail(QMV_EINVAL, "%s: S=%lld out of range", fn, (long long)S);
  const AttendPlan p = attend_plan(*c, B, cols, group, weights, max_length);
  if (mask && mask_cols < p.max_len)
    return fail(QMV_EINVAL, "%s: mask has %lld columns, %d are needed", fn, (long long)mask_cols, p.max_len);
  if (p.bytes && (!workspace || workspace_bytes < p.bytes))
    return fail(QMV_EINVAL, "%s: workspace of %zu bytes, %zu are needed", fn, workspace ? workspace_bytes : size_t(0), p.bytes);
  if (misaligned(workspace, 16)) return fail(QMV_EINVAL, "%s: workspace must be 16-byte aligned", fn);
  // heads add to their own slots in no order of theirs
  if (weights && overlapping(B, c->heads, S, w_b, w_h))
    return fail(QMV_EINVAL, "%s: the slots of weights overlap (strides %lld, %lld)", fn, (long long)w_b, (long long)w_h);

  constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.69314718055994531f;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  AttendArgs a{};
  a.q = q;
  a.q_b = q_b;
  a.q_h = q_h;
  a.pool = pools_of(*c);
  a.tab = tables_of(*c, tables, B, cols, ld);
  a.lengths = lengths;
  a.mask = mask;
  a.mask_b = mask_b;
  a.mask_h = mask_h;
  a.y = y;
  a.lse = lse;
  const bool finish = !p.whole || weights;
  a.part = finish ? reinterpret_cast<float *>(ws + p.part) : nullptr;
  a.part_ml = reinterpret_cast<float *>(ws + p.ml);
  a.scores = weights ? reinterpret_cast<float *>(ws + p.scores) : nullptr;
  a.scores_ld = p.scores_ld;
  a.heads = c->heads;
  a.group = group;
  a.head_blocks = p.head_blocks;
  a.whole = p.whole;
  a.share = p.share;
  a.most_chunk = p.most_chunk;
  a.max_len = p.max_len;
  a.waves = p.waves;
  // Without a mask the scores are kept in powers of 2.  With one they stay in
  // powers of e: a mask of the type's lowest value times log2 e would overflow.
  a.scale = mask ? scale : scale * kLog2e;
  a.unit = mask ? kLog2e : 1.0f;
  a.natural = mask ? 1.0f : kLn2;
  a.f32 = out_dtype == QMV_OUT_F32;
  int rc = c->bits == 16 ? attend_b16(a, p.chunks, c->head_dim, 0, p.hb, st)
         : c->bits == 8  ? attend_b8(a, p.chunks, c->head_dim, c->group_size, p.hb, st)
                         : attend_b4(a, p.chunks, c->head_dim, c->group_size, p.hb, st);
  if (rc || !finish) return rc;
  WeightArgs w{};
  w.in = weights_in;
  w.out = weights_out;
  w.out_b = w_b;
  w.out_h = w_h;
  w.S = static_cast<int>(S);
  const int64_t join = B * c->heads * group, parts = weights ? (S + kWeightSlots - 1) / kWeightSlots : 0;
  if (join + parts * B * c->heads > 0x7FFFFFFF) return fail(QMV_EUNSUPPORTED, "%s: too many heads", fn);
  auto kern = c->head_dim == 64 ? attend_finish_kernel<64> : c->head_dim == 128 ? attend_finish_kernel<128> : attend_finish_kernel<256>;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(join + parts * B * c->heads)), dim3(kFinishThreads),
                     static_cast<size_t>(weights ? group * 8 : 0), st, a, w, static_cast<unsigned>(join),
                     static_cast<int>(parts));
  return check_launch(fn);
}

// ------------------------------------------------------------------ evict
struct EvictPlan {
  int most, mask_words;
  size_t stay, counts, bytes;
};

EvictPlan evict_plan(int64_t B, int heads, int64_t S, int64_t budget) {
  EvictPlan p{};
  const int64_t over = S > budget ? S - budget : 0;
  p.most = static_cast<int>(budget < over ? budget : over);
  p.mask_words = static_cast<int>(((p.most ? budget : 0) + kEvictStep - 1) / kEvictStep * 4);   // no eviction, no mask
  p.stay = round_up(B * heads * 2 * p.most * 4, 16);
  p.counts = p.stay + static_cast<size_t>(B) * heads * p.mask_words * 8;
  p.bytes = p.counts + static_cast<size_t>(round_up(B * heads * 4, 16));
  return p;
}

int check_evict(const char *fn, int64_t B, int heads, int64_t S, int64_t budget) {
  if (B < 1 || B > (1 << 24) || heads < 1) return fail(QMV_EINVAL, "%s: B=%lld or heads=%d out of range", fn, (long long)B, heads);
  if (S < 1 || S > kMaxSlots) return fail(QMV_EINVAL, "%s: S=%lld out of range", fn, (long long)S);
  if (budget < 1 || budget > kMaxSlots) return fail(QMV_EINVAL, "%s: budget=%lld must be positive", fn, (long long)budget);
  if (B * heads > 0x7FFFFFFF || B * heads > (int64_t(1) << 40) / S)
    return fail(QMV_EUNSUPPORTED, "%s: %lld sequences of %d heads with S=%lld are too many", fn, (long long)B, heads, (long long)S);
  return QMV_OK;
}

// ------------------------------------------------------------------ beam
struct BeamPlan {
  int per, chunks;
  size_t m, l, left, list, bytes;
};

// Logits a thread of the scan: 64 where that leaves 768 workgroups or more (16 x 8
// beams over 131072: the scan 17.8 us with 32, 15.8 with 64), 32 where that
// leaves 1024, else 16.
BeamPlan beam_plan(int64_t rows, int64_t V, int num) {
  BeamPlan p{};
  p.per = rows * V >= int64_t(768) * kScanThreads * 64 ? 64 : (rows * V >= int64_t(1024) * kScanThreads * 32 ? 32 : 16);
  p.chunks = static_cast<int>((V + kScanThreads * p.per - 1) / (kScanThreads * p.per));
  const size_t each = static_cast<size_t>(rows) * p.chunks;
  const size_t one = round_up(each * 4, 16);
  p.l = one;
  p.left = 2 * one;
  p.list = 3 * one;
  p.bytes = p.list + round_up(each * num * 8, 16);
  return p;
}

int check_beam(const char *fn, int64_t B, int64_t W, int64_t V, int num) {
  if (B < 1 || W < 1 || V < 1)
    return fail(QMV_EINVAL, "%s: B=%lld, W=%lld and V=%lld must be positive", fn, (long long)B, (long long)W, (long long)V);
  if (W > 4096 || V > 0x7FFFFFFF || W * V >= 0xFFFFFFFFLL)
    return fail(QMV_EINVAL, "%s: W=%lld beams of V=%lld tokens are too many", fn, (long long)W, (long long)V);
  if (num < 1 || num > kBeamMost || num > W * V)
    return fail(QMV_EINVAL, "%s: num=%d not in [1,%d] or more than the candidates", fn, num, kBeamMost);
  const BeamPlan p = beam_plan(B * W, V, num);
  if (B * W * p.chunks > 0x7FFFFFFF - kJoinThreads || W * p.chunks * num > 0x7FFFFFFF - kJoinThreads)
    return fail(QMV_EUNSUPPORTED, "%s: too many rows", fn);
  return QMV_OK;
}

}  // namespace
}  // namespace qmvd

using namespace qmvd;

extern "C" {

int qmv_kv_append(const uint16_t *k, int64_t k_t, int64_t k_h, const uint16_t *v, int64_t v_t, int64_t v_h,
                  const qmv_kv_cache *cache, const int32_t *block_tables, int64_t table_ld, int64_t cols, int64_t B,
                  const int32_t *rows, const int32_t *slots, int64_t T, float *weights, int32_t *positions,
                  const int32_t *token_positions, int64_t meta_b, int64_t meta_h, int64_t S, void *stream) {
  const char *fn = "qmv_kv_append";
  if (int rc = check_cache(fn, cache)) return rc;
  if (int rc = check_tables(fn, cache, block_tables, B, cols, table_ld)) return rc;
  if (T < 0) return fail(QMV_EINVAL, "%s: T=%lld is negative", fn, (long long)T);
  if (T == 0) return ok();
  if (!k || !v || !slots) return fail(QMV_EINVAL, "%s: null k, v or slots", fn);
  if (misaligned(k, 16) || misaligned(v, 16) || k_t % 8 || k_h % 8 || v_t % 8 || v_h % 8)
    return fail(QMV_EINVAL, "%s: k and v must be 16-byte aligned in every row", fn);
  if ((weights || positions) && S < 1) return fail(QMV_EINVAL, "%s: S=%lld must be positive", fn, (long long)S);
  AppendArgs a{};
  a.k = k;
  a.v = v;
  a.k_t = k_t;
  a.k_h = k_h;
  a.v_t = v_t;
  a.v_h = v_h;
  a.pool = pools_of(*cache);
  a.tab = tables_of(*cache, block_tables, B, cols, table_ld);
  a.rows = rows;
  a.slots = slots;
  a.token_positions = token_positions;
  a.weights = weights;
  a.positions = positions;
  a.meta_b = meta_b;
  a.meta_h = meta_h;
  a.B = B;
  a.S = S;
  if (T * cache->heads > 0x3FFFFFFF) return fail(QMV_EUNSUPPORTED, "%s: too many tokens", fn);
  a.per_token = divider(static_cast<uint32_t>(cache->heads));
  a.T = static_cast<int>(T);
  a.heads = cache->heads;
  a.D = cache->head_dim;
  a.piece_bits = cache->head_dim == 64 ? 3 : cache->head_dim == 128 ? 4 : 5;
  const bool codes = cache->bits != 16;
  a.line_bits = codes && T >= 64 ? 4 : 0;
  const int64_t threads = round_up(T, int64_t(1) << a.line_bits) * cache->heads * (cache->head_dim / 8);
  const int64_t blocks = (threads + kAppendThreads - 1) / kAppendThreads;
  if (blocks > 0x7FFFFFFF) return fail(QMV_EUNSUPPORTED, "%s: too many tokens", fn);
  const dim3 grid(static_cast<unsigned>(blocks)), block(kAppendThreads);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (!codes) hipLaunchKernelGGL(append_bf16_kernel, grid, block, 0, st, a);
  else if (cache->bits == 8 && cache->group_size == 32) hipLaunchKernelGGL((append_codes_kernel<8, 32>), grid, block, 0, st, a);
  else if (cache->bits == 8 && cache->group_size == 64) hipLaunchKernelGGL((append_codes_kernel<8, 64>), grid, block, 0, st, a);
  else if (cache->bits == 8) hipLaunchKernelGGL((append_codes_kernel<8, 128>), grid, block, 0, st, a);
  else if (cache->group_size == 32) hipLaunchKernelGGL((append_codes_kernel<4, 32>), grid, block, 0, st, a);
  else if (cache->group_size == 64) hipLaunchKernelGGL((append_codes_kernel<4, 64>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((append_codes_kernel<4, 128>), grid, block, 0, st, a);
  return check_launch(fn);
}

int qmv_kv_attend_workspace_bytes(const qmv_kv_cache *cache, int64_t B, int64_t cols, int group, int weights,
                                  int64_t max_length, size_t *bytes) {
  const char *fn = "qmv_kv_attend_workspace_bytes";
  if (!bytes) return fail(QMV_EINVAL, "%s: null bytes", fn);
  if (int rc = check_attend(fn, cache, B, cols, group, max_length)) return rc;
  *bytes = attend_plan(*cache, B, cols, group, weights != 0, max_length).bytes;
  return ok();
}

int qmv_kv_attend(const uint16_t *q, int64_t q_b, int64_t q_h, const qmv_kv_cache *cache, const int32_t *block_tables,
                  int64_t table_ld, int64_t cols, const int32_t *lengths, int64_t B, int group, float scale,
                  const float *mask, int64_t mask_b, int64_t mask_h, int64_t mask_cols, const float *weights_in,
                  float *weights_out, int64_t w_b, int64_t w_h, int64_t S, void *y, float *lse, int64_t max_length,
                  int out_dtype, void *workspace, size_t workspace_bytes, void *stream) {
  return attend(q, q_b, q_h, cache, block_tables, table_ld, cols, lengths, B, group, scale, mask, mask_b, mask_h,
                mask_cols, weights_in, weights_out, w_b, w_h, S, y, lse, max_length, out_dtype, workspace,
                workspace_bytes, static_cast<hipStream_t>(stream));
}

int qmv_kv_evict_workspace_bytes(int64_t B, int heads, int64_t S, int64_t budget, size_t *bytes) {
  const char *fn = "qmv_kv_evict_workspace_bytes";
  if (!bytes) return fail(QMV_EINVAL, "%s: null bytes", fn);
  if (int rc = check_evict(fn, B, heads, S, budget)) return rc;
  *bytes = evict_plan(B, heads, S, budget).bytes;
  return ok();
}

int qmv_kv_evict(const qmv_kv_cache *cache, const int32_t *block_tables, int64_t table_ld, int64_t cols,
                 const int32_t *lengths, int64_t B, const float *weights, const int32_t *positions, int64_t meta_b,
                 int64_t meta_h, int64_t S, const int32_t *next_positions, int64_t budget, int64_t recent,
                 int32_t *lengths_out, float *weights_out, int32_t *positions_out, void *workspace,
                 size_t workspace_bytes, void *stream) {
  const char *fn = "qmv_kv_evict";
  if (int rc = check_cache(fn, cache)) return rc;
  if (int rc = check_tables(fn, cache, block_tables, B, cols, table_ld)) return rc;
  if (int rc = check_evict(fn, B, cache->heads, S, budget)) return rc;
  if (recent < 0 || recent > budget)
    return fail(QMV_EINVAL, "%s: recent=%lld not in [0,budget=%lld]", fn, (long long)recent, (long long)budget);
  if (!lengths || !weights || !positions || !next_positions || !lengths_out || !weights_out || !positions_out)
    return fail(QMV_EINVAL, "%s: null array", fn);
  if (lengths_out == lengths || weights_out == weights || positions_out == positions)
    return fail(QMV_EINVAL, "%s: the outputs must not be the inputs", fn);
  const EvictPlan p = evict_plan(B, cache->heads, S, budget);
  if (!workspace || workspace_bytes < p.bytes)
    return fail(QMV_EINVAL, "%s: workspace of %zu bytes, %zu are needed", fn, workspace ? workspace_bytes : size_t(0), p.bytes);
  if (misaligned(workspace, 16)) return fail(QMV_EINVAL, "%s: workspace must be 16-byte aligned", fn);
  EvictArgs a{};
  a.pool = pools_of(*cache);
  a.tab = tables_of(*cache, block_tables, B, cols, table_ld);
  a.lengths = lengths;
  a.next = next_positions;
  a.weights = weights;
  a.positions = positions;
  a.meta_b = meta_b;
  a.meta_h = meta_h;
  a.weights_out = weights_out;
  a.positions_out = positions_out;
  a.lengths_out = lengths_out;
  a.moves = static_cast<int32_t *>(workspace);
  a.stay = reinterpret_cast<uint64_t *>(static_cast<uint8_t *>(workspace) + p.stay);
  a.mask_words = p.mask_words;
  a.counts = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(workspace) + p.counts);
  a.heads = cache->heads;
  a.S = static_cast<int>(S);
  a.budget = static_cast<int>(budget);
  a.recent = static_cast<int>(recent);
  a.most = p.most;
  a.row_bytes = row_bytes(*cache);
  a.groups = groups(*cache);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t bh = B * cache->heads;
  const int64_t cap = cols * cache->page_size, longest = S < cap ? S : cap;
  const dim3 grid(static_cast<unsigned>(bh)), block(kEvictThreads);
  if (longest <= kEvictResident) {
    const size_t lds = static_cast<size_t>(round_up(longest, kEvictWaves * kEvictStep)) * 4;
    auto kern = evict_select_kernel<true>;
    if (lds > 32 * 1024)
      (void)hipFuncSetAttribute(reinterpret_cast<const void *>(kern), hipFuncAttributeMaxDynamicSharedMemorySize,
                                kEvictResident * 4);
    hipLaunchKernelGGL(kern, grid, block, lds, st, a);
  } else {
    hipLaunchKernelGGL(evict_select_kernel<false>, grid, block, 0, st, a);
  }
  if (int rc = check_launch(fn)) return rc;
  // about 8192 workgroups that move rows, with 16 rows or more each
  constexpr int64_t kRows = kMoveThreads / 16;
  const int64_t share = 8192 / bh > 1 ? 8192 / bh : 1;
  int64_t move = (p.most + kRows - 1) / kRows, meta = (S + 4 * kMoveThreads - 1) / (4 * kMoveThreads);
  if (move > share) move = share;
  if (meta > share) meta = share;
  if (bh * (move + meta) > 0x7FFFFFFF) return fail(QMV_EUNSUPPORTED, "%s: too many heads", fn);
  hipLaunchKernelGGL(evict_move_kernel, dim3(static_cast<unsigned>(bh * (move + meta))), dim3(kMoveThreads), 0, st, a,
                     static_cast<int>(move), static_cast<int>(meta));
  return check_launch(fn);
}

int qmv_beam_select_workspace_bytes(int64_t B, int64_t W, int64_t V, int num, size_t *bytes) {
  const char *fn = "qmv_beam_select_workspace_bytes";
  if (!bytes) return fail(QMV_EINVAL, "%s: null bytes", fn);
  if (int rc = check_beam(fn, B, W, V, num)) return rc;
  *bytes = beam_plan(B * W, V, num).bytes;
  return ok();
}

int qmv_beam_select(const void *logits, int logits_dtype, int64_t logits_ld, const float *scores, int64_t B,
                    int64_t W, int64_t V, int num, float *out_scores, int32_t *out_parents, int32_t *out_tokens,
                    void *workspace, size_t workspace_bytes, void *stream) {
  const char *fn = "qmv_beam_select";
  if (int rc = check_beam(fn, B, W, V, num)) return rc;
  if (logits_dtype != QMV_OUT_BF16 && logits_dtype != QMV_OUT_F32) return fail(QMV_EINVAL, "%s: logits_dtype=%d", fn, logits_dtype);
  if (!logits || !scores || !out_scores || !out_parents || !out_tokens) return fail(QMV_EINVAL, "%s: null array", fn);
  if (misaligned(logits, logits_dtype == QMV_OUT_F32 ? 4 : 2) || logits_ld < V)
    return fail(QMV_EINVAL, "%s: logits misaligned, or row stride %lld below V=%lld", fn, (long long)logits_ld, (long long)V);
  const BeamPlan p = beam_plan(B * W, V, num);
  if (!workspace || workspace_bytes < p.bytes)
    return fail(QMV_EINVAL, "%s: workspace of %zu bytes, %zu are needed", fn, workspace ? workspace_bytes : size_t(0), p.bytes);
  if (misaligned(workspace, 16)) return fail(QMV_EINVAL, "%s: workspace must be 16-byte aligned", fn);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  BeamArgs a{};
  a.logits = logits;
  a.scores = scores;
  a.logits_ld = logits_ld;
  a.m = reinterpret_cast<float *>(ws + p.m);
  a.l = reinterpret_cast<float *>(ws + p.l);
  a.left_out = reinterpret_cast<float *>(ws + p.left);
  a.list = reinterpret_cast<u32x2 *>(ws + p.list);
  a.out_scores = out_scores;
  a.out_parents = out_parents;
  a.out_tokens = out_tokens;
  a.B = static_cast<int>(B);
  a.W = static_cast<int>(W);
  a.V = static_cast<int>(V);
  a.num = num;
  a.chunks = p.chunks;
  a.f32 = logits_dtype == QMV_OUT_F32;
  hipStream_t st = static_cast<hipStream_t>(stream);
  a.per_row = divider(static_cast<uint32_t>(p.chunks * num));
  a.per_chunk = divider(static_cast<uint32_t>(p.chunks));
  const dim3 grid(static_cast<unsigned>(B * W * p.chunks)), block(kScanThreads);
  if (p.per == 64) hipLaunchKernelGGL(beam_scan_kernel<64>, grid, block, 0, st, a);
  else if (p.per == 32) hipLaunchKernelGGL(beam_scan_kernel<32>, grid, block, 0, st, a);
  else hipLaunchKernelGGL(beam_scan_kernel<16>, grid, block, 0, st, a);
  if (int rc = check_launch(fn)) return rc;
  hipLaunchKernelGGL(beam_join_kernel, dim3(static_cast<unsigned>(B)), dim3(kJoinThreads), static_cast<size_t>(W) * 8,
                     st, a);
  return check_launch(fn);
}

int qmv_beam_reorder(const qmv_kv_cache *cache, const int32_t *block_tables, const int32_t *lengths, int64_t B,
                     int64_t W, int64_t cols, const int32_t *parents, int64_t parents_ld, int64_t M,
                     const int32_t *spare_pages, int32_t *tables_out, int32_t *lengths_out, void *stream) {
  const char *fn = "qmv_beam_reorder";
  if (int rc = check_cache(fn, cache)) return rc;
  if (B < 1 || W < 1 || M < 1) return fail(QMV_EINVAL, "%s: B=%lld, W=%lld and M=%lld must be positive", fn, (long long)B, (long long)W, (long long)M);
  if (W > (1 << 20) || M > (1 << 20)) return fail(QMV_EINVAL, "%s: W=%lld or M=%lld too large", fn, (long long)W, (long long)M);
  if (int rc = check_tables(fn, cache, block_tables, B, cols, cols)) return rc;
  if (!lengths || !parents || !spare_pages || !tables_out || !lengths_out) return fail(QMV_EINVAL, "%s: null array", fn);
  if (parents_ld < M) return fail(QMV_EINVAL, "%s: parents stride %lld below M=%lld", fn, (long long)parents_ld, (long long)M);
  if (tables_out == block_tables || lengths_out == lengths) return fail(QMV_EINVAL, "%s: the outputs must not be the inputs", fn);
  if (static_cast<int64_t>(cache->heads) * cache->page_size > kMaxSlots)   // a page's rows are numbered in 32 bits
    return fail(QMV_EUNSUPPORTED, "%s: %d heads of %d slots a page are too many", fn, cache->heads, cache->page_size);
  ReorderArgs a{};
  a.pool = pools_of(*cache);
  a.tables = block_tables;
  a.lengths = lengths;
  a.parents = parents;
  a.spare = spare_pages;
  a.tables_out = tables_out;
  a.lengths_out = lengths_out;
  a.parents_ld = parents_ld;
  a.per_page = divider(static_cast<uint32_t>(cache->page_size));
  a.W = static_cast<int>(W);
  a.M = static_cast<int>(M);
  a.cols = static_cast<int>(cols);
  a.heads = cache->heads;
  a.row_bytes = row_bytes(*cache);
  a.groups = groups(*cache);
  int64_t parts = 1 + (static_cast<int64_t>(cache->heads) * cache->page_size + 15) / 16;
  const int64_t most = 4096 / (B * M) > 2 ? 4096 / (B * M) : 2;
  if (parts > most) parts = most;
  a.parts = static_cast<int>(parts);
  if (B * M * parts > 0x7FFFFFFF) return fail(QMV_EUNSUPPORTED, "%s: too many beams", fn);
  hipLaunchKernelGGL(reorder_kernel, dim3(static_cast<unsigned>(B * M * parts)), dim3(kReorderThreads), 0,
                     static_cast<hipStream_t>(stream), a);
  return check_launch(fn);
}

}  // extern "C"
