// Launching the attention kernel; its instances are compiled in one
// translation unit per row type.
#pragma once

#include "host_error.h"
#include "kv_attend_kernels.h"

namespace qmvd {

int attend_b16(const AttendArgs &a, int64_t chunks, int D, int gs, int hb, hipStream_t st);
int attend_b8(const AttendArgs &a, int64_t chunks, int D, int gs, int hb, hipStream_t st);
int attend_b4(const AttendArgs &a, int64_t chunks, int D, int gs, int hb, hipStream_t st);

// Pages of whole 16-token lines, and 16 slots' bytes within a 32-bit offset.
inline bool attend_paged16(const AttendArgs &a) { return a.pool.page_size % 16 == 0 && a.pool.slot_rows < (1 << 18); }

template <typename S>
int launch_attend(const AttendArgs &a, int64_t chunks, hipStream_t st) {
  const int64_t blocks = chunks * a.heads * a.head_blocks;
  if (blocks > 0x7FFFFFFF) return fail(QMV_EUNSUPPORTED, "qmv_kv_attend: too many workgroups");
  constexpr int kWave = 4 * attend_wave_lds(S::D, S::BITS, S::NG, S::HB);
  static_assert(attend_most_waves(S::D) * kWave <= 67 * 1024, "two workgroups of the most waves a CU");
  const int lds = a.waves * kWave;
  auto kern = attend_kernel<S>;
  if (lds > 64 * 1024)
    (void)hipFuncSetAttribute(reinterpret_cast<const void *>(kern), hipFuncAttributeMaxDynamicSharedMemorySize,
                              lds);
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(blocks)), dim3(64 * a.waves), static_cast<size_t>(lds), st, a);
  return check_launch("qmv_kv_attend");
}

}  // namespace qmvd
