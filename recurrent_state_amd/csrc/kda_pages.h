// Device helpers of the paged attention calls (kda_pages.hip, kda_attn.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "kda_common.h"
#include "kda_internal.h"

namespace kda {
namespace {

__device__ __forceinline__ void set_err(int32_t* dev_err, int32_t bit) { atomicOr(dev_err, bit); }

// x, as a value that the compiler knows nothing of: what is computed from it
// stays where it is used, instead of being hoisted out of the loops around
// and held in registers (or spilled) for all of them.
__device__ __forceinline__ int here(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// A value clamped to e4m3's largest (the type has no infinity); NaN stays NaN.
__device__ __forceinline__ float to_range(float y) { return y != y ? y : fminf(fmaxf(y, -448.f), 448.f); }

// Inclusive sum over the wave's lanes: inside each 16-lane row by shifts of 1,
// 2, 4 and 8, then the last lane of a row to the row after it and of the lower
// half to the upper.  No LDS, no barrier.
__device__ __forceinline__ int32_t wave_scan(int32_t x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, true);   // row_shr:1
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, true);   // row_shr:2
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, true);   // row_shr:4
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, true);   // row_shr:8
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // row_bcast:15 into rows 1 and 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // row_bcast:31 into rows 2 and 3
  return x;
}

// The new tokens of sequence b: packed rows row0 .. row0 + n - 1.  n = 0 for a
// sequence that sits the call out; bad: its range does not fit the launch.
struct SeqRows {
  int32_t row0, n;
  bool bad;
};
// Whether rows r0 .. r1 - 1 can be a sequence's.
__device__ __forceinline__ bool fits(const KvBatch& kb, int64_t r0, int64_t r1) {
  return r0 >= 0 && r1 >= r0 && r1 <= kb.n_tokens && r1 - r0 <= kb.s.T;
}
__device__ __forceinline__ SeqRows seq_rows(const KvBatch& kb, int b) {
  if (!kb.tok_start) return SeqRows{b * kb.s.T, kb.s.T, false};
  const int64_t r0 = kb.tok_start[b], r1 = kb.tok_start[b + 1];
  if (!fits(kb, r0, r1)) return SeqRows{0, 0, true};
  return SeqRows{(int32_t)r0, (int32_t)(r1 - r0), false};
}

}  // namespace
}  // namespace kda
