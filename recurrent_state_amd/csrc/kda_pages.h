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
