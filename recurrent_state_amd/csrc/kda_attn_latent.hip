// Attention of a sequence's new tokens over a latent cache.
//
// One wave per query row and head walks the tokens that the row sees, with the
// softmax's running maximum and sum: m' = max(m, s), l = l e^(m - m') +
// e^(s - m'), and the output the same.  Everything after the loads is fp32.

#include "kda_pages.h"

namespace kda {
namespace {

struct AttnArgs {
  KvBatch kb;
  KvRows q;
  float scale;
  int32_t window;
  void* o;
  float* lse;
};

__device__ __forceinline__ float widen1(bf16_t x) { return __uint_as_float((uint32_t)x << 16); }
__device__ __forceinline__ void store1(bf16_t* p, float x) { *p = __builtin_bit_cast(uint16_t, (__bf16)x); }

template <int DK, int DV, typename TIn, typename TC>
__global__ void __launch_bounds__(kWave) attn_kernel(AttnArgs a) {
  constexpr bool kLatent = DK != DV;
  const KvBatch& kb = a.kb;
  const int lane = threadIdx.x, b = blockIdx.x / kb.s.T, i = blockIdx.x % kb.s.T, h = blockIdx.y;
  const int hk = h / (kb.s.Hq / kb.s.Hkv);
  const SeqRows sr = seq_rows(kb, b);
  if (sr.bad && lane == 0) set_err(kb.dev_err, KDA_DEV_ERR_TOKENS);
  if (sr.bad || i >= sr.n) return;
  const int64_t pos = kb.pos[b], p = pos + i, end = pos + sr.n;
  const int32_t* table = kb.table + (int64_t)b * kb.max_pages;
  bool bad = end > ((int64_t)kb.max_pages << kb.page_shift);
  if (!bad && end > 0) {
    const int64_t lo = a.window > 0 && pos + 1 > a.window ? pos + 1 - a.window : 0;
    for (int64_t g = (lo >> kb.page_shift) + lane; g <= (end - 1) >> kb.page_shift; g += kWave)
      bad |= table[g] < 0 || table[g] >= kb.pages.n_pages;
  }
  if (__ballot(bad) != 0) {
    if (lane == 0) set_err(kb.dev_err, KDA_DEV_ERR_PAGE);
    return;
  }
  const int row = sr.row0 + i;
  const TIn* q = static_cast<const TIn*>(a.q.p) + row * a.q.stride + h * DK;
  float qv[DK / kWave], acc[DV / kWave], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int d = 0; d < DK / kWave; ++d) qv[d] = widen1(q[d * kWave + lane]);
#pragma unroll
  for (int d = 0; d < DV / kWave; ++d) acc[d] = 0.f;
  const float ks = kb.pages.k_scale ? kb.pages.k_scale[hk] : 1.f;
  const float vs = kb.pages.v_scale && !kLatent ? kb.pages.v_scale[hk] : 1.f;
  for (int64_t j = a.window > 0 && p + 1 > a.window ? p + 1 - a.window : 0; j <= p; ++j) {
    const int64_t at = (((int64_t)table[j >> kb.page_shift] * kb.s.Hkv + hk) << kb.page_shift) +
                       (j & (kb.pages.page_size - 1));
    const TC* k = static_cast<const TC*>(kb.pages.k) + at * DK;
    const TC* v = kLatent ? k : static_cast<const TC*>(kb.pages.v) + at * DV;
    float s = 0.f;
#pragma unroll
    for (int d = 0; d < DK / kWave; ++d) s = __builtin_fmaf(qv[d], widen1(k[d * kWave + lane]), s);
    s = wave_sum(s) * ks * a.scale;
    const float mn = fmaxf(m, s), keep = m == mn ? 1.f : __expf(m - mn);
    const float w = s == -INFINITY ? 0.f : __expf(s - mn);
    m = mn;
    l = l * keep + w;
#pragma unroll
    for (int d = 0; d < DV / kWave; ++d) acc[d] = acc[d] * keep + w * widen1(v[d * kWave + lane]);
  }
  const float inv = l == 0.f ? 0.f : vs / l;
  TIn* o = static_cast<TIn*>(a.o) + ((int64_t)row * kb.s.Hq + h) * DV;
#pragma unroll
  for (int d = 0; d < DV / kWave; ++d) store1(o + d * kWave + lane, acc[d] * inv);
  if (a.lse && lane == 0) a.lse[(int64_t)row * kb.s.Hq + h] = m + __logf(l);
}

template <int DK, int DV, typename TIn, typename TC>
hipError_t run(const AttnArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((attn_kernel<DK, DV, TIn, TC>), dim3(a.kb.s.B * a.kb.s.T, a.kb.s.Hq), dim3(kWave), 0, st, a);
  return hipGetLastError();
}

}  // namespace

size_t latent_workspace_bytes(const kda_kv_shape&, int32_t, int32_t) { return 256; }

hipError_t launch_attn_latent(const KvBatch& b, KvRows q, float scale, int32_t window, void* o, float* lse, void*,
                              hipStream_t st) {
  const AttnArgs a{b, q, scale, window, o, lse};
  return run<576, 512, bf16_t, bf16_t>(a, st);
}

}  // namespace kda
