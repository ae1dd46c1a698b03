// Eviction from the paged cache: which tokens each kv head keeps, and their move
// to other pages.
//
//   select  One workgroup to a (sequence, kv head).  The keys that order the
//           candidates are 32-bit numbers; the k-th greatest is found digit by
//           digit (11, 11 and 10 bits), each a histogram in the LDS of those that
//           share the digits above.  Then every wave counts, in its own stretch
//           of tokens, those above it and those equal to it, and after one scan
//           over the waves writes its kept places in order.
//   move    Rows go from their places to the new ones.  Pages without scales or
//           with scales by heads are copied 16 bytes to a thread; where scales go
//           by blocks, a group of waves takes a new block, whose scale is that of
//           its largest value.

#include "kda_blocks.h"

namespace kda {
namespace {

struct EvictArgs {
  KvBatch kb;  // pos: the lengths
  BlockScales scales;
  const float* weights;
  int64_t stride;  // of weights and new_weights: a (sequence, kv head)
  int32_t keep, recent;
  const int32_t* dst_table;
  int32_t dst_max_pages;
  int64_t* new_len;
  float* new_weights;
  int32_t* kept;
};

constexpr int kSelect = 1024, kSelectWaves = kSelect / kWave, kBins = 2048;

// Numbers that order as the weights do: NaN first, -0 and 0 alike.
__device__ __forceinline__ uint32_t order(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  return w != w ? 0u : (u >> 31) ? ~u : u | 0x80000000u;
}

// Inclusive sum over the workgroup's threads.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* lds) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const uint32_t upto = (uint32_t)wave_scan((int32_t)x);
  __syncthreads();
  if (lane == kWave - 1) lds[wave] = upto;
  __syncthreads();
  uint32_t before = 0;
#pragma unroll
  for (int i = 0; i < kSelectWaves; ++i) before += i < wave ? lds[i] : 0;
  return before + upto;
}

__global__ void __launch_bounds__(kSelect) select_kernel(EvictArgs a) {
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t lds_scan[kSelectWaves];
  __shared__ uint32_t found[2];  // the digit, and how many keys are above it
  __shared__ uint2 counts[kSelectWaves];
  const KvBatch& kb = a.kb;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int b = blockIdx.x / kb.s.Hkv;
  const float* const w = a.weights + (int64_t)blockIdx.x * a.stride;
  float* const out_w = a.new_weights + (int64_t)blockIdx.x * a.stride;
  int32_t* const kept = a.kept + (int64_t)blockIdx.x * a.keep;
  const int64_t len = kb.pos[b];
  bool bad = len < 0 || len > ((int64_t)kb.max_pages << kb.page_shift);
  const int L = bad ? 0 : (int)len;
  const bool stays = L <= a.keep;
  if (!bad && !stays) {
    const int page_size = kb.pages.page_size;
    const auto outside = [&](int32_t id) { return id < 0 || id >= kb.pages.n_pages; };
    bool off = false;
    for (int i = tid; i < (L + page_size - 1) >> kb.page_shift; i += kSelect)
      off |= outside(kb.table[(int64_t)b * kb.max_pages + i]);
    for (int i = tid; i < (a.keep + page_size - 1) >> kb.page_shift; i += kSelect)
      off |= outside(a.dst_table[(int64_t)b * a.dst_max_pages + i]);
    bad = __syncthreads_or(off);
  }
  if (bad && tid == 0) set_err(kb.dev_err, KDA_DEV_ERR_PAGE);
  if (bad || stays) {
    for (int i = tid; i < a.keep; i += kSelect) kept[i] = -1;
    for (int64_t j = tid; j < a.stride; j += kSelect) out_w[j] = !bad && j < L ? w[j] : 0.f;
    return;
  }

  // The threshold: of the n candidates' keys the k-th greatest, and how many are above.
  const int n = L - a.recent, k = a.keep - a.recent;
  uint32_t top = 0, above = 0;  // digits so far; keys greater than any with these
  if (k > 0) {
    constexpr int kShift[3] = {21, 10, 0}, kBits[3] = {11, 11, 10};
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = kShift[pass];
      const uint32_t mask = (1u << kBits[pass]) - 1;
      hist[tid] = 0, hist[tid + kSelect] = 0;
      __syncthreads();
#pragma unroll 4
      for (int j = tid; j < n; j += kSelect) {
        const uint32_t key = order(w[j]);
        if (pass == 0 || key >> (shift + kBits[pass]) == top) atomicAdd(&hist[key >> shift & mask], 1u);
      }
      __syncthreads();
      // From the greatest digit down, two to a thread.
      const int d0 = kBins - 1 - 2 * tid;
      const uint32_t c0 = hist[d0], c1 = hist[d0 - 1], upto = block_scan(c0 + c1, lds_scan) + above;
      const uint32_t before = upto - c0 - c1;
      if (before < (uint32_t)k && upto >= (uint32_t)k) {  // one thread
        const bool second = before + c0 < (uint32_t)k;
        found[0] = second ? d0 - 1 : d0;
        found[1] = second ? before + c0 : before;
      }
      __syncthreads();
      top = top << kBits[pass] | found[0];
      above = found[1];
    }
  }
  const uint32_t equal = k > 0 ? (uint32_t)k - above : 0;  // of those at the threshold, the first so many

  // Each wave's stretch of the candidates.
  const int each = (n + kSelect - 1) / kSelect * kWave, j0 = min(wave * each, n), j1 = min(j0 + each, n);
  if (k > 0) {
    uint32_t gt = 0, eq = 0;
#pragma unroll 4
    for (int j = j0 + lane; j - lane < j1; j += kWave) {
      const uint32_t key = j < j1 ? order(w[j]) : 0;
      gt += __popcll(__ballot(j < j1 && key > top));
      eq += __popcll(__ballot(j < j1 && key == top));
    }
    if (lane == 0) counts[wave] = make_uint2(gt, eq);
    __syncthreads();
    gt = eq = 0;
    for (int i = 0; i < wave; ++i) gt += counts[i].x, eq += counts[i].y;
    const uint64_t below = ((uint64_t)1 << lane) - 1;
#pragma unroll 4
    for (int j = j0 + lane; j - lane < j1; j += kWave) {
      const float x = j < j1 ? w[j] : 0.f;
      const uint32_t key = order(x);
      const uint64_t is_gt = __ballot(j < j1 && key > top), is_eq = __ballot(j < j1 && key == top);
      const uint32_t g = gt + __popcll(is_gt & below), e = eq + __popcll(is_eq & below);
      if (j < j1 && (key > top || (key == top && e < equal))) {
        const uint32_t at = g + min(e, equal);
        kept[at] = j;
        out_w[at] = x;
      }
      gt += __popcll(is_gt);
      eq += __popcll(is_eq);
    }
  }
  for (int i = tid; i < a.recent; i += kSelect) {
    kept[k + i] = n + i;
    out_w[k + i] = w[n + i];
  }
  for (int64_t j = a.keep + tid; j < a.stride; j += kSelect) out_w[j] = 0.f;
}

// Where a place of a sequence lies, in rows of the pool.
__device__ __forceinline__ int64_t row_at(const KvBatch& kb, const int32_t* table, int h, int place) {
  return (((int64_t)table[place >> kb.page_shift] * kb.s.Hkv + h) << kb.page_shift) +
         (place & (kb.pages.page_size - 1));
}
// The first workgroup of a sequence sets its length.
__device__ __forceinline__ void set_length(const EvictArgs& a, int b) {
  if (threadIdx.x == 0) a.new_len[b] = a.kept[(int64_t)b * a.kb.s.Hkv * a.keep] >= 0 ? a.keep : a.kb.pos[b];
}

constexpr int kMove = 256;

// Rows of `units` 16-byte units.  Workgroups (b, part) by x; y: kv heads, of keys and then of values.
__global__ void __launch_bounds__(kMove) move_kernel(EvictArgs a, int units, int parts) {
  const KvBatch& kb = a.kb;
  const int b = blockIdx.x / parts, part = blockIdx.x % parts;
  const bool values = (int)blockIdx.y >= kb.s.Hkv;
  const int h = values ? blockIdx.y - kb.s.Hkv : blockIdx.y;
  if (part == 0 && blockIdx.y == 0) set_length(a, b);
  const int32_t* const kept = a.kept + ((int64_t)b * kb.s.Hkv + h) * a.keep;
  if (kept[0] < 0) return;
  u32x4* const pool = static_cast<u32x4*>(values ? kb.pages.v : kb.pages.k);
  const int32_t* const from = kb.table + (int64_t)b * kb.max_pages;
  const int32_t* const to = a.dst_table + (int64_t)b * a.dst_max_pages;
  const int64_t total = (int64_t)a.keep * units;
#pragma unroll 4
  for (int64_t x = (int64_t)part * kMove + threadIdx.x; x < total; x += (int64_t)parts * kMove) {
    const int i = (int)(x / units), c = (int)(x - (int64_t)i * units);
    pool[row_at(kb, to, h, i) * units + c] = pool[row_at(kb, from, h, kept[i]) * units + c];
  }
}

// W waves to a new block of one kv head; NW waves to a workgroup.
template <int D, int W>
__global__ void __launch_bounds__(64 * (W > 4 ? W : 4)) move_blocks_kernel(EvictArgs a, int parts) {
  constexpr int NW = W > 4 ? W : 4, HELD = NW / W;
  constexpr int LPR = D / 16, RPP = kWave / LPR, PASSES = 16 / RPP;
  __shared__ uint32_t lds_max[NW];
  const KvBatch& kb = a.kb;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = threadIdx.x & 63, group = wave % W;
  const int b = blockIdx.x / parts, part = blockIdx.x % parts;
  const bool values = (int)blockIdx.y >= kb.s.Hkv;
  const int h = values ? blockIdx.y - kb.s.Hkv : blockIdx.y;
  if (part == 0 && blockIdx.y == 0) set_length(a, b);
  const int32_t* const kept = a.kept + ((int64_t)b * kb.s.Hkv + h) * a.keep;
  if (kept[0] < 0) return;
  uint8_t* const pool = static_cast<uint8_t*>(values ? kb.pages.v : kb.pages.k);
  float* const scales = values ? a.scales.v : a.scales.k;
  const int32_t* const from = kb.table + (int64_t)b * kb.max_pages;
  const int32_t* const to = a.dst_table + (int64_t)b * a.dst_max_pages;
  const int shift = a.scales.shift, blocks = (a.keep + (1 << shift) - 1) >> shift;
  for (int at = part * HELD; at < blocks; at += parts * HELD) {
    const int block = at + wave / W;
    const int begin = block << shift, count = block < blocks ? min(a.keep - begin, 1 << shift) : 0;
    codes16 x[PASSES];
    float was[PASSES];
    uint32_t m = 0;
    auto load = [&](int first) __attribute__((always_inline)) {
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int i = first + group * 16 + p * RPP + lane / LPR;
        x[p] = codes16{};
        was[p] = 0.f;
        if (i >= count) continue;
        const int64_t row = row_at(kb, from, h, kept[begin + i]);
        x[p] = *reinterpret_cast<const codes16*>(pool + row * D + 16 * (lane % LPR));
        was[p] = scales[row >> shift];
      }
    };
    for (int first = 0; first < 1 << shift; first += 16 * W) {
      load(first);
#pragma unroll
      for (int p = 0; p < PASSES; ++p)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)x[p][n], false);
          const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)x[p][n], true);
          m = max(max(m, max(finite_bits(lo[0] * was[p]), finite_bits(lo[1] * was[p]))),
                  max(finite_bits(hi[0] * was[p]), finite_bits(hi[1] * was[p])));
        }
    }
    m = wave_max(m);
    if (W > 1) {
      __syncthreads();
      if (lane == 0) lds_max[wave] = m;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < W; ++i) m = max(m, lds_max[wave - group + i]);
    }
    const uint32_t s = scale_for(m);
    const int64_t dst = count > 0 ? row_at(kb, to, h, begin) : 0;
    if (count > 0 && group == 0 && lane == 0) scales[dst >> shift] = __uint_as_float(s);
    for (int first = 0; first < 1 << shift; first += 16 * W) {
      if (1 << shift > 16 * W) load(first);
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int i = first + group * 16 + p * RPP + lane / LPR;
        if (i < count)
          *reinterpret_cast<codes16*>(pool + (dst + i) * D + 16 * (lane % LPR)) = rescaled(x[p], was[p] * inverse(s));
      }
    }
  }
}

template <int D, int W>
hipError_t run_blocks(const EvictArgs& a, hipStream_t st) {
  constexpr int NW = W > 4 ? W : 4;
  const int blocks = (a.keep + (1 << a.scales.shift) - 1) >> a.scales.shift;
  const int64_t groups = (int64_t)a.kb.s.B * a.kb.s.Hkv * 2;
  int64_t parts = (blocks + NW / W - 1) / (NW / W);
  const int64_t most = (((int64_t)1 << 32) - 1) / (groups * NW * kWave);  // threads of a launch
  if (parts > most) parts = most < 1 ? 1 : most;
  hipLaunchKernelGGL((move_blocks_kernel<D, W>), dim3((unsigned)(a.kb.s.B * parts), a.kb.s.Hkv * 2), dim3(NW * kWave), 0,
                     st, a, (int)parts);
  return hipGetLastError();
}
template <int D>
hipError_t by_block(const EvictArgs& a, hipStream_t st) {
  switch (a.scales.shift) {
    case 4: return run_blocks<D, 1>(a, st);
    case 5: return run_blocks<D, 2>(a, st);
    case 6: return run_blocks<D, 4>(a, st);
    case 7: return run_blocks<D, 8>(a, st);
  }
  return run_blocks<D, 16>(a, st);
}

}  // namespace

hipError_t launch_kv_evict(const KvBatch& b, const BlockScales& scales, const float* weights, int64_t stride,
                           int32_t keep, int32_t recent, const int32_t* dst_table, int32_t dst_max_pages,
                           int64_t* new_len, float* new_weights, int32_t* kept, hipStream_t st) {
  const EvictArgs a{b, scales, weights, stride, keep, recent, dst_table, dst_max_pages, new_len, new_weights, kept};
  const kda_kv_shape& s = b.s;
  hipLaunchKernelGGL(select_kernel, dim3((unsigned)(s.B * s.Hkv)), dim3(kSelect), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (scales.k) return s.dk == 128 ? by_block<128>(a, st) : by_block<64>(a, st);
  const int es = s.cache_dtype == KDA_F32 ? 4 : s.cache_dtype == KDA_BF16 ? 2 : 1;
  const int units = s.dk * es / 16, sides = b.pages.v ? 2 : 1;
  int64_t parts = ((int64_t)keep * units + 4 * kMove - 1) / (4 * kMove);
  const int64_t most = (((int64_t)1 << 32) - 1) / ((int64_t)s.B * s.Hkv * sides * kMove);
  if (parts > most) parts = most < 1 ? 1 : most;
  hipLaunchKernelGGL(move_kernel, dim3((unsigned)(s.B * parts), s.Hkv * sides), dim3(kMove), 0, st, a, units,
                     (int)parts);
  return hipGetLastError();
}

}  // namespace kda
