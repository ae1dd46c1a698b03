// Eviction from the paged cache: which tokens each kv head keeps, and their move
// to other pages.
//
//   select  One workgroup to a (sequence, kv head), or, for few long rows, one to
//           every 8192 of its tokens.  The keys that order the candidates are
//           32-bit numbers; the k-th greatest is found digit by digit (11, 11 and
//           10 bits), each a histogram in the LDS of those that share the digits
//           above.  Then every wave counts, in its own stretch of tokens, those
//           above it and those equal to it, and after one scan over the waves
//           writes its kept places in order.  Bound by the passes' latency:
//           8 heads' 100001 tokens take 26 us in parts, 64 by one workgroup each;
//           64 sequences of up to 8191 tokens, 8 heads, 15 us.
//   move    Rows go from their places to the new ones.  Pages without scales or
//           with scales by heads are copied 16 bytes to a thread; where scales go
//           by blocks, a group of waves takes a new block, whose scale is that of
//           its largest value.  Bound by memory: 20000 tokens of 8 heads of 128 in
//           bf16 32 us (5.2 TB/s), those 64 sequences cut to 2000 e4m3 tokens 58.

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

constexpr int kSelect = 1024, kSelectWaves = kSelect / kWave, kBins = 2048, kList = 8192;
constexpr int kShort = 8 * kSelect;  // candidates that a workgroup holds in registers

// Numbers that order as the weights do: NaN first, -0 and 0 alike.
__device__ __forceinline__ uint32_t order(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  return w != w ? 0u : u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// How many lanes of a mask come before this one, added to `n`.
__device__ __forceinline__ uint32_t lanes_before(uint64_t mask, uint32_t n) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, n));
}

struct SelectLds {
  uint32_t hist[kBins];
  uint32_t scan[kSelectWaves];
  uint32_t found[3];           // the digit, how many keys are above it, and how many have it
  uint32_t gt[kSelectWaves], eq[kSelectWaves];  // of each wave's candidates, above the threshold and at it
  uint32_t length;
  uint32_t list[kList];        // keys that share the first digit
  uint8_t wave[kList];         // and whose candidates they are
};

// The digit of the k-th greatest key, from the histogram of `bins` digits and the
// count of keys above them all; sets lds.found.
__device__ __forceinline__ void find_digit(SelectLds& lds, uint32_t above, uint32_t k) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  __syncthreads();
  // From the greatest digit down, two to a thread.
  const int d0 = kBins - 1 - 2 * tid;
  const uint32_t c0 = lds.hist[d0], c1 = lds.hist[d0 - 1];
  uint32_t upto = (uint32_t)wave_scan((int32_t)(c0 + c1));
  if (lane == kWave - 1) lds.scan[wave] = upto;
  __syncthreads();
  upto += above;
#pragma unroll
  for (int i = 0; i < kSelectWaves; ++i) upto += i < wave ? lds.scan[i] : 0;
  const uint32_t before = upto - c0 - c1;
  if (before < k && upto >= k) {  // one thread
    const bool second = before + c0 < k;
    lds.found[0] = second ? d0 - 1 : d0;
    lds.found[1] = second ? before + c0 : before;
    lds.found[2] = second ? c1 : c0;
  }
  __syncthreads();
}
__device__ __forceinline__ void clear_hist(SelectLds& lds) {
  __syncthreads();
  lds.hist[threadIdx.x] = 0, lds.hist[threadIdx.x + kSelect] = 0;
  __syncthreads();
}

// The places that a wave keeps: behind those of the waves before it (lds.gt and
// lds.eq, which all have set) and gt and eq of the parts before those.
struct Kept {
  uint32_t gt, eq;  // so far: above the threshold, and at it

  __device__ __forceinline__ Kept(const SelectLds& lds, uint32_t gt0, uint32_t eq0) : gt(gt0), eq(eq0) {
    const int wave = threadIdx.x >> 6;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSelectWaves; ++i) gt += i < wave ? lds.gt[i] : 0, eq += i < wave ? lds.eq[i] : 0;
    gt = __builtin_amdgcn_readfirstlane(gt), eq = __builtin_amdgcn_readfirstlane(eq);
  }
  // Of those at the threshold `top` the first `equal` are kept.
  __device__ __forceinline__ void put(int32_t* kept, int j, uint32_t key, bool there, uint32_t top, uint32_t equal) {
    const uint64_t is_gt = __ballot(there && key > top), is_eq = __ballot(there && key == top);
    const uint32_t e = lanes_before(is_eq, eq);
    if (there && (key > top || (key == top && e < equal))) kept[lanes_before(is_gt, gt) + min(e, equal)] = j;
    gt += __popcll(is_gt);
    eq += __popcll(is_eq);
  }
};

// The k greatest of n weights, 0 < k < n: their places to kept, in order.  A wave
// has a stretch of neighbours, 64 at a time.  V: a thread's share, held in
// registers; 0: more than that, read again for every pass, kBatch at once.
template <int V>
__device__ __forceinline__ void select(const float* w, int n, int k, int32_t* kept, SelectLds& lds) {
  constexpr int kBatch = 16;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int each = V > 0 ? V * kWave : (n + kSelect * kBatch - 1) / (kSelect * kBatch) * (kWave * kBatch);
  const int j0 = wave * each, j1 = min(j0 + each, n);  // j1 <= j0: nothing
  float held[V > 0 ? V : 1];
  if constexpr (V > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int j = j0 + i * kWave + lane;
      held[i] = j < j1 ? w[j] : 0.f;
    }
  }
  // f(place, weight, whether it is there) for the wave's stretch, by whole waves.
  auto all = [&](auto f) __attribute__((always_inline)) {
    if constexpr (V > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int j = j0 + i * kWave;
        if (j < j1) f(j + lane, held[i], j + lane < j1);
      }
    } else {
      for (int at = j0; at < j1; at += kWave * kBatch) {
        float x[kBatch];
        if (at + kWave * kBatch <= j1) {
#pragma unroll
          for (int i = 0; i < kBatch; ++i) x[i] = w[at + i * kWave + lane];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) f(at + i * kWave + lane, x[i], true);
        } else {
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int j = at + i * kWave + lane;
            x[i] = j < j1 ? w[j] : 0.f;
          }
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
            if (at + i * kWave < j1) f(at + i * kWave + lane, x[i], at + i * kWave + lane < j1);
        }
      }
    }
  };

  // The threshold, digit by digit, and how many keys are above it.
  clear_hist(lds);
  all([&](int, float x, bool there) {
    if (there) atomicAdd(&lds.hist[order(x) >> 21], 1u);
  });
  find_digit(lds, 0, k);
  uint32_t top = lds.found[0], above = lds.found[1];
  const bool listed = V == 0 && lds.found[2] <= kList;
  if (tid == 0) lds.length = 0;
  if (tid < kSelectWaves) lds.gt[tid] = lds.eq[tid] = 0;
  if (listed) {
    // The keys with that digit fit a list; the others need not be looked at for
    // what is left of the threshold.
    __syncthreads();
    const uint32_t digit = top;
    uint32_t gt = 0;
    all([&](int, float x, bool there) {
      const uint32_t key = order(x);
      gt += __popcll(__ballot(there && key >> 21 > digit));
      const bool in = there && key >> 21 == digit;
      const uint64_t mask = __ballot(in);
      if (mask == 0) return;
      uint32_t at = 0;
      if (lane == 0) at = atomicAdd(&lds.length, (uint32_t)__popcll(mask));
      at = lanes_before(mask, __builtin_amdgcn_readfirstlane(at));
      if (in) lds.list[at] = key, lds.wave[at] = wave;
    });
    if (lane == 0) lds.gt[wave] = gt;
  }
#pragma unroll
  for (int pass = 1; pass < 3; ++pass) {
    const int shift = pass == 1 ? 10 : 0, bits = pass == 1 ? 11 : 10;
    clear_hist(lds);
    if (listed) {
      for (uint32_t i = tid; i < lds.length; i += kSelect)
        if (lds.list[i] >> (shift + bits) == top) atomicAdd(&lds.hist[lds.list[i] >> shift & ((1u << bits) - 1)], 1u);
    } else {
      all([&](int, float x, bool there) {
        const uint32_t key = order(x);
        if (there && key >> (shift + bits) == top) atomicAdd(&lds.hist[key >> shift & ((1u << bits) - 1)], 1u);
      });
    }
    find_digit(lds, above, k);
    top = top << bits | lds.found[0];
    above = lds.found[1];
  }
  const uint32_t equal = (uint32_t)k - above;  // of those at the threshold, the first so many

  // How many of the waves before this one's are kept, then which of its own.
  if (listed) {
    for (uint32_t i = tid; i < lds.length; i += kSelect) {
      const uint32_t key = lds.list[i];
      if (key >= top) atomicAdd(key > top ? &lds.gt[lds.wave[i]] : &lds.eq[lds.wave[i]], 1u);
    }
  } else {
    uint32_t gt = 0, eq = 0;
    all([&](int, float x, bool there) {
      const uint32_t key = order(x);
      gt += __popcll(__ballot(there && key > top));
      eq += __popcll(__ballot(there && key == top));
    });
    if (lane == 0) lds.gt[wave] = gt, lds.eq[wave] = eq;
  }
  __syncthreads();
  Kept from(lds, 0, 0);
  all([&](int j, float x, bool there) { from.put(kept, j, order(x), there, top, equal); });
}

// What is done with a (sequence, kv head).
struct Row {
  const float* w;
  float* out_w;
  int32_t* kept;
  int L, n, k;  // length, candidates, how many of them are kept
  bool bad, stays;

  __device__ __forceinline__ Row(const EvictArgs& a, int64_t bh) {
    const int64_t len = a.kb.pos[bh / a.kb.s.Hkv];
    w = a.weights + bh * a.stride;
    out_w = a.new_weights + bh * a.stride;
    kept = a.kept + bh * a.keep;
    bad = len < 0 || len > ((int64_t)a.kb.max_pages << a.kb.page_shift);
    L = bad ? 0 : (int)len;
    stays = L <= a.keep;
    n = L - a.recent;
    k = a.keep - a.recent;
  }
  // Whether the pages of a sequence to be cut are all there; by a whole workgroup.
  __device__ __forceinline__ void check_pages(const EvictArgs& a, int b) {
    const KvBatch& kb = a.kb;
    if (bad || stays) return;
    const auto outside = [&](int32_t id) { return id < 0 || id >= kb.pages.n_pages; };
    const int last = kb.pages.page_size - 1;
    bool off = false;
    for (int i = threadIdx.x; i < (L + last) >> kb.page_shift; i += kSelect)
      off |= outside(kb.table[(int64_t)b * kb.max_pages + i]);
    for (int i = threadIdx.x; i < (a.keep + last) >> kb.page_shift; i += kSelect)
      off |= outside(a.dst_table[(int64_t)b * a.dst_max_pages + i]);
    bad = __syncthreads_or(off);
  }
  // Part `part` of `parts` of the results that no choice enters: of a row that is
  // left alone all of them, of another the last tokens.
  __device__ __forceinline__ void plain(const EvictArgs& a, int part, int parts) const {
    const int tid = part * kSelect + threadIdx.x, step = parts * kSelect;
    if (bad || stays) {
      for (int i = tid; i < a.keep; i += step) kept[i] = -1;
      for (int64_t j = tid; j < a.stride; j += step) out_w[j] = !bad && j < L ? w[j] : 0.f;
    } else {
      for (int i = tid; i < a.recent; i += step) kept[k + i] = n + i;
    }
  }
};

// LONG: rows may have more than kShort candidates.
template <bool LONG>
__global__ void __launch_bounds__(kSelect, LONG ? 4 : 8) select_kernel(EvictArgs a) {
  __shared__ SelectLds lds;
  Row r(a, blockIdx.x);
  r.check_pages(a, blockIdx.x / a.kb.s.Hkv);
  if (r.bad && threadIdx.x == 0) set_err(a.kb.dev_err, KDA_DEV_ERR_PAGE);
  r.plain(a, 0, 1);
  if (r.bad || r.stays || r.k == 0) return;
  if (!LONG || r.n <= kShort)
    select<kShort / kSelect>(r.w, r.n, r.k, r.kept, lds);
  else
    select<0>(r.w, r.n, r.k, r.kept, lds);
}

// The same with a row's candidates shared out to workgroups, kShort to each, for
// few long rows: a launch for each digit's histogram, by parts, and one that adds
// up the last one's and writes the places.  The row's new_weights, which the move
// writes after them, hold the histograms meanwhile.
struct Parts {
  uint32_t* hist[3];  // [part][bins of the digit]
  uint32_t* gt;       // [part]: keys above the first two digits
  uint32_t* row;      // first digit, keys above it, first two digits, keys above them

  static constexpr int kBinsOf[3] = {2048, 2048, 1024};
  __device__ __forceinline__ Parts(const Row& r, int parts) {
    hist[0] = reinterpret_cast<uint32_t*>(r.out_w);
    hist[1] = hist[0] + parts * 2048;
    hist[2] = hist[1] + parts * 2048;
    gt = hist[2] + parts * 1024;
    row = gt + parts;
  }
  // Words of a row that this takes; no more than a row of (parts - 1) kShort has, from three parts on.
  static constexpr int64_t words(int64_t parts) { return parts * (2048 + 2048 + 1024 + 1) + 4; }

  // The sum of a digit's histograms of the row's parts to lds.hist.  Returned: that
  // of the parts before `part`, of the thread's bin.
  __device__ __forceinline__ uint32_t add_up(int digit, int count, SelectLds& lds, int part) const {
    uint32_t c[2] = {0, 0}, before = 0;
    const uint32_t* p = hist[digit] + threadIdx.x;
#pragma unroll 8
    for (int i = 0; i < count; ++i) {
      const uint32_t x = p[i * kBinsOf[digit]];
      c[0] += x;
      before += i < part ? x : 0;
      if (digit < 2) c[1] += p[i * kBinsOf[digit] + kSelect];
    }
    lds.hist[threadIdx.x] = c[0], lds.hist[threadIdx.x + kSelect] = c[1];
    return before;
  }
};

// Rows are shared out where one workgroup to a row leaves most of the chip idle
// and takes longer than four launches.  Whole calls, shared out and not: 8 rows of
// 41000 tokens 28 and 28 us, of 57000 30 and 35, of 180000 40 and 70; 32 rows 38 and
// 37, 40 and 45, 80 and 82; 64 rows of 57000 57 and 52, of 120000 95 and 72.  The host
// knows the table only: rows that are short in a long one lose by it (8 rows of a
// table of 100001, of 5000 tokens 27 and 18 us, of 20000 30 and 26, of 40000 32 and
// 32, of 60000 30 and 38).
constexpr int kFewestParts = 6, kMostRows = 32, kMostParts = 1024;
constexpr int kEach = kShort / kSelect;  // of a thread: every 64th of its wave's stretch

struct Stretch {
  int j0;
  uint32_t key[kEach];

  __device__ __forceinline__ Stretch(const Row& r, int part) : j0(part * kShort + (threadIdx.x >> 6) * (kEach * kWave)) {
    float x[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) x[i] = there(r, i) ? r.w[place(i)] : 0.f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) key[i] = order(x[i]);
  }
  __device__ __forceinline__ int place(int i) const { return j0 + i * kWave + (threadIdx.x & 63); }
  __device__ __forceinline__ bool there(const Row& r, int i) const { return place(i) < r.n; }
};

template <int DIGIT>
__global__ void __launch_bounds__(kSelect) hist_kernel(EvictArgs a, int parts) {
  __shared__ SelectLds lds;
  const int part = blockIdx.y, tid = threadIdx.x, lane = tid & 63;
  const Row r(a, blockIdx.x);
  if (r.bad || r.stays || r.k == 0 || part * kShort >= r.n) return;
  const Parts p(r, parts);
  const Stretch mine(r, part);
  uint32_t top = 0;
  if (DIGIT > 0) {
    p.add_up(DIGIT - 1, (r.n + kShort - 1) / kShort, lds, 0);
    find_digit(lds, DIGIT == 1 ? 0 : p.row[1], r.k);
    top = DIGIT == 1 ? lds.found[0] : p.row[0] << 11 | lds.found[0];
    if (part == 0 && tid == 0) p.row[2 * DIGIT - 2] = top, p.row[2 * DIGIT - 1] = lds.found[1];
  }
  if (tid == 0) lds.length = 0;
  clear_hist(lds);
  constexpr int kShift[3] = {21, 10, 0};
  uint32_t gt = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const uint32_t key = mine.key[i], digits = key >> kShift[DIGIT];
    const bool there = mine.there(r, i);
    const uint32_t before = DIGIT == 0 ? 0 : DIGIT == 1 ? key >> 21 : key >> 10;
    if (DIGIT == 2) gt += __popcll(__ballot(there && before > top));
    if (there && (DIGIT == 0 || before == top)) atomicAdd(&lds.hist[digits & (Parts::kBinsOf[DIGIT] - 1)], 1u);
  }
  if (DIGIT == 2 && lane == 0) atomicAdd(&lds.length, gt);
  __syncthreads();
  for (int i = tid; i < Parts::kBinsOf[DIGIT]; i += kSelect) p.hist[DIGIT][part * Parts::kBinsOf[DIGIT] + i] = lds.hist[i];
  if (DIGIT == 2 && tid == 0) p.gt[part] = lds.length;
}

__global__ void __launch_bounds__(kSelect) places_kernel(EvictArgs a, int parts) {
  __shared__ SelectLds lds;
  const int part = blockIdx.y, tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  Row r(a, blockIdx.x);
  r.check_pages(a, blockIdx.x / a.kb.s.Hkv);
  if (r.bad && part == 0 && tid == 0) set_err(a.kb.dev_err, KDA_DEV_ERR_PAGE);
  r.plain(a, part, parts);
  if (r.bad || r.stays || r.k == 0 || part * kShort >= r.n) return;
  const Parts p(r, parts);
  const Stretch mine(r, part);
  const uint32_t before = p.add_up(2, (r.n + kShort - 1) / kShort, lds, part);
  find_digit(lds, p.row[3], r.k);
  const uint32_t digit = lds.found[0], top = p.row[2] << 10 | digit, equal = (uint32_t)r.k - lds.found[1];
  // Kept ones of the parts before this, then of the waves.
  __syncthreads();
  if (tid == 0) lds.found[0] = lds.found[1] = 0;
  __syncthreads();
  uint32_t gt = tid < part ? p.gt[tid] : 0, eq = tid < part ? p.hist[2][tid * 1024 + digit] : 0;
  if ((uint32_t)tid > digit) gt += before;
  if (gt) atomicAdd(&lds.found[0], gt);
  if (eq) atomicAdd(&lds.found[1], eq);
  gt = eq = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    gt += __popcll(__ballot(mine.there(r, i) && mine.key[i] > top));
    eq += __popcll(__ballot(mine.there(r, i) && mine.key[i] == top));
  }
  if (lane == 0) lds.gt[wave] = gt, lds.eq[wave] = eq;
  __syncthreads();
  Kept from(lds, lds.found[0], lds.found[1]);
#pragma unroll
  for (int i = 0; i < kEach; ++i) from.put(r.kept, mine.place(i), mine.key[i], mine.there(r, i), top, equal);
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

// The weights of the kept tokens, and zeros behind them: a workgroup's share.
__device__ __forceinline__ void move_weights(const EvictArgs& a, int64_t bh, const int32_t* kept, int part, int parts) {
  const float* const w = a.weights + bh * a.stride;
  float* const out = a.new_weights + bh * a.stride;
  for (int64_t j = (int64_t)part * blockDim.x + threadIdx.x; j < a.stride; j += (int64_t)parts * blockDim.x)
    out[j] = j < a.keep ? w[kept[j]] : 0.f;
}

// kAtOnce: loads on their way of a thread (2 and 8 took as long).
constexpr int kMove = 256, kAtOnce = 4;

// Rows of `units` 16-byte units, keys and values together.  Workgroups (b, part) by
// x; kv heads by y.  The tokens' old places are read for the last time, so past the
// caches (100001 tokens to 20000, 8 heads of 128 in bf16: 33 us for 40).
template <bool VALUES>
__global__ void __launch_bounds__(kMove) move_kernel(EvictArgs a, int units, int parts) {
  const KvBatch& kb = a.kb;
  const int b = blockIdx.x / parts, part = blockIdx.x % parts, h = blockIdx.y;
  if (part == 0 && h == 0) set_length(a, b);
  const int32_t* const kept = a.kept + ((int64_t)b * kb.s.Hkv + h) * a.keep;
  if (kept[0] < 0) return;
  move_weights(a, (int64_t)b * kb.s.Hkv + h, kept, part, parts);
  u32x4* const k = static_cast<u32x4*>(kb.pages.k);
  u32x4* const v = static_cast<u32x4*>(kb.pages.v);
  const int32_t* const from = kb.table + (int64_t)b * kb.max_pages;
  const int32_t* const to = a.dst_table + (int64_t)b * a.dst_max_pages;
  const int64_t total = (int64_t)a.keep * units;
  const uint32_t by = (1u << 20) / units + 1;  // x / units = x * by >> 20 for x < 2^11, units up to 2^9
  for (int64_t x0 = (int64_t)part * (kMove * kAtOnce); x0 < total; x0 += (int64_t)parts * (kMove * kAtOnce)) {
    const int i0 = (int)(x0 / units), c0 = (int)(x0 - (int64_t)i0 * units);
    u32x4 xk[kAtOnce], xv[kAtOnce];
    int64_t dst[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const uint32_t x = c0 + u * kMove + threadIdx.x, row = x * by >> 20, c = x - row * units;
      const int i = i0 + (int)row;
      dst[u] = -1;
      if (i >= a.keep) continue;
      const int64_t src = row_at(kb, from, h, kept[i]) * units + c;
      xk[u] = __builtin_nontemporal_load(k + src);
      if (VALUES) xv[u] = __builtin_nontemporal_load(v + src);
      dst[u] = row_at(kb, to, h, i) * units + c;
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      if (dst[u] < 0) continue;
      k[dst[u]] = xk[u];
      if (VALUES) v[dst[u]] = xv[u];
    }
  }
}

// Rows of one side of a new block in a wave's registers: 16 values of a row to a lane.
template <int PASSES>
struct Held {
  codes16 x[PASSES];
  float scale[PASSES];  // 0 for a row that is not there

  __device__ __forceinline__ void load(int p, const void* pool, const float* scales, int64_t row, int64_t at, int shift) {
    x[p] = __builtin_nontemporal_load(reinterpret_cast<const codes16*>(static_cast<const uint8_t*>(pool) + at));
    scale[p] = scales[row >> shift];
  }
  // The largest finite magnitude, as bits; one past fp32's largest counts as that
  // (256 at 2^120 is 2^128, and what an append makes of the largest fp32 values).
  // Among codes: one more than the magnitude's, which orders as the values do and
  // sends NaN (0x7f) to 0; two bytes at a time.
  __device__ __forceinline__ uint32_t top() const {
    typedef __attribute__((ext_vector_type(2))) uint16_t u16x2;
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      u16x2 most = {0, 0};
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const uint32_t y = ((x[p][n] & 0x7f7f7f7fu) + 0x01010101u) & 0x7f7f7f7fu;
        most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, y & 0x00ff00ffu));
        most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, y >> 8 & 0x00ff00ffu));
      }
      const int code = max((int)most[0], (int)most[1]);
      const float value = code ? __builtin_amdgcn_cvt_f32_fp8(code - 1, 0) : 0.f;
      m = max(m, magnitude(scale[p]) <= kLargest ? min(magnitude(value * scale[p]), kLargest) : 0);
    }
    return m;
  }
};

// A wave takes 16 or 32 rows of a new block, keys and values together, so that many
// loads are on their way; W waves to a block, NW to a workgroup.  16 rows leave the
// chip more waves, but waves of a block wait for each other.  Whole calls with 16 and
// 32 rows, into blocks of 32, 64, 128 and 256: 64 sequences of 500 to 8191 tokens to
// 2000 74 and 76 us, 75 and 76, 79 and 76, 97 and 82; 8 of 4000 to 30000 to 3000 43 and
// 44, 43 and 45, 45 and 45, 50 and 48; 256 of 300 to 1200 to 256 99 and 98, 98 and 98,
// 97 and 98, 106 and 98; one of 30000 to 8000 30 to 32 in each.
template <int D, int ROWS, int W>
__global__ void __launch_bounds__(64 * (W > 4 ? W : 4)) move_blocks_kernel(EvictArgs a, int parts) {
  constexpr int NW = W > 4 ? W : 4, BLOCKS = NW / W, SHIFT = __builtin_ctz(ROWS * W);
  constexpr int LPR = D / 16, RPP = kWave / LPR, PASSES = ROWS / RPP;
  __shared__ uint2 lds_max[NW];
  const KvBatch& kb = a.kb;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = threadIdx.x & 63, group = wave % W;
  const int b = blockIdx.x / parts, part = blockIdx.x % parts, h = blockIdx.y;
  if (part == 0 && h == 0) set_length(a, b);
  const int32_t* const kept = a.kept + ((int64_t)b * kb.s.Hkv + h) * a.keep;
  if (kept[0] < 0) return;
  move_weights(a, (int64_t)b * kb.s.Hkv + h, kept, part, parts);
  const int32_t* const from = kb.table + (int64_t)b * kb.max_pages;
  const int32_t* const to = a.dst_table + (int64_t)b * a.dst_max_pages;
  const int blocks = (a.keep + (1 << SHIFT) - 1) >> SHIFT, column = 16 * (lane % LPR);
  for (int at = part * BLOCKS; at < blocks; at += parts * BLOCKS) {
    const int block = at + wave / W, begin = block << SHIFT;
    const int count = block < blocks ? min(a.keep - begin, 1 << SHIFT) : 0;
    const int first = group * ROWS + lane / LPR;  // this lane's rows: every RPP-th from here on
    int64_t src[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) src[p] = first + p * RPP < count ? kept[begin + first + p * RPP] : 0;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) src[p] = row_at(kb, from, h, (int)src[p]);
    Held<PASSES> k, v;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      k.load(p, kb.pages.k, a.scales.k, src[p], src[p] * D + column, SHIFT);
      v.load(p, kb.pages.v, a.scales.v, src[p], src[p] * D + column, SHIFT);
      if (first + p * RPP >= count) k.scale[p] = v.scale[p] = 0.f;
    }
    uint32_t mk = wave_max(k.top()), mv = wave_max(v.top());
    if (W > 1) {
      __syncthreads();
      if (lane == 0) lds_max[wave] = make_uint2(mk, mv);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < W; ++i) mk = max(mk, lds_max[wave - group + i].x), mv = max(mv, lds_max[wave - group + i].y);
    }
    if (count == 0) continue;
    const uint32_t sk = scale_for(mk), sv = scale_for(mv);
    const int64_t dst = row_at(kb, to, h, begin);
    if (group == 0 && lane == 0) {
      a.scales.k[dst >> SHIFT] = __uint_as_float(sk);
      a.scales.v[dst >> SHIFT] = __uint_as_float(sv);
    }
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int i = first + p * RPP;
      if (i >= count) continue;
      const int64_t to_at = (dst + i) * D + column;
      *reinterpret_cast<codes16*>(static_cast<uint8_t*>(kb.pages.k) + to_at) = rescaled(k.x[p], k.scale[p], sk);
      *reinterpret_cast<codes16*>(static_cast<uint8_t*>(kb.pages.v) + to_at) = rescaled(v.x[p], v.scale[p], sv);
    }
  }
}

template <int D, int ROWS, int W>
hipError_t run_blocks(const EvictArgs& a, hipStream_t st) {
  constexpr int NW = W > 4 ? W : 4;
  const int blocks = (a.keep + ROWS * W - 1) / (ROWS * W);
  const int64_t groups = (int64_t)a.kb.s.B * a.kb.s.Hkv;
  int64_t parts = (blocks + NW / W - 1) / (NW / W);
  const int64_t most = (((int64_t)1 << 32) - 1) / (groups * NW * kWave);  // threads of a launch
  if (parts > most) parts = most;
  hipLaunchKernelGGL((move_blocks_kernel<D, ROWS, W>), dim3((unsigned)(a.kb.s.B * parts), a.kb.s.Hkv), dim3(NW * kWave),
                     0, st, a, (int)parts);
  return hipGetLastError();
}
template <int D>
hipError_t by_block(const EvictArgs& a, hipStream_t st) {
  switch (a.scales.shift) {
    case 4: return run_blocks<D, 16, 1>(a, st);
    case 5: return run_blocks<D, 16, 2>(a, st);
    case 6: return run_blocks<D, 16, 4>(a, st);
    case 7: return run_blocks<D, 32, 4>(a, st);
  }
  return run_blocks<D, 32, 8>(a, st);
}

hipError_t run_select(const EvictArgs& a, hipStream_t st) {
  const kda_kv_shape& s = a.kb.s;
  const int64_t longest = (int64_t)a.kb.max_pages << a.kb.page_shift, parts = (longest + kShort - 1) / kShort;
  const dim3 rows((unsigned)(s.B * s.Hkv));
  if (parts >= kFewestParts && rows.x <= kMostRows && parts * rows.x <= kMostParts && Parts::words(parts) <= a.stride) {
    const dim3 grid(rows.x, (unsigned)parts);
    hipLaunchKernelGGL((hist_kernel<0>), grid, dim3(kSelect), 0, st, a, (int)parts);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((hist_kernel<1>), grid, dim3(kSelect), 0, st, a, (int)parts);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL((hist_kernel<2>), grid, dim3(kSelect), 0, st, a, (int)parts);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(places_kernel, grid, dim3(kSelect), 0, st, a, (int)parts);
  } else if (longest > kShort) {
    hipLaunchKernelGGL((select_kernel<true>), rows, dim3(kSelect), 0, st, a);
  } else {
    hipLaunchKernelGGL((select_kernel<false>), rows, dim3(kSelect), 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_evict(const KvBatch& b, const BlockScales& scales, const float* weights, int64_t stride,
                           int32_t keep, int32_t recent, const int32_t* dst_table, int32_t dst_max_pages,
                           int64_t* new_len, float* new_weights, int32_t* kept, hipStream_t st) {
  const EvictArgs a{b, scales, weights, stride, keep, recent, dst_table, dst_max_pages, new_len, new_weights, kept};
  const kda_kv_shape& s = b.s;
  const hipError_t e = run_select(a, st);
  if (e != hipSuccess) return e;
  if (scales.k) return s.dk == 128 ? by_block<128>(a, st) : by_block<64>(a, st);
  const int es = s.cache_dtype == KDA_F32 ? 4 : s.cache_dtype == KDA_BF16 ? 2 : 1;
  const int units = s.dk * es / 16;
  int64_t parts = ((int64_t)keep * units + kAtOnce * kMove - 1) / (kAtOnce * kMove);
  const int64_t most = (((int64_t)1 << 32) - 1) / ((int64_t)s.B * s.Hkv * kMove);
  if (parts > most) parts = most;
  const dim3 grid((unsigned)(s.B * parts), s.Hkv);
  if (b.pages.v)
    hipLaunchKernelGGL((move_kernel<true>), grid, dim3(kMove), 0, st, a, units, (int)parts);
  else
    hipLaunchKernelGGL((move_kernel<false>), grid, dim3(kMove), 0, st, a, units, (int)parts);
  return hipGetLastError();
}

}  // namespace kda
