// Appending to e4m3 pages whose scales go by blocks of tokens.
//
// A block's new scale needs the largest of all its new values before the first
// is stored, so the work is cut along the blocks: a workgroup takes a block's
// new tokens ("item") for one head of keys, values or queries ("kind"; queries
// are only rotated), or for several where few tokens make few rows.  A group of
// W waves holds 16 W rows of a head in registers, 16 values to a lane, laid out
// as in kda_pages.hip; the maximum is exchanged by lane swaps and, for W > 1,
// through the LDS.
//
// The host knows neither lengths nor positions: the grid has an item for every
// block that well-formed ranges can touch, each finds its sequence by a scan of
// the sequences' block counts, 64 at a time, and those past the last end there.

#include "kda_append_impl.h"
#include "kda_blocks.h"

namespace kda {
namespace {

struct BlocksArgs {
  KvBatch kb;
  BlockScales scales;
  KvRows k, v, q;
  void* q_out;
  int64_t q_out_stride;
  kda_rotation rot;
  int32_t kinds;  // kv heads of keys, then of values, then query heads
  Axes axes;
};

// The new tokens of a sequence that have places: row0 + i at place pos + i for
// places [first, end), and the blocks that these touch.
struct Places {
  int32_t row0;
  int64_t pos;
  int32_t first, end, blocks;
  int32_t err;
};
__device__ __forceinline__ Places places_of(const BlocksArgs& a, int b) {
  const KvBatch& kb = a.kb;
  const int64_t pos = kb.pos[b];  // asked for together with the token range
  const SeqRows sr = seq_rows(kb, b);
  Places s{sr.row0, pos, 0, 0, 0, sr.bad ? KDA_DEV_ERR_TOKENS : 0};
  if (sr.n == 0) return s;
  // Outside of +-2^30 no token of the sequence has a place.
  const int64_t p = min(max(pos, -((int64_t)1 << 31)), (int64_t)1 << 31), past = p + sr.n;
  int64_t end = past;
  if (a.rot.cos_sin && !a.axes.n) end = min(end, max((int64_t)a.rot.max_pos, p));
  if (p < 0 || end < past) s.err |= KDA_DEV_ERR_POS;
  const int64_t limit = (int64_t)kb.max_pages << kb.page_shift;
  if (end > limit && end > p) s.err |= KDA_DEV_ERR_PAGE;
  end = min(end, limit);
  s.first = (int32_t)min(max(p, (int64_t)0), limit);
  if (end <= s.first) return s;
  s.end = (int32_t)end;
  s.blocks = ((s.end - 1) >> a.scales.shift) - (s.first >> a.scales.shift) + 1;
  return s;
}

// One block's part of a sequence: places [lo, hi), whose block begins at `begin`;
// token row row0 + i is at place begin + i (row0 itself may be none).
struct Item {
  int b;
  int32_t row0, lo, hi, begin;
  int32_t total;  // of all items, where the scan came to the last; else INT32_MAX
};
// Called by a whole wave; false: there is no item `item`.
__device__ __forceinline__ bool find_item(const BlocksArgs& a, int item, Item& it) {
  const int lane = threadIdx.x & 63, B = a.kb.s.B;
  int before = 0;
#pragma unroll 1
  for (int c = 0; c < B; c += kWave) {
    const Places s = c + lane < B ? places_of(a, c + lane) : Places{};
    const int upto = wave_scan(s.blocks), sum = __builtin_amdgcn_readlane(upto, kWave - 1);
    if (before + sum > item) {
      const int at = __ffsll((unsigned long long)__ballot(before + upto > item)) - 1;
      const int nth = item - before - __builtin_amdgcn_readlane(upto - s.blocks, at);
      const int first = __builtin_amdgcn_readlane(s.first, at), end = __builtin_amdgcn_readlane(s.end, at);
      it.b = c + at;
      it.begin = ((first >> a.scales.shift) + nth) << a.scales.shift;
      it.row0 = it.begin + __builtin_amdgcn_readlane((int32_t)((uint32_t)s.row0 - (uint32_t)s.pos), at);
      it.lo = max(first, it.begin);
      it.hi = min(end, it.begin + (1 << a.scales.shift));
      it.total = c + kWave < B ? INT32_MAX : before + sum;
      return true;
    }
    before += sum;
  }
  return false;
}

// 16 values of a row of bf16 as loaded.
struct Raw16 {
  u32x4 lo, hi;
};

// W waves to a (block, kind); NW waves to a workgroup, which takes every
// gridDim.y-th set of kinds of its item.  The angles of the item's rows stay in
// registers, and the next kind's values are asked for before this one's are used
// (each kind's angles read anew and no loads ahead: 484 us for 300, see below).
// Large calls are bound by memory: 8 prompts of 8192 tokens, 8 kv heads and 32 query
// heads of 128, 1.48 GB, 300 us (4.9 TB/s; a copy of 768 MiB 5.3) into blocks of 64.
// Into blocks of 16, 32, 128 and 256 they take 260, 294, 313 and 374 us; with positions
// on three axes, by sections and dealt to the pairs, blocks of 64 take 359 and 359, of
// 256 414 and 694: there every head's angles are read anew.  Small calls are bound by
// the chain of loads: lengths, page, old scale, codes.
template <int D, int W, bool NT, bool AXES>
__global__ void __launch_bounds__(64 * (W > 4 ? W : 4)) append_blocks_kernel(BlocksArgs a) {
  constexpr int NW = W > 4 ? W : 4, SETS = NW / W;
  constexpr int LPR = D / 16, RPP = kWave / LPR, PASSES = 16 / RPP;  // lanes to a row, rows of a wave's pass
  constexpr bool KEEP = W < 16 || D == 64;  // 1024 threads have no registers for angles and loads ahead
  __shared__ uint32_t lds_max[2][NW];
  const KvBatch& kb = a.kb;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int part = wave % W, set = wave / W, w = lane % LPR;
  const int n_rot = a.rot.cos_sin ? a.rot.dim >> 4 : 0;
  const bool rotates = w < n_rot;
  const Chunks c = chunks_of(a.rot, n_rot, w);
  const bool names = blockIdx.y == 0 && set == 0;  // of the waves of an item's rows, those that name errors

  if (names && wave == 0 && blockIdx.x == 0)
    for (int b = lane; b < kb.s.B; b += kWave) {
      const int err = places_of(a, b).err;
      if (err) set_err(kb.dev_err, err);
    }
  // The grid covers all items but where ranges overlap; where the count of items
  // is known, no scan says so (KEEP or not: the count takes registers too).
  Item it;
  it.total = INT32_MAX;
  for (int item = blockIdx.x; (!KEEP || item < it.total) && find_item(a, item, it); item += gridDim.x) {
    const int32_t page = kb.table[(int64_t)it.b * kb.max_pages + (it.begin >> kb.page_shift)];
    // The lane's rows: token row, and place counted from the block's first.
    int32_t row[PASSES], slot[PASSES];
    bool live[PASSES];
    float cc[KEEP ? PASSES : 1][8], ss[KEEP ? PASSES : 1][8];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int p = it.lo + part * 16 + i * RPP + lane / LPR;
      live[i] = p < it.hi;  // others stand for the first row, and are not stored
      slot[i] = (live[i] ? p : it.lo) - it.begin;
      row[i] = it.row0 + slot[i];
    }
    auto fetch = [&](int kind, Raw16 (&x)[PASSES]) __attribute__((always_inline)) {
      if (kind >= a.kinds) return;
      const bool is_key = kind < kb.s.Hkv, is_value = !is_key && kind < 2 * kb.s.Hkv;
      const int h = is_key ? kind : is_value ? kind - kb.s.Hkv : kind - 2 * kb.s.Hkv;
      const void* const base = is_key ? a.k.p : is_value ? a.v.p : a.q.p;
      const int64_t stride = is_key ? a.k.stride : is_value ? a.v.stride : a.q.stride;
      const bf16_t* const src = static_cast<const bf16_t*>(base) + h * D;
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const bf16_t* const at = src + here(row[i]) * stride;
        x[i].lo = get<NT>(reinterpret_cast<const u32x4*>(at + c.c0));
        x[i].hi = get<NT>(reinterpret_cast<const u32x4*>(at + c.c1));
      }
    };
    int kind = blockIdx.y * SETS + set;
    Raw16 next[PASSES] = {};
    if (KEEP) fetch(kind, next);
    // Of a token that is skipped for its position, some angles.
    auto turns = [&](int i, float (&c)[8], float (&s)[8]) __attribute__((always_inline)) {
      if constexpr (AXES) {
        AxisPos at = axis_positions(a.axes, a.rot, here(row[i]));
        if (at.bad) at.p0 = at.p1 = at.p2 = at.p3 = 0;
        angles(a.rot, at, axes_of_unit<BlocksArgs>(w), w, c, s);
      } else {
        angles(a.rot, it.begin + here(slot[i]), w, c, s);
      }
    };
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      if (AXES && axis_positions(a.axes, a.rot, row[i]).bad) {
        if (names && w == 0) set_err(kb.dev_err, KDA_DEV_ERR_POS);
        live[i] = false;
      }
      if (KEEP && rotates) turns(i, cc[i], ss[i]);
    }
    const bool bad = page < 0 || page >= kb.pages.n_pages;
    if (bad && names && wave == 0 && lane == 0) set_err(kb.dev_err, KDA_DEV_ERR_PAGE);
    if (bad) continue;  // the whole workgroup agrees
    const int in_page = it.begin & (kb.pages.page_size - 1);

#pragma unroll 1
    for (int turn = 0; kind - set < a.kinds; ++turn, kind += gridDim.y * SETS) {
      const bool is_key = kind < kb.s.Hkv, is_value = !is_key && kind < 2 * kb.s.Hkv;
      const int h = is_key ? kind : is_value ? kind - kb.s.Hkv : kind - 2 * kb.s.Hkv;
      const bool stored = is_key || is_value;
      const int64_t head = (int64_t)page * kb.s.Hkv + h;
      float* const scale = (is_key ? a.scales.k : a.scales.v) + (head << (kb.page_shift - a.scales.shift)) +
                           (in_page >> a.scales.shift);
      uint8_t* const dst =
          static_cast<uint8_t*>(is_key ? kb.pages.k : kb.pages.v) + ((head << kb.page_shift) + in_page) * D;
      const bool joins = stored && it.lo > it.begin;
      const float old = joins ? *scale : 0.f;
      Raw16 now[PASSES];
      if (!KEEP) fetch(kind, next);
#pragma unroll
      for (int i = 0; i < PASSES; ++i) now[i] = next[i];
      if (KEEP) fetch(kind + gridDim.y * SETS, next);
      // The lane's values of pass i, rotated: made twice, for the maximum and to
      // be stored, as keeping them takes twice the registers.
      float x[8], y[8];
      auto make = [&](int i) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const uint32_t lo = here(now[i].lo[n]), hi = here(now[i].hi[n]);
          x[2 * n] = bf16_lo(lo), x[2 * n + 1] = bf16_hi(lo);
          y[2 * n] = bf16_lo(hi), y[2 * n + 1] = bf16_hi(hi);
        }
        if (rotates && !is_value) {
          if constexpr (!KEEP) turns(i, cc[0], ss[0]);
          rotate(x, y, cc[KEEP ? i : 0], ss[KEEP ? i : 0], a.rot.pairs);
        }
      };
      uint32_t s = 0;
      bool odd = false;  // some value of the lane's is not finite
      // Sets of one workgroup may be at keys, values and queries: those of the
      // first one come first.
      if (kind - set < 2 * kb.s.Hkv) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
          uint32_t top = 0;
          make(i);
#pragma unroll
          for (int n = 0; n < 8; ++n) top = max(top, max(magnitude(x[n]), magnitude(y[n])));
          if (top > kLargest) {
            odd = true;
            top = 0;
#pragma unroll
            for (int n = 0; n < 8; ++n) top = max(top, max(finite_bits(x[n]), finite_bits(y[n])));
          }
          m = max(m, live[i] ? top : 0);
        }
        m = wave_max(m);
        if (W > 1) {
          if (lane == 0) lds_max[turn & 1][wave] = m;
          __syncthreads();
#pragma unroll
          for (int i = 0; i < W; ++i) m = max(m, lds_max[turn & 1][wave - part + i]);
        }
        s = scale_for(m);
        if (joins) {
          s = max(s, power_of_two(old));
          if (s != __float_as_uint(old)) {
            const float f = old * inverse(s);  // at most 1, but for a scale past 2^120
#pragma unroll 1
            for (int r = part * RPP + lane / LPR; r < it.lo - it.begin; r += W * RPP) {
              codes16* const at = reinterpret_cast<codes16*>(dst + r * D + 16 * w);
              *at = times<true>(*at, f);
            }
          }
        }
        if (stored && part == 0 && lane == 0) *scale = __uint_as_float(s);
      }
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        make(i);
        if (stored) {
          const float inv = inverse(s);
#pragma unroll
          for (int n = 0; n < 8; ++n) x[n] *= inv, y[n] *= inv;
          if (odd) {  // the others are at most 448
#pragma unroll
            for (int n = 0; n < 8; ++n) x[n] = to_range(x[n]), y[n] = to_range(y[n]);
          }
          uint8_t* const to = dst + here(slot[i]) * D;
          if (live[i]) {
            put<NT>(reinterpret_cast<u32x2*>(to + c.c0), e4m3_of(x));
            put<NT>(reinterpret_cast<u32x2*>(to + c.c1), e4m3_of(y));
          }
        } else if (kind < a.kinds) {
          bf16_t* const to = static_cast<bf16_t*>(a.q_out) + here(row[i]) * a.q_out_stride + h * D;
          if (live[i]) {
            store8<NT>(to + c.c0, x);
            store8<NT>(to + c.c1, y);
          }
        }
      }
    }
    if (W > 1) __syncthreads();  // the last maxima have been read
  }
}

template <int D, int W, bool NT>
hipError_t run(const BlocksArgs& a, hipStream_t st) {
  constexpr int NW = W > 4 ? W : 4, SETS = NW / W;
  const int64_t N = a.kb.n_tokens, B = a.kb.s.B;
  int64_t items = (N >> a.scales.shift) + 2 * B;
  if (items > N) items = N;
  // Workgroups to an item: as many as it has sets of kinds, or fewer where the
  // items alone make 2048 workgroups.
  const int64_t sets = (a.kinds + SETS - 1) / SETS;
  int64_t y = 2048 / items;
  y = y < 1 ? 1 : y > sets ? sets : y;
  const int64_t most = (((int64_t)1 << 32) - 1) / (y * NW * kWave);  // threads of a launch
  if (items > most) items = most;
  const dim3 grid((unsigned)items, (unsigned)y), block(NW * kWave);
  if (a.axes.n)
    hipLaunchKernelGGL((append_blocks_kernel<D, W, NT, true>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((append_blocks_kernel<D, W, NT, false>), grid, block, 0, st, a);
  return hipGetLastError();
}

template <int D, bool NT>
hipError_t by_rows(const BlocksArgs& a, hipStream_t st) {
  // Waves enough for the rows that a call can bring to a block.
  const int block = 1 << a.scales.shift, rows = a.kb.s.T < block ? a.kb.s.T : block;
  if (rows <= 16) return run<D, 1, NT>(a, st);
  if (rows <= 32) return run<D, 2, NT>(a, st);
  if (rows <= 64) return run<D, 4, NT>(a, st);
  if (rows <= 128) return run<D, 8, NT>(a, st);
  return run<D, 16, NT>(a, st);
}

}  // namespace

hipError_t launch_kv_append_blocks(const KvBatch& b, const BlockScales& scales, KvRows k, KvRows v, KvRows q,
                                   void* q_out, int64_t q_out_stride, const kda_rotation& rot, const Axes& axes,
                                   hipStream_t st) {
  const BlocksArgs a{b, scales, k, v, q, q_out, q_out_stride, rot, 2 * b.s.Hkv + (q.p ? b.s.Hq : 0), axes};
  // Calls that touch more than the 256 MB Infinity Cache go past it, as the plain
  // append's do: 8 prompts of 8192 tokens 300 us for 316, 64 sequences of 4 tokens 7.9
  // either way.
  const int64_t bytes = append_blocks_bytes(b.n_tokens, b.s, q.p != nullptr);
  const bool large = bytes > (int64_t)256 << 20;
  if (b.s.dk == 128) return large ? by_rows<128, true>(a, st) : by_rows<128, false>(a, st);
  return large ? by_rows<64, true>(a, st) : by_rows<64, false>(a, st);
}

}  // namespace kda
