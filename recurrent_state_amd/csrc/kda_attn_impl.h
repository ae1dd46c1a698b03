// What the two attention kernels over the paged cache share: how the cache is
// split over the chip, how a wave reaches the pages, and how partial results
// are joined.
//
// Split.  The visible tokens of all sequences, cut into tiles, form one list,
// and the grid's workers take equal runs of it, whatever the lengths are: a
// batch of one long and many short sequences keeps every CU busy to the end.
// The runs follow from the positions on the device, so the host needs no
// lengths.  A run may hold whole sequences, whose outputs its worker writes
// itself, and at most two pieces of sequences, which go to the workspace (slot
// 0: a sequence that an earlier worker began, slot 1: one that a later worker
// ends) and are joined, in the workers' order, by a second kernel.
#pragma once

#include "kda_pages.h"

namespace kda {
namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(4))) float f32x4;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

struct AttnArgs {
  KvBatch kb;
  KvRows q;
  float scale;
  int32_t window;
  void* o;
  float* lse;
  int32_t workers;     // runs of the tile list
  int32_t row_blocks;  // blocks of query rows of a (sequence, kv head)
  int32_t rows;        // query rows of a block
  // Workspace: first tile of each sequence [B + 1], then for every piece
  // (worker, slot, kv head, row block) a flag, (max, sum) and output rows.
  int64_t* first_tile;
  int32_t* piece_bad;
  f32x2* piece_ml;
  float* piece_o;
};

__device__ __forceinline__ int64_t piece_index(const AttnArgs& a, int worker, int slot, int hk, int rb) {
  return (((int64_t)worker * 2 + slot) * a.kb.s.Hkv + hk) * a.row_blocks + rb;
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// max over the four 16-lane rows of a wave: every lane gets its column's.
__device__ __forceinline__ float max_over_rows(float x) {
  float a = x, b = x;
  asm volatile("s_nop 1\n\tv_permlane16_swap_b32 %0, %1" : "+v"(a), "+v"(b));
  x = fmaxf(a, b);
  a = x, b = x;
  asm volatile("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(a), "+v"(b));
  return fmaxf(a, b);
}

// A value that every lane holds, moved to scalar registers.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
  const uint32_t lo = (uint32_t)uniform((int)(uint32_t)x), hi = (uint32_t)uniform((int)(x >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// x, as a value that the compiler knows nothing of: what is computed from it
// stays where it is used, instead of being hoisted out of the loops around
// and held in registers (or spilled) for all of them.
__device__ __forceinline__ int here(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// A sequence's part in the call: rows row0 .. row0 + n - 1, its visible tokens
// [lo, end) of all its rows together, and its tiles (of TILE tokens, from the
// one that holds lo).  A sequence whose rows all come before its first token
// has one empty tile, so that a worker writes its rows; one that is refused
// or idle has none.
struct Seq {
  int32_t row0, n;
  int64_t pos;
  int32_t lo, end, tiles;
  int32_t err;
};
template <int TILE>
__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int b) {
  const KvBatch& kb = a.kb;
  const SeqRows sr = seq_rows(kb, b);
  Seq s{sr.row0, sr.n, 0, 0, 0, 0, sr.bad ? KDA_DEV_ERR_TOKENS : 0};
  if (sr.n == 0) return s;
  s.pos = kb.pos[b];
  const int64_t end = s.pos + sr.n;
  if (s.pos > (int64_t)1 << 30 || end > ((int64_t)kb.max_pages << kb.page_shift)) {
    s.err = KDA_DEV_ERR_PAGE;
    return s;
  }
  s.tiles = 1;
  if (end > 0) {
    s.end = (int32_t)end;
    if (a.window > 0 && s.pos + 1 > a.window) s.lo = (int32_t)(s.pos + 1 - a.window);
    s.tiles = (s.end - (s.lo & ~(TILE - 1)) + TILE - 1) / TILE;
  }
  return s;
}

// The same for a sequence that the whole wave works on.
template <int TILE>
__device__ __forceinline__ Seq uniform_seq(const AttnArgs& a, int b) {
  Seq s = seq_of<TILE>(a, b);
  s.row0 = uniform(s.row0);
  s.n = uniform(s.n);
  s.pos = uniform(s.pos);
  s.lo = uniform(s.lo);
  s.end = uniform(s.end);
  s.tiles = uniform(s.tiles);
  return s;
}

// Inclusive sum over the wave's lanes.
__device__ __forceinline__ int64_t wave_scan(int64_t x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const int64_t y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// A worker's run [tile, end) of the tile list and where it begins: in
// sequence b, whose own tiles begin at `first`.
struct Run {
  int64_t tile, end, first;
  int b;
};

// Workers with something to do: no run is empty.
__device__ __forceinline__ int64_t busy_workers(const AttnArgs& a, int64_t total) {
  return total < a.workers ? total : a.workers;
}

// Called by a whole wave.  `record`: this wave also names refused sequences
// and writes the sequences' first tiles for the join.
template <int TILE>
__device__ __forceinline__ Run find_run(const AttnArgs& a, int worker, bool record) {
  const int lane = threadIdx.x & 63, B = a.kb.s.B;
  int64_t total = 0, upto = 0;
  int32_t tiles = 0;
  for (int c = 0; c < B; c += kWave) {
    Seq s{};
    if (c + lane < B) s = seq_of<TILE>(a, c + lane);
    tiles = s.tiles;
    upto = wave_scan(tiles);
    if (record && c + lane < B) {
      a.first_tile[c + lane] = total + upto - tiles;
      if (s.err) set_err(a.kb.dev_err, s.err);
    }
    total += uniform(__shfl(upto, kWave - 1));
  }
  if (record && lane == 0) a.first_tile[B] = total;
  const int64_t w = busy_workers(a, total);
  if (worker >= w) return Run{0, 0, 0, 0};
  Run r{worker * total / w, (worker + 1) * total / w, 0, 0};
  // The chunk that holds r.tile: with up to 64 sequences the one at hand.
  int c = 0;
  int64_t before = 0;
  if (B > kWave) {
    for (; c < B; c += kWave) {
      tiles = c + lane < B ? seq_of<TILE>(a, c + lane).tiles : 0;
      upto = wave_scan(tiles);
      const int64_t sum = uniform(__shfl(upto, kWave - 1));
      if (before + sum > r.tile) break;
      before += sum;
    }
  }
  // The first lane whose tiles reach past r.tile.
  const int at = __ffsll((unsigned long long)__ballot(before + upto > r.tile)) - 1;
  r.b = c + at;
  r.first = before + uniform(__shfl(upto - tiles, at));
  return r;
}

// Where the visible tokens of one sequence are, for a wave that walks them in
// groups of 16 (which no page splits).  Table entries come through the scalar
// cache, and only those of visible tokens are read: a group outside them
// stands for the nearest one inside.  An id outside the pool is noted and
// replaced by page 0.
struct PageWalk {
  const int32_t __attribute__((address_space(4)))* table;
  int lo, hi;  // first and last visible group's first token
  int shift, n_pages;
  int64_t page_rows, head;
  bool bad;

  __device__ __forceinline__ PageWalk(const KvBatch& kb, const Seq& s, int b, int hk)
      : table((const int32_t __attribute__((address_space(4)))*)(kb.table + (int64_t)b * kb.max_pages)),
        lo(s.lo & ~15), hi((s.end - 1) & ~15), shift(kb.page_shift), n_pages(kb.pages.n_pages),
        page_rows((int64_t)kb.s.Hkv << kb.page_shift), head((int64_t)hk << kb.page_shift), bad(false) {}
  __device__ __forceinline__ int32_t entry(int token) const { return table[min(max(token, lo), hi) >> shift]; }
  // First row, in the pool's rows, of the group at `token`, whose page entry is id.
  __device__ __forceinline__ int64_t row(int token, int32_t id) {
    const bool out = id < 0 || id >= n_pages;
    bad |= out;
    return (int64_t)(out ? 0 : id) * page_rows + head + (min(max(token, lo), hi) & ((1 << shift) - 1));
  }
};

// Joins the pieces of the sequences that more than one worker had a part of.
// One workgroup takes `rows_each` query rows of a (sequence, kv head); DV / 4
// lanes hold a row, so several pieces are read at once, and the groups' sums
// meet in LDS.  o = sum_w 2^(m_w - m) o_w / sum_w 2^(m_w - m) l_w.
constexpr int kJoinThreads = 256;

template <int DV>
__device__ __forceinline__ void store4(bf16_t* p, const f32x4& x) {
  const uint32_t lo = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){x[0], x[1]}, bf16x2));
  const uint32_t hi = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){x[2], x[3]}, bf16x2));
  *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
}
template <int DV>
__device__ __forceinline__ void store4(float* p, const f32x4& x) {
  *reinterpret_cast<f32x4*>(p) = x;
}

template <int DV, typename TIn>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttnArgs a, int rows_each) {
  constexpr int LANES = DV / 4, GROUPS = kJoinThreads / LANES;
  __shared__ f32x4 sum_o[GROUPS][LANES];
  __shared__ f32x2 sum_ml[GROUPS];
  const KvBatch& kb = a.kb;
  const int b = blockIdx.x, hk = blockIdx.y;
  const int64_t first = a.first_tile[b], past = a.first_tile[b + 1], total = a.first_tile[kb.s.B];
  if (past == first) return;
  // The worker whose run holds tile x: the last one that begins at or before it.
  const int64_t busy = busy_workers(a, total);
  const int w0 = (int)(((first + 1) * busy - 1) / total);
  const int w1 = (int)((past * busy - 1) / total);
  if (w0 == w1) return;
  const int G = kb.s.Hq / kb.s.Hkv;
  const SeqRows sr = seq_rows(kb, b);
  const int R = sr.n * G;
  const int group = threadIdx.x / LANES, lane = threadIdx.x % LANES;
  const int r0 = blockIdx.z * rows_each, r1 = min(r0 + rows_each, R);
  const float vs = kb.pages.v_scale ? kb.pages.v_scale[hk] : 1.f;
  for (int r = r0; r < r1; ++r) {
    const int rb = r / a.rows, in = r % a.rows;
    float m = -INFINITY, l = 0.f;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    int bad = 0;
    for (int w = w0 + group; w <= w1; w += GROUPS) {
      const int64_t at = piece_index(a, w, w == w0 ? 1 : 0, hk, rb);
      bad |= a.piece_bad[at];
      const f32x2 ml = a.piece_ml[at * a.rows + in];
      const f32x4 x = *reinterpret_cast<const f32x4*>(a.piece_o + (at * a.rows + in) * DV + 4 * lane);
      const float mn = fmaxf(m, ml[0]);
      // A piece without visible tokens has m = -inf and zeros.
      const float f = m == -INFINITY ? 0.f : exp2_(m - mn), g = ml[0] == -INFINITY ? 0.f : exp2_(ml[0] - mn);
      l = l * f + ml[1] * g;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = o[i] * f + x[i] * g;
      m = mn;
    }
    bad = __syncthreads_or(bad);
    if (lane == 0) sum_ml[group] = (f32x2){m, l};
    sum_o[group][lane] = o;
    __syncthreads();
    if (!bad && group == 0) {
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) M = fmaxf(M, sum_ml[g][0]);
      f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        const float f = sum_ml[g][0] == -INFINITY ? 0.f : exp2_(sum_ml[g][0] - M);
        L += sum_ml[g][1] * f;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] += sum_o[g][lane][i] * f;
      }
      const float inv = L == 0.f ? 0.f : vs / L;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] *= inv;
      const int64_t row = (int64_t)(sr.row0 + r / G) * kb.s.Hq + hk * G + r % G;
      store4<DV>(static_cast<TIn*>(a.o) + row * DV + 4 * lane, x);
      if (a.lse && lane == 0) a.lse[row] = (M + __log2f(L)) * kLn2;
    }
    __syncthreads();
  }
}

}  // namespace
}  // namespace kda
