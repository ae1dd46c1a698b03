// What the two attention kernels over the paged cache share: how the cache is
// split over the chip, how a wave reaches the pages, and how partial results
// are joined.
//
// Split.  The visible tokens of each sequence are cut into tiles, and the grid's
// workers share the tiles out by the positions on the device, so that the host
// needs no lengths.
//   many sequences  All tiles form one list, of which every worker takes an
//                   equal run: a batch of long and short sequences keeps every
//                   CU busy to the end.  A run may hold whole sequences, whose
//                   outputs its worker writes itself, and at most two pieces
//                   of others.  Where one more sequence in a run costs its
//                   worker much (queries to load, a piece to write), each
//                   sequence begins with some places of the list that stand
//                   for this and hold no tile.
//   few (up to 64, with `few` workers or more to each)  Every worker takes a
//                   piece of one sequence, of the shortest length with which
//                   the workers suffice: somewhat less even, but a worker
//                   loads queries and writes results once.
// Pieces go to the workspace (slot 0: a sequence that an earlier worker began,
// slot 1: the others) and are joined, in the workers' order, by a second kernel.
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
  int32_t workers;     // runs of the tile list at most
  int32_t run_tiles;   // tiles of a run at least, while there are enough
  int32_t start_tiles; // what a sequence's beginning costs a worker, in tiles
  int32_t few;         // workers to a sequence, from which on each takes one piece
  int32_t row_blocks;  // blocks of query rows of a (sequence, kv head)
  int32_t rows;        // query rows of a block
  // Workspace: each sequence's first and last worker [B], then for every piece
  // (worker, slot, kv head, row block) its rows' (max, sum) and outputs.  A sum
  // below zero refuses the sequence.
  int2* span;
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

// A value that every lane holds, moved to a scalar register.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
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
  const int64_t pos = kb.pos[b];  // asked for together with the token range
  const SeqRows sr = seq_rows(kb, b);
  Seq s{sr.row0, sr.n, pos, 0, 0, 0, sr.bad ? KDA_DEV_ERR_TOKENS : 0};
  if (sr.n == 0) return s;
  const int64_t end = pos + sr.n;
  if (pos > (int64_t)1 << 30 || end > ((int64_t)kb.max_pages << kb.page_shift)) {
    s.err = KDA_DEV_ERR_PAGE;
    return s;
  }
  s.tiles = 1;
  if (end > 0) {
    s.end = (int32_t)end;
    if (a.window > 0 && pos + 1 > a.window) s.lo = (int32_t)(pos + 1 - a.window);
    s.tiles = (s.end - (s.lo & ~(TILE - 1)) + TILE - 1) / TILE;
  }
  return s;
}

// Lane `from`'s sequence, in scalar registers.
__device__ __forceinline__ Seq seq_of_lane(const Seq& x, int from) {
  Seq s;
  s.row0 = __builtin_amdgcn_readlane(x.row0, from);
  s.n = __builtin_amdgcn_readlane(x.n, from);
  s.pos = (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(x.pos >> 32), from) << 32 |
                    (uint32_t)__builtin_amdgcn_readlane((int)x.pos, from));
  s.lo = __builtin_amdgcn_readlane(x.lo, from);
  s.end = __builtin_amdgcn_readlane(x.end, from);
  s.tiles = __builtin_amdgcn_readlane(x.tiles, from);
  s.err = 0;
  return s;
}

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

// How `total` places of the list fall to the workers: `count` of them have a run (none is
// empty), the first `more` of one tile more than the others' `each`.
struct Shares {
  uint32_t count, each, more;

  __device__ __forceinline__ Shares(uint32_t total, uint32_t count_) : count(count_) {
    each = count ? total / count : 0;
    more = total - each * count;
  }
  __device__ __forceinline__ uint32_t begin(uint32_t worker) const { return worker * each + min(worker, more); }
  // The worker that has tile x.
  __device__ __forceinline__ uint32_t of(uint32_t x) const {
    const uint32_t y = more * (each + 1);
    return x < y ? x / (each + 1) : more + (x - y) / each;
  }
};

// A worker's run [tile, end) of the list, and the sequence that it is at: number
// b, whose own tiles begin at `first`.
template <int TILE>
struct Run {
  const AttnArgs& a;
  int32_t tile, end, first;
  int b;
  Seq s;

  // Called by a whole wave.  `record`: this wave also names refused sequences
  // and writes the sequences' workers for the join.
  __device__ __forceinline__ Run(const AttnArgs& args, int worker, bool record)
      : a(args), tile(0), end(0), first(0), b(0), s{} {
    const int lane = threadIdx.x & 63, B = a.kb.s.B;
    Seq lanes{};  // 64 sequences, one to a lane
    int32_t total = 0, upto = 0;
    for (int c = 0; c < B; c += kWave) {
      lanes = c + lane < B ? seq_of<TILE>(a, c + lane) : Seq{};
      upto = wave_scan(places(lanes));
      if (record && lanes.err) set_err(a.kb.dev_err, lanes.err);
      total += __builtin_amdgcn_readlane(upto, kWave - 1);
    }
    if (B <= kWave && a.few * B <= a.workers) {
      one_piece(worker, record, lanes, total);
      return;
    }
    const Shares shares(total, min((total + a.run_tiles - 1) / a.run_tiles, a.workers));
    if (worker < (int)shares.count) {
      tile = shares.begin(worker);
      end = shares.begin(worker + 1);
    }
    // The chunk that holds `tile`: with up to 64 sequences the one at hand.
    int32_t before = 0;
    if (B > kWave) {
      for (; b < B; b += kWave) {
        lanes = b + lane < B ? seq_of<TILE>(a, b + lane) : Seq{};
        upto = wave_scan(places(lanes));
        const int32_t sum = __builtin_amdgcn_readlane(upto, kWave - 1);
        if (record) write_span(shares, b + lane, before + upto, lanes.tiles);
        // The recording wave goes through all of them; its worker is the first.
        if (before + sum > tile && !record) break;
        before += sum;
      }
      if (record) {
        b = before = 0;
        if (tile < end) {  // back to the first sequence with tiles
          for (; b < B; b += kWave) {
            lanes = b + lane < B ? seq_of<TILE>(a, b + lane) : Seq{};
            upto = wave_scan(places(lanes));
            if (__builtin_amdgcn_readlane(upto, kWave - 1) > 0) break;
          }
        }
      }
    } else if (record) {
      write_span(shares, lane, upto, lanes.tiles);
    }
    if (tile >= end) return;
    // The first lane whose tiles reach past `tile`.
    const int at = uniform(__ffsll((unsigned long long)__ballot(before + upto > tile)) - 1);
    b += at;
    first = before + __builtin_amdgcn_readlane(upto - lanes.tiles, at);
    tile = max(tile, first);
    s = seq_of_lane(lanes, at);
  }

  // Pieces of single sequences: see the top of the file.
  __device__ __forceinline__ void one_piece(int worker, bool record, const Seq& lanes, int32_t total) {
    const int lane = threadIdx.x & 63;
    const int busy = __popcll(__ballot(lanes.tiles > 0));
    total -= busy * a.start_tiles;
    // Of n pieces of a sequence the last is half empty on average.
    int32_t each = max(a.run_tiles, (int)((uint32_t)total / (uint32_t)(a.workers - busy / 2)));
    int32_t count, upto;
    for (;; each += max(1, each / 16)) {  // ends: from total / (workers - busy) on there are enough
      count = (lanes.tiles + each - 1) / each;
      upto = wave_scan(count);
      if (__builtin_amdgcn_readlane(upto, kWave - 1) <= a.workers) break;
    }
    if (record && lane < a.kb.s.B) a.span[lane] = make_int2(upto - count, max(upto - 1, upto - count));
    const uint64_t past = __ballot(upto > worker);
    if (past == 0) return;
    b = __ffsll((unsigned long long)past) - 1;
    s = seq_of_lane(lanes, b);
    const Shares shares(s.tiles, __builtin_amdgcn_readlane(count, b));
    const int piece = worker - __builtin_amdgcn_readlane(upto - count, b);
    tile = shares.begin(piece);
    end = shares.begin(piece + 1);
  }

  // A sequence's places in the list: its tiles come last.
  __device__ __forceinline__ int32_t places(const Seq& x) const { return x.tiles > 0 ? x.tiles + a.start_tiles : 0; }

  // Sequence `seq`, whose tiles end before place `upto`.
  __device__ __forceinline__ void write_span(const Shares& shares, int seq, int32_t upto, int32_t tiles) const {
    if (seq < a.kb.s.B)
      a.span[seq] = tiles > 0 ? make_int2(shares.of(upto - tiles), shares.of(upto - 1)) : make_int2(0, 0);
  }

  // Past the sequence's tiles that end at `stop`.
  __device__ __forceinline__ void next(int32_t stop) {
    tile = stop;
    first += s.tiles;
    if (tile >= end) return;
    do {
      if (++b >= a.kb.s.B) {  // only if the positions change under the call
        tile = end;
        return;
      }
      s = seq_of_lane(seq_of<TILE>(a, b), 0);
    } while (s.tiles == 0);
    first += a.start_tiles;
    tile = first;
  }
};

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

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}
__device__ __forceinline__ bf16x8 as_op(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(bf16x8, (u32x4){a, b, c, d});
}
__device__ __forceinline__ f32x4 mfma_bf16(const bf16x8& a, const bf16x8& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ void store4(bf16_t* p, const f32x4& x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
}
__device__ __forceinline__ void store4(float* p, const f32x4& x) { *reinterpret_cast<f32x4*>(p) = x; }
__device__ __forceinline__ void store8(bf16_t* p, const float (&x)[8]) {
  *reinterpret_cast<u32x4*>(p) =
      (u32x4){pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7])};
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  store4(p, (f32x4){x[0], x[1], x[2], x[3]});
  store4(p + 4, (f32x4){x[4], x[5], x[6], x[7]});
}

// Joins the pieces of the sequences that more than one worker had a part of:
// with m the largest of the pieces' maxima,
//   o = sum_w 2^(m_w - m) o_w / sum_w 2^(m_w - m) l_w.
// DV / 4 lanes hold a row of outputs, and a workgroup has several such groups.
// `split` of them (a power of two) share a row, each with every split-th
// piece, so that a long sequence's many pieces are read side by side, and a
// batch's few pieces of many rows are too; a workgroup takes `rows_each` query
// rows of a (sequence, kv head).  Every wave finds m and the sum by itself, a
// piece to a lane.  What bounds it is the pieces' way back from the caches and,
// for few of them, three dependent loads: 65 MB of latent pieces (64 sequences,
// 128 rows) take 16 us, the one or two of a row of one short sequence 3 us.
template <int DV>
constexpr int kJoinFirst = DV == 512 ? 6 : 4;  // pieces of a row that a group asks for at once
template <int DV>
constexpr int kJoinGroups = DV == 512 ? 8 : 16;  // of a workgroup, at most

template <int DV, typename TIn>
__global__ void __launch_bounds__(DV / 4 * kJoinGroups<DV>) join_kernel(AttnArgs a, int rows_each, int split) {
  constexpr int LANES = DV / 4;
  __shared__ f32x4 part[kJoinGroups<DV>][LANES];
  const KvBatch& kb = a.kb;
  const int b = blockIdx.x, hk = blockIdx.y;
  const int w0 = a.span[b].x, w1 = a.span[b].y;
  if (w0 == w1) return;
  const int G = kb.s.Hq / kb.s.Hkv;
  const int64_t pos = kb.pos[b];
  const SeqRows sr = seq_rows(kb, b);
  constexpr int SAME = LANES < kWave ? LANES : kWave;  // lanes of a wave that hold one row
  const int group = threadIdx.x / LANES, lane = threadIdx.x % LANES, same = threadIdx.x % SAME;
  const int share = group & (split - 1), rows_at_once = blockDim.x / LANES / split;
  const int r0 = blockIdx.z * rows_each, r1 = min(r0 + rows_each, sr.n * G);
  if (r0 >= r1) return;
  const float vs = kb.pages.v_scale ? kb.pages.v_scale[hk] : 1.f;
  // Piece d of the sequence is worker w0 + d's: rows from the first worker's
  // first slot on (a workspace is far below 2^32 bytes).
  const int pieces = w1 - w0 + 1;
  const uint32_t slot = (uint32_t)kb.s.Hkv * a.row_blocks * a.rows;
  const char* outs = reinterpret_cast<const char*>(a.piece_o + (int64_t)w0 * 2 * slot * DV);
  const char* stats = reinterpret_cast<const char*>(a.piece_ml + (int64_t)w0 * 2 * slot);
  for (int rr = r0; rr < r1; rr += rows_at_once) {
    const bool live = rr + group / split < r1;
    const int r = live ? rr + group / split : r0;
    const uint32_t at = ((uint32_t)hk * a.row_blocks + r / a.rows) * a.rows + r % a.rows;
    const auto row_of = [&](int d) { return (d == 0 ? slot : 2u * d * slot) + at; };
    const auto out = [&](int d) {
      return *reinterpret_cast<const f32x4*>(outs + (row_of(d) * (uint32_t)(DV * 4) + 16u * lane));
    };
    const auto stat = [&](int d) { return *reinterpret_cast<const f32x2*>(stats + row_of(d) * 8u); };
    // The first pieces' outputs are asked for before their weights are known.
    constexpr int FIRST = kJoinFirst<DV>;
    f32x4 x[FIRST];
    float xm[FIRST];
#pragma unroll
    for (int j = 0; j < FIRST; ++j) {
      const int d = share + j * split;
      x[j] = f32x4{}, xm[j] = -INFINITY;
      if (d < pieces) x[j] = out(d), xm[j] = stat(d)[0];
    }
    const f32x2 none = {-INFINITY, 0.f};
    const f32x2 ml = same < pieces ? stat(same) : none;
    float m = ml[0];
    int refused = ml[1] < 0.f;
    for (int d = same + SAME; d < pieces; d += SAME) {
      const f32x2 y = stat(d);
      m = fmaxf(m, y[0]);
      refused |= y[1] < 0.f;
    }
    // Every row of the sequence comes out the same, so the workgroup agrees.
    if (__ballot(refused) != 0) return;
#pragma unroll
    for (int i = 1; i < SAME; i *= 2) m = fmaxf(m, __shfl_xor(m, i));
    // A piece in which the row sees no token has m = -inf and zeros.
    const float top = m == -INFINITY ? 0.f : m;
    float l = ml[1] * exp2_(ml[0] - top);
    for (int d = same + SAME; d < pieces; d += SAME) {
      const f32x2 y = stat(d);
      l += y[1] * exp2_(y[0] - top);
    }
#pragma unroll
    for (int i = 1; i < SAME; i *= 2) l += __shfl_xor(l, i);
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < FIRST; ++j) {
      const float f = exp2_(xm[j] - top);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] += x[j][i] * f;
    }
#pragma unroll 4
    for (int d = share + FIRST * split; d < pieces; d += split) {
      const float f = exp2_(stat(d)[0] - top);
      const f32x4 y = out(d);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] += y[i] * f;
    }
    if (split > 1) {
      part[group][lane] = o;
      __syncthreads();
      for (int g = 1; g < split; ++g) {
        const f32x4 x = part[group - share + (share + g & (split - 1))][lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] += x[i];
      }
      __syncthreads();
    }
    if (live && share == 0) {
      const float inv = pos + r / G < 0 ? 0.f : vs / l;  // 0 / 0 where every score is -inf
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] *= inv;
      const int64_t row = (int64_t)(sr.row0 + r / G) * kb.s.Hq + hk * G + r % G;
      store4(static_cast<TIn*>(a.o) + row * DV + 4 * lane, o);
      if (a.lse && lane == 0) a.lse[row] = (m + __log2f(l)) * kLn2;
    }
  }
}

// Whether the pool is larger than the 256 MB that the memory side caches.  (How
// much of it a call reads is known on the device only: a short window in a large
// pool counts as the pool.)
inline bool outgrows_cache(const KvBatch& kb) {
  const int64_t es = kb.s.cache_dtype == KDA_F32 ? 4 : kb.s.cache_dtype == KDA_BF16 ? 2 : 1;
  const int64_t row = kb.pages.v ? kb.s.dk + kb.s.dv : kb.s.dk;
  return ((int64_t)kb.pages.n_pages * kb.s.Hkv << kb.page_shift) * row * es > (int64_t)256 << 20;
}

// How a call is split: see split_of() of each kernel.
struct Split {
  int tile, rows, row_blocks, workers, run_tiles, start_tiles, few;
};

// Workers for `wgs` workgroups on the chip at once: at most one to a shortest
// run of the longest possible cache.
inline int workers_of(const kda_kv_shape& s, int64_t wgs, const Split& d, int32_t page_size, int32_t max_pages) {
  int64_t w = wgs / ((int64_t)s.Hkv * d.row_blocks);
  const int64_t run = (int64_t)d.tile * d.run_tiles;
  const int64_t most = (int64_t)s.B * (((int64_t)max_pages * page_size + run - 1) / run + 1);
  if (w > most) w = most;
  return w < 1 ? 1 : (int)w;
}

struct Workspace {
  size_t ml, o, total;
};
inline Workspace workspace_of(const kda_kv_shape& s, const Split& d) {
  const size_t pieces = (size_t)d.workers * 2 * s.Hkv * d.row_blocks;
  Workspace L;
  L.ml = round_up((size_t)s.B * 8, 256);
  L.o = round_up(L.ml + pieces * d.rows * 8, 256);
  L.total = round_up(L.o + pieces * d.rows * s.dv * 4, 256);
  return L;
}

inline AttnArgs make_args(const KvBatch& b, KvRows q, float scale, int32_t window, void* o, float* lse,
                          void* workspace, const Split& d) {
  const Workspace L = workspace_of(b.s, d);
  char* ws = static_cast<char*>(workspace);
  return AttnArgs{b,         q,
                  scale,     window,
                  o,         lse,
                  d.workers, d.run_tiles, d.start_tiles, d.few, d.row_blocks,
                  d.rows,    reinterpret_cast<int2*>(ws),
                  reinterpret_cast<f32x2*>(ws + L.ml), reinterpret_cast<float*>(ws + L.o)};
}

// The join after an attention kernel.  A sequence has about workers / B pieces
// (the lengths are not known here): enough groups share a row to ask for all of
// them at once, and a workgroup takes rows enough that about 2048 of them cover
// all.
template <int DV, typename TIn>
hipError_t run_join(const AttnArgs& a, hipStream_t st) {
  if (a.workers == 1) return hipSuccess;
  const kda_kv_shape& s = a.kb.s;
  const int rows = s.T * (s.Hq / s.Hkv);
  int split = 1;
  while (split < kJoinGroups<DV> && a.workers > (int64_t)split * kJoinFirst<DV> * s.B) split *= 2;
  const int groups = split > 1024 / DV ? split : 1024 / DV;  // 256 threads or more
  const int at_once = groups / split;
  int64_t each = ((int64_t)s.B * s.Hkv * rows + 2047) / 2048;
  each = (each + at_once - 1) / at_once * at_once;
  hipLaunchKernelGGL((join_kernel<DV, TIn>), dim3(s.B, s.Hkv, (unsigned)((rows + each - 1) / each)),
                     dim3(DV / 4 * groups), 0, st, a, (int)each, split);
  return hipGetLastError();
}

}  // namespace
}  // namespace kda
