// The attention weights that cached tokens get, summed over the query rows of a
// call and the query heads of a kv head.
//
// The weight e^(s - lse) of a row and a token needs the row's lse, so the keys
// are read a second time after the attention, without the values.  A workgroup
// takes a run of tiles (kda_attn_impl.h) of one kv head, and keys go from memory
// into the registers of the matrix instructions, as in kda_attn.hip.  Here
// S = Q K^T leaves the MFMA with a token to each lane column, so the sum over a
// tile's 16 rows is one over registers and two lane swaps: no pieces, no atomics,
// one order.
//
//   few rows (up to 32)  Each wave takes a quarter of every tile and all rows, whose
//                        queries and lse stay in its registers: bound by the read
//                        of the keys, and no wave waits for another.  A decode step
//                        of 64 sequences of 60 to 8191 tokens, 8 kv heads of 128 in
//                        bf16, 230 MB: 49 us (4.7 TB/s); e4m3 30, with scales by blocks
//                        29, f32 96.
//   more                 Each wave takes a quarter of the rows, 16 or 32 at a time,
//                        and every tile: bound by the vector instructions (25 us of
//                        issue at 2.4 GHz, 8 of them exponentials; the matrix cores'
//                        work is 7).  The keys come through the LDS, and the waves'
//                        sums meet there, every kRing tiles.  The last 32 tokens of
//                        four prompts of 7001 to 30000, 8 kv heads of 128 in e4m3 with
//                        128 rows each: 34 us (0.51 PFLOP/s, 74 MB), 38 for the first
//                        hundred calls, until the clock has risen; bf16 39, f32 162.
//
// Rounding: all in fp32.  lse times log2 e is rounded once for a row, which moves its
// weights by as much as half a step of lse itself does, and the exponential is the
// hardware's.  Those prompts' sums are 5.4e-8 of their size from those in 64 bits, and
// 4.1e-8 where elementary fp32 operations make them.

#include <type_traits>

#include "kda_attn_cache.h"

namespace kda {
namespace {

constexpr int kWaves = 4;

struct WeightsArgs {
  AttnArgs a;
  const float* lse;
  float* weights;
  int64_t stride;  // of a (sequence, kv head)
};

// Rows r0 .. r0 + 16 NQ - 1 of a sequence's R: queries by lane column, lse and the
// last visible token by register.  A row that is not there has the first one's
// query, an lse that makes its weights 0, and sees no token.
template <int D, typename TIn, typename C, int NQ>
struct Rows {
  typename C::Query q[NQ];
  f32x4 lse[NQ];
  int vis[NQ][4];

  __device__ __forceinline__ void load(const WeightsArgs& w, const Seq& s, int hk, int r0, int R) {
    const KvBatch& kb = w.a.kb;
    const int lane = threadIdx.x & 63, G = kb.s.Hq / kb.s.Hkv;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int rq = r0 + 16 * n + (lane & 15), r = rq < R ? rq : r0, tq = r / G;
      C::load_query(q[n], static_cast<const TIn*>(w.a.q.p) + (int64_t)(s.row0 + tq) * w.a.q.stride +
                              (hk * G + r - tq * G) * D, true);
    }
    // All are asked for at once: a branch around each would wait for it.
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int r4 = r0 + 16 * n + 4 * (lane >> 4), rl = r4 < R ? r4 : r0;
      int t = rl / G, h = rl - t * G;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lse[n][i] = w.lse[(int64_t)(s.row0 + t) * kb.s.Hq + hk * G + h];
        vis[n][i] = r4 + i < R ? (int)max(s.pos + t, (int64_t)-1) : -1;
        const bool next = rl + i + 1 < R;  // else the same row again
        h += next ? 1 : 0;
        if (h == G) h = 0, ++t;
      }
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        lse[n][i] = r0 + 16 * n + 4 * (lane >> 4) + i < R ? lse[n][i] * kLog2e : INFINITY;
  }

  // A tile's sums over these rows, for the token of the lane's column in each
  // group of 16: the scores, and from them the weights, t0 the first token.
  // PART: some row does not see some token.
  typedef f32x4 Scores[C::GROUPS][NQ];
  __device__ __forceinline__ void score(const typename C::Keys& keys, Scores& c) const {
    // The products of one contraction step together: a product does not wait for the one before it.
#pragma unroll
    for (int s = 0; s < C::Keys::STEPS; ++s)
#pragma unroll
      for (int u = 0; u < C::GROUPS; ++u)
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          if (s == 0) c[u][n] = f32x4{};
          keys.add(u, s, q[n], c[u][n]);
        }
  }
  template <bool PART>
  __device__ __forceinline__ void weigh(const Scores& c, const float (&scale)[C::GROUPS], int t0, int window,
                                        float (&sum)[C::GROUPS]) const {
#pragma unroll
    for (int u = 0; u < C::GROUPS; ++u) {
      const int j = t0 + 16 * u + (threadIdx.x & 15);
      // Four sums: no exponential waits for the one before it to be added.
      float x[4] = {};
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = exp2_(__builtin_fmaf(c[u][n][i], scale[u], -lse[n][i]));
          const bool hidden = PART && (j > vis[n][i] || (window > 0 && j <= vis[n][i] - window));
          x[i] += hidden ? 0.f : e;
        }
      sum[u] = pair_sum32(pair_sum16((x[0] + x[1]) + (x[2] + x[3])));
    }
  }
};

// The keys of a tile in flight and the scales of their blocks; the page entries of
// the one after, `step` tokens on.
template <int D, typename TC, bool NT, bool BLK>
struct Keys {
  typedef Cache<D, TC, NT> C;
  C cache;
  int32_t id[C::GROUPS];
  float block[C::GROUPS];

  __device__ __forceinline__ void begin(const PageWalk& walk, int token) {
#pragma unroll
    for (int u = 0; u < C::GROUPS; ++u) id[u] = walk.entry(token + 16 * u);
  }
  __device__ __forceinline__ void load(const AttnArgs& a, PageWalk& walk, int token, int step) {
#pragma unroll
    for (int u = 0; u < C::GROUPS; ++u) {
      const int64_t at = walk.row(token + 16 * u, id[u]);
      cache.load_k(u, static_cast<const TC*>(a.kb.pages.k) + at * D);
      if constexpr (BLK) block[u] = block_scale(a.scales.k, a.scales.shift, at);
      id[u] = walk.entry(token + step + 16 * u);
    }
  }
  __device__ __forceinline__ void scales(float x_scale, float (&x)[C::GROUPS]) const {
#pragma unroll
    for (int u = 0; u < C::GROUPS; ++u) x[u] = BLK ? x_scale * block[u] : x_scale;
  }
};

template <typename TC, bool BLK>
__device__ __forceinline__ float x_scale_of(const AttnArgs& a, int hk) {
  const float x = a.scale * kLog2e;
  return sizeof(TC) == 1 && !BLK ? x * a.kb.pages.k_scale[hk] : x;
}

// Few rows: NQ blocks of 16.
template <int D, typename TIn, typename TC, int NQ, bool NT, bool BLK>
__global__ void __launch_bounds__(kWaves * kWave, NQ == 1 ? 3 : 2) tokens_kernel(WeightsArgs w) {
  typedef Cache<D, TC, NT> C;
  constexpr int SUB = C::SUB, GROUPS = C::GROUPS, TILE = kWaves * SUB;
  const AttnArgs& a = w.a;
  const KvBatch& kb = a.kb;
  const int wave = uniform((int)threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 4;
  const int hk = blockIdx.y, worker = blockIdx.x;
  Run<TILE, false> run(a, worker, worker == 0 && hk == 0 && wave == 0);
  const float x_scale = x_scale_of<TC, BLK>(a, hk);
  // Lane group u holds the sums of tokens 16 u + (lane & 15) of a tile.
  const int group = min(g, GROUPS - 1), mine = 16 * group + (lane & 15);

  while (run.tile < run.end) {
    const Seq& s = run.s;
    const int32_t stop = min(run.end, run.first + s.tiles);
    Rows<D, TIn, C, NQ> rows;
    rows.load(w, s, hk, 0, s.n * (kb.s.Hq / kb.s.Hkv));
    const int base = (s.lo & ~(TILE - 1)) + wave * SUB;
    const int past = min(s.end, base - wave * SUB + (stop - run.first) * TILE);
    const int all_lo = a.window > 0 ? max((int)(s.pos + s.n) - a.window, 0) : 0;
    float* const out = w.weights + ((int64_t)run.b * kb.s.Hkv + hk) * w.stride;
    PageWalk walk(kb, s, run.b, hk);
    Keys<D, TC, NT, BLK> keys;
    bool there = false;  // the page of this lane's token of the tile that is loaded
    float was = 0.f;     // and its sum so far
    auto load = [&](int token) __attribute__((always_inline)) {
      const int j = token + mine, id = group == 0 ? keys.id[0] : keys.id[GROUPS - 1];
      there = g < GROUPS && j >= s.lo && j < s.end && id >= 0 && id < walk.n_pages;
      keys.load(a, walk, token, TILE);
      was = there && j < s.pos ? out[j] : 0.f;
    };
    int t0 = base + (run.tile - run.first) * TILE;
    if (t0 < past) {
      keys.begin(walk, t0);
      load(t0);
    }
    auto tile = [&](auto part) __attribute__((always_inline)) {
      typename Rows<D, TIn, C, NQ>::Scores c;
      float scale[GROUPS], sum[GROUPS];
      keys.scales(x_scale, scale);
      rows.score(keys.cache.keys(), c);
      const bool keep = there;
      const float old = was;
      if (t0 + TILE < past) load(t0 + TILE);
      rows.template weigh<decltype(part)::value>(c, scale, t0, a.window, sum);
      if (keep) out[t0 + mine] = old + (group == 0 ? sum[0] : sum[GROUPS - 1]);
    };
    for (; t0 < past; t0 += TILE)
      if (t0 >= all_lo && t0 + SUB - 1 <= s.pos)
        tile(std::false_type{});
      else
        tile(std::true_type{});
    if (walk.bad && lane == 0) set_err(kb.dev_err, KDA_DEV_ERR_PAGE);
    run.next(stop);
  }
}

// A tile of keys in the LDS, as in the pages but for the order of a row's 16-byte
// chunks: chunk c of row r lies at c ^ f(r), so that the 16 lanes which a 16-byte
// read serves at a time (0-3, 12-15 and 20-27, or the others of the half wave: eight
// rows of one chunk, eight of the next) touch every bank once.
template <int D, typename TC>
struct Staged {
  typedef Cache<D, TC, false> C;
  static constexpr int TILE = C::SUB, ROW = D * (int)sizeof(TC), CHUNKS = ROW / 16, BYTES = TILE * ROW;
  static constexpr int LOADS = BYTES / 1024;                           // of a wave, 16 bytes a lane
  static constexpr int EACH = LOADS >= kWaves ? LOADS / kWaves : 1;    // to a wave that loads
  static constexpr int STEPS = CHUNKS / 4;                             // chunks of a row that a lane reads

  static __device__ __forceinline__ int swizzle(int row) {
    return CHUNKS >= 16 ? row & 15 : CHUNKS == 8 ? row >> 1 & 7 : -(row >> 2) & 3;
  }
  // Load i of this wave: where its lane reads, from the row's group of 16 on, and
  // where the wave's 1024 bytes go.
  static __device__ __forceinline__ uint32_t from(int load) {
    const uint32_t slot = load * kWave + (threadIdx.x & 63), row = slot / CHUNKS & 15;
    return row * ROW + ((slot % CHUNKS ^ swizzle(row)) << 4);
  }
  // Chunk 4 s + (lane group) of the lane's row of group u.
  static __device__ __forceinline__ u32x4 chunk(const unsigned char* tile, int u, int s) {
    const int lane = threadIdx.x & 63, row = lane & 15;
    return *reinterpret_cast<const u32x4*>(tile + (16 * u + row) * ROW + ((4 * s + (lane >> 4) ^ swizzle(row)) << 4));
  }
  // c[n][u] += the products with what chunk s of group u holds.
  template <int NQ>
  static __device__ __forceinline__ void add(const u32x4& k, int s, const typename C::Query (&q)[NQ], f32x4 (&c)[NQ]) {
    if constexpr (sizeof(TC) == 2) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) c[n] = mfma_bf16(q[n].q[s], __builtin_bit_cast(bf16x8, k), c[n]);
    } else if constexpr (sizeof(TC) == 1) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bf16x8 x = as_op(widen_e4m3<false>(k[2 * i]), widen_e4m3<true>(k[2 * i]), widen_e4m3<false>(k[2 * i + 1]),
                               widen_e4m3<true>(k[2 * i + 1]));
#pragma unroll
        for (int n = 0; n < NQ; ++n) c[n] = mfma_bf16(q[n].q[2 * s + i], x, c[n]);
      }
    } else {
      const f32x4 x = __builtin_bit_cast(f32x4, k);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < NQ; ++n) c[n] = __builtin_amdgcn_mfma_f32_16x16x4f32(q[n].q[s][i], x[i], c[n], 0, 0, 0);
    }
  }
};

// BYTES of a lane from memory to the LDS, a wave's in the order of its lanes.
template <int BYTES>
__device__ __forceinline__ void to_lds(const void* from, unsigned char* to) {
  typedef __attribute__((address_space(3))) void lds_void;
  typedef const __attribute__((address_space(1))) void global_void;
  if constexpr (BYTES == 16)
    __builtin_amdgcn_global_load_lds((global_void*)from, (lds_void*)to, 16, 0, 0);
  else
    __builtin_amdgcn_global_load_lds((global_void*)from, (lds_void*)to, 4, 0, 0);
}
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// All of the workgroup's LDS accesses so far are done; loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

constexpr int kRing = 16, kBufs = 4;
// Workgroups that registers and LDS leave room for on a CU.
template <int D, typename TIn, int NQ>
constexpr int kRowsWaves = sizeof(TIn) == 4 && D == 128 && NQ == 2 ? 3 : 4;

// More rows: NQ blocks of 16 to a wave, and chunks of 64 NQ rows in turn.  The keys
// go through the LDS, once for all four waves and three tiles ahead (read by every
// wave into its registers, one ahead, it waited most of the time: 62 us for 34).
template <int D, typename TIn, typename TC, int NQ, bool BLK>
__global__ void __launch_bounds__(kWaves * kWave, (kRowsWaves<D, TIn, NQ>)) rows_kernel(WeightsArgs w) {
  typedef Staged<D, TC> S;
  typedef Cache<D, TC, false> C;
  constexpr int TILE = S::TILE, GROUPS = C::GROUPS, CHUNK = kWaves * 16 * NQ, PER = S::EACH + (BLK ? 1 : 0);
  // A buffer: the tile, and for scales by blocks each group's, 64 times.
  constexpr int BUF = S::BYTES + (BLK ? GROUPS * 4 * kWave : 0);
  __shared__ __attribute__((aligned(1024))) unsigned char lds[kBufs * BUF];
  __shared__ float lds_sum[kWaves][kRing * TILE];
  const AttnArgs& a = w.a;
  const KvBatch& kb = a.kb;
  const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63, g = lane >> 4;
  const int hk = blockIdx.y, worker = blockIdx.x;
  Run<TILE, false> run(a, worker, worker == 0 && hk == 0 && wave == 0);
  const float x_scale = x_scale_of<TC, BLK>(a, hk);
  const int group = min(g, GROUPS - 1), mine = 16 * group + (lane & 15);
  // The loads of this wave are of one group of 16 rows.
  const bool loads = wave * S::EACH < S::LOADS;
  const int load_group = loads ? wave * S::EACH * kWave / S::CHUNKS / 16 : 0;
  uint32_t from[S::EACH];
#pragma unroll
  for (int x = 0; x < S::EACH; ++x) from[x] = S::from(wave * S::EACH + x);

  while (run.tile < run.end) {
    const Seq& s = run.s;
    const int32_t stop = min(run.end, run.first + s.tiles);
    const int R = s.n * (kb.s.Hq / kb.s.Hkv), chunks = (R + CHUNK - 1) / CHUNK;
    const int all_lo = a.window > 0 ? max((int)(s.pos + s.n) - a.window, 0) : 0;
    float* const out = w.weights + ((int64_t)run.b * kb.s.Hkv + hk) * w.stride;
    const int32_t* const table = kb.table + (int64_t)run.b * kb.max_pages;
    PageWalk walk(kb, s, run.b, hk);
    Rows<D, TIn, C, NQ> rows;
    const int last_whole = uniform((int)max(min(s.pos, (int64_t)INT32_MAX), (int64_t)0) - TILE + 1);
    // The whole run at once, or, where rows come in chunks, kRing tiles.
    const int piece = chunks > 1 ? kRing : stop - run.tile;
    for (int32_t at = run.tile; at < stop; at += piece) {
      const int first = (s.lo & ~(TILE - 1)) + (at - run.first) * TILE;
      const int past = min(s.end, first + min(stop - at, piece) * TILE), tiles = (past - first + TILE - 1) / TILE;
      for (int chunk = 0; chunk < chunks; ++chunk) {
        const int r0 = chunk * CHUNK + wave * 16 * NQ;
        if (r0 < R) rows.load(w, s, hk, r0, R);
        // vmcnt(0), in a form that the compiler sees: it would wait for the rows, and
        // with them for the tiles on their way, where they are used.
        __builtin_amdgcn_s_waitcnt(0x0f70);
        int32_t id = tiles > 0 ? walk.entry(first + 16 * load_group) : 0;
        auto load = [&](int i) __attribute__((always_inline)) {
          if (!loads) return;
          const int token = first + i * TILE + 16 * load_group;
          const int64_t row = walk.row(token, id);
          const unsigned char* base = static_cast<const unsigned char*>(kb.pages.k) + row * S::ROW;
          unsigned char* dst = lds + i % kBufs * BUF;
#pragma unroll
          for (int x = 0; x < S::EACH; ++x) to_lds<16>(base + from[x], dst + (wave * S::EACH + x) * 1024);
          if (BLK) to_lds<4>(a.scales.k + (row >> a.scales.shift), dst + S::BYTES + load_group * 4 * kWave);
          id = walk.entry(token + TILE);
        };
        lds_barrier();  // the chunk before has been read
        for (int i = 0; i < min(tiles, kBufs - 1); ++i) load(i);
        for (int i = 0; i < tiles; ++i) {
          const int behind = tiles - 1 - i, t0 = first + i * TILE;
          // Of this wave's loads at most the next two tiles' are in flight after
          // this: loads end in their order, and what else is in flight (sums) only
          // makes it wait longer.
          if (behind >= 2)
            wait_loads<2 * PER>();
          else if (behind == 1)
            wait_loads<PER>();
          else
            wait_loads<0>();
          lds_barrier();  // tile i is there, and tile i - 1 has been read
          const unsigned char* buf = lds + i % kBufs * BUF;
          f32x4 c[GROUPS][NQ];
          float scale[GROUPS], sum[GROUPS] = {};
#pragma unroll
          for (int u = 0; u < GROUPS; ++u) {
            scale[u] = x_scale;
            if (BLK) scale[u] *= *reinterpret_cast<const float*>(buf + S::BYTES + u * 4 * kWave);
#pragma unroll
            for (int n = 0; n < NQ; ++n) c[u][n] = f32x4{};
          }
          if (r0 < R) {
            u32x4 k[S::STEPS][GROUPS];
#pragma unroll
            for (int x = 0; x < S::STEPS; ++x)
#pragma unroll
              for (int u = 0; u < GROUPS; ++u) k[x][u] = S::chunk(buf, u, x);
            __builtin_amdgcn_sched_barrier(0);  // all reads first: else each is waited for before the next
#pragma unroll
            for (int x = 0; x < S::STEPS; ++x)
#pragma unroll
              for (int u = 0; u < GROUPS; ++u) S::template add<NQ>(k[x][u], x, rows.q, c[u]);
          }
          // After this tile's reads: the compiler has every read of the LDS wait for
          // the loads to it that come before it in an iteration.
          if (i + kBufs - 1 < tiles) load(i + kBufs - 1);
          if (r0 < R) {  // else zeros
            if (t0 >= all_lo && t0 <= last_whole)
              rows.template weigh<false>(c, scale, t0, a.window, sum);
            else
              rows.template weigh<true>(c, scale, t0, a.window, sum);
          }
          float* const to = &lds_sum[wave][i % kRing * TILE + mine];
          const float x = group == 0 ? sum[0] : sum[GROUPS - 1];
          if (g < GROUPS) *to = chunk == 0 ? x : *to + x;
          if (chunk < chunks - 1 || (i % kRing < kRing - 1 && i < tiles - 1)) continue;
          // The sums of kRing tiles, or of the last ones.
          lds_barrier();
          const int begin = first + i / kRing * kRing * TILE, end = min(past, t0 + TILE);
          for (int x = tid; x < end - begin; x += kWaves * kWave) {
            const int j = begin + x;
            if (j < s.lo) continue;
            const int32_t id = table[j >> kb.page_shift];
            if (id < 0 || id >= kb.pages.n_pages) continue;
            const float old = j < s.pos ? out[j] : 0.f;
            out[j] = old + ((lds_sum[0][x] + lds_sum[1][x]) + (lds_sum[2][x] + lds_sum[3][x]));
          }
          lds_barrier();
        }
      }
    }
    if (walk.bad && lane == 0) set_err(kb.dev_err, KDA_DEV_ERR_PAGE);
    run.next(stop);
  }
}

// As many workgroups as the chip's 256 CUs hold at once; a fourth to a CU for up to 16
// rows costs 64 sequences 51 us for 49 (16 of them 13.2 for 14.5).
void split(WeightsArgs& w, int tile, int at_once) {
  const Split d{tile, 0, 1, 0, 1, 1, 6};
  w.a.workers = workers_of(w.a.kb.s, 256 * at_once, d, w.a.kb.pages.page_size, w.a.kb.max_pages);
  w.a.run_tiles = d.run_tiles, w.a.start_tiles = d.start_tiles, w.a.few = d.few, w.a.row_blocks = 1;
}

template <int D, typename TIn, typename TC, int NQ, bool BLK>
hipError_t run_tokens(WeightsArgs w, hipStream_t st) {
  split(w, kWaves * Cache<D, TC, false>::SUB, NQ == 1 ? 3 : 2);
  const dim3 grid(w.a.workers, w.a.kb.s.Hkv), block(kWaves * kWave);
  if (outgrows_cache(w.a.kb))
    hipLaunchKernelGGL((tokens_kernel<D, TIn, TC, NQ, true, BLK>), grid, block, 0, st, w);
  else
    hipLaunchKernelGGL((tokens_kernel<D, TIn, TC, NQ, false, BLK>), grid, block, 0, st, w);
  return hipGetLastError();
}

template <int D, typename TIn, typename TC, int NQ, bool BLK>
hipError_t run_rows(WeightsArgs w, hipStream_t st) {
  split(w, Cache<D, TC, false>::SUB, kRowsWaves<D, TIn, NQ>);
  hipLaunchKernelGGL((rows_kernel<D, TIn, TC, NQ, BLK>), dim3(w.a.workers, w.a.kb.s.Hkv), dim3(kWaves * kWave), 0, st, w);
  return hipGetLastError();
}

// Four prompts of 7001 to 30000 tokens, us by query rows of a kv head:
//                  16 rows  32      48      64      96      128
//   bf16, tokens     32.1   33.2
//         rows, 16   32.8   33.3    33.9    34.6    56.6    57.8
//         rows, 32                  35.7    35.9    37.3    38.6
//   e4m3 in blocks   16.8   19.0
//         rows, 16   21.6   23.6    25.3    27.0    48.9    51.1
//         rows, 32                  27.1    27.1    31.2    34.3
//   f32, tokens      63.8   83.1
//         rows, 16   58.5   70.5    87.0    98.5    179     193
//         rows, 32                  125     125     158     162
// So the border at 32 rows costs f32, whose operands take twice the registers.
template <int D, typename TIn, typename TC, bool BLK>
hipError_t by_rows(const WeightsArgs& w, hipStream_t st) {
  const kda_kv_shape& s = w.a.kb.s;
  const int rows = s.T * (s.Hq / s.Hkv);
  if (rows <= 16) return run_tokens<D, TIn, TC, 1, BLK>(w, st);
  if (rows <= 32) return run_tokens<D, TIn, TC, 2, BLK>(w, st);
  return rows <= 64 ? run_rows<D, TIn, TC, 1, BLK>(w, st) : run_rows<D, TIn, TC, 2, BLK>(w, st);
}

template <typename TIn, typename TC, bool BLK = false>
hipError_t by_size(const WeightsArgs& w, hipStream_t st) {
  return w.a.kb.s.dk == 128 ? by_rows<128, TIn, TC, BLK>(w, st) : by_rows<64, TIn, TC, BLK>(w, st);
}

}  // namespace

hipError_t launch_attn_weights(const KvBatch& b, const BlockScales& scales, KvRows q, float scale, int32_t window,
                               const float* lse, float* weights, int64_t stride, hipStream_t st) {
  WeightsArgs w{};
  w.a.kb = b;
  w.a.scales = scales;
  w.a.q = q;
  w.a.scale = scale;
  w.a.window = window;
  w.lse = lse;
  w.weights = weights;
  w.stride = stride;
  if (b.s.in_dtype == KDA_F32) return by_size<float, float>(w, st);
  if (scales.k) return by_size<bf16_t, uint8_t, true>(w, st);
  if (b.s.cache_dtype == KDA_E4M3) return by_size<bf16_t, uint8_t>(w, st);
  return by_size<bf16_t, bf16_t>(w, st);
}

}  // namespace kda
