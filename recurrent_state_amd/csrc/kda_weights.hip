// The attention weights that cached tokens get, summed over the query rows of a
// call and the query heads of a kv head.
//
// The weight e^(s - lse) of a row and a token needs the row's lse, so the keys
// are read a second time after the attention, without the values.  A workgroup
// takes a run of tiles (kda_attn_impl.h) of one kv head, each wave a quarter of
// every tile, and keys go from memory into the registers of the matrix
// instructions, as in kda_attn.hip.  Here S = Q K^T leaves the MFMA with a token
// to each lane column, so the sum over a tile's 16 rows is one over registers
// and two lane swaps, and no result leaves the wave that made it: no pieces, no
// atomics, one order.  The rows' queries and lse stay in registers where a call
// has up to 64 (two blocks of 16 in fp32); more are read again, from the caches,
// for every 32 tokens.

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

// NQ blocks of 16 query rows at a time.  With NQ > 1 a sequence may have more:
// each chunk of rows takes kAgain tiles before the next one does, which finds
// their keys in the caches and adds to the sums that it finds.
constexpr int kAgain = 8;

template <int D, typename TIn, typename TC, int NQ, bool NT, bool BLK>
__global__ void __launch_bounds__(kWaves * kWave, NQ == 1 ? 3 : 2) weights_kernel(WeightsArgs w) {
  typedef Cache<D, TC, NT> C;
  constexpr int SUB = C::SUB, GROUPS = C::GROUPS, TILE = kWaves * SUB;
  constexpr bool MANY = NQ > 1;
  const AttnArgs& a = w.a;
  const KvBatch& kb = a.kb;
  const int wave = uniform((int)threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 4;
  const int hk = blockIdx.y, worker = blockIdx.x, G = kb.s.Hq / kb.s.Hkv;
  Run<TILE> run(a, worker, worker == 0 && hk == 0 && wave == 0);
  float x_scale = a.scale * kLog2e;
  if (sizeof(TC) == 1 && !BLK) x_scale *= kb.pages.k_scale[hk];
  // Lane group u holds the sums of tokens 16 u + (lane & 15) of a tile.
  const int mine = 16 * min(g, GROUPS - 1) + (lane & 15);

  while (run.tile < run.end) {
    const Seq& s = run.s;
    const int32_t first = run.first, stop = min(run.end, first + s.tiles);
    const int R = s.n * G, chunks = MANY ? (R + 16 * NQ - 1) / (16 * NQ) : 1;
    // Rows [16 NQ chunk, + 16 NQ): queries by lane column, lse and the last
    // visible token by register.  A row that is not there has the first one's
    // query, an lse that makes its weights 0, and sees no token.
    typename C::Query q[NQ];
    f32x4 lse[NQ];
    int vis[NQ][4];
    auto rows = [&](int chunk) __attribute__((always_inline)) {
      const int r0 = chunk * NQ * 16;
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const int rq = r0 + 16 * n + (lane & 15), r = rq < R ? rq : r0, tq = r / G;
        C::load_query(q[n], static_cast<const TIn*>(a.q.p) + (int64_t)(s.row0 + tq) * a.q.stride +
                                (hk * G + r - tq * G) * D, true);
        const int r4 = r0 + 16 * n + 4 * g;
        int t = r4 / G, h = r4 - t * G;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool live = r4 + i < R;
          lse[n][i] = live ? w.lse[(int64_t)(s.row0 + t) * kb.s.Hq + hk * G + h] * kLog2e : INFINITY;
          vis[n][i] = live ? (int)max(s.pos + t, (int64_t)-1) : -1;
          if (++h == G) h = 0, ++t;
        }
      }
    };

    const int base = (s.lo & ~(TILE - 1)) + wave * SUB;
    const int all_lo = a.window > 0 ? max((int)(s.pos + s.n) - a.window, 0) : 0;
    const TC* const pages = static_cast<const TC*>(kb.pages.k);
    float* const out = w.weights + ((int64_t)run.b * kb.s.Hkv + hk) * w.stride;
    PageWalk walk(kb, s, run.b, hk);
    for (int32_t tile = run.tile; tile < stop; tile += MANY ? kAgain : stop - run.tile) {
      const int32_t upto = MANY ? min(stop, tile + kAgain) : stop;
      for (int chunk = 0; chunk < chunks; ++chunk) {
        rows(chunk);
        int t0 = base + (tile - first) * TILE;
        const int past = min(s.end, base - wave * SUB + (upto - first) * TILE);
        C cache;
        int32_t id[GROUPS];  // page entries of the tile to be loaded next
        float k_block[GROUPS];
        bool there;          // the page of this lane's token of the tile that is loaded
        float was;           // and its sum so far
        auto load = [&](int token) __attribute__((always_inline)) {
          there = true;
#pragma unroll
          for (int u = 0; u < GROUPS; ++u) {
            const int64_t at = walk.row(token + 16 * u, id[u]);
            if (min(g, GROUPS - 1) == u) there = id[u] >= 0 && id[u] < walk.n_pages;
            cache.load_k(u, pages + at * D);
            if constexpr (BLK) k_block[u] = block_scale(a.scales.k, a.scales.shift, at);
            id[u] = walk.entry(token + TILE + 16 * u);
          }
          const int j = token + mine;
          there &= g < GROUPS && j >= s.lo && j < s.end;
          was = there && (j < s.pos || chunk > 0) ? out[j] : 0.f;
        };
        if (t0 < past) {
#pragma unroll
          for (int u = 0; u < GROUPS; ++u) id[u] = walk.entry(t0 + 16 * u);
          load(t0);
        }
        // One tile; PART: some row does not see some token.
        auto weigh = [&](auto part) __attribute__((always_inline)) {
          constexpr bool PART = decltype(part)::value;
          f32x4 c[NQ][GROUPS];
          float xs[GROUPS], sum[GROUPS] = {};
#pragma unroll
          for (int u = 0; u < GROUPS; ++u) {
            xs[u] = BLK ? x_scale * k_block[u] : x_scale;
#pragma unroll
            for (int n = 0; n < NQ; ++n) c[n][u] = cache.score_t(u, q[n]);
          }
          const bool keep = there;
          const float old = was;
          if (t0 + TILE < past) load(t0 + TILE);
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int u = 0; u < GROUPS; ++u) {
              const int j = t0 + 16 * u + (lane & 15);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float e = exp2_(__builtin_fmaf(c[n][u][i], xs[u], -lse[n][i]));
                const bool hidden = PART && (j > vis[n][i] || (a.window > 0 && j <= vis[n][i] - a.window));
                sum[u] += hidden ? 0.f : e;
              }
            }
          float mine_sum = 0.f;
#pragma unroll
          for (int u = 0; u < GROUPS; ++u) {
            const float x = pair_sum32(pair_sum16(sum[u]));
            if (min(g, GROUPS - 1) == u) mine_sum = x;
          }
          if (keep) out[t0 + mine] = old + mine_sum;
        };
        for (; t0 < past; t0 += TILE)
          if (t0 >= all_lo && t0 + SUB - 1 <= s.pos)
            weigh(std::false_type{});
          else
            weigh(std::true_type{});
      }
    }
    if (walk.bad && lane == 0) set_err(kb.dev_err, KDA_DEV_ERR_PAGE);
    run.next(stop);
  }
}

template <int D, typename TIn, typename TC, int NQ, bool BLK>
hipError_t run(WeightsArgs w, hipStream_t st) {
  constexpr int kTile = kWaves * Cache<D, TC, false>::SUB;
  const kda_kv_shape& s = w.a.kb.s;
  const Split d{kTile, 16 * NQ, 1, 0, 1, 1, 6};
  // As many workgroups as the chip's 256 CUs hold at once.
  w.a.workers = workers_of(s, 256 * (NQ == 1 ? 3 : 2), d, w.a.kb.pages.page_size, w.a.kb.max_pages);
  w.a.run_tiles = d.run_tiles, w.a.start_tiles = d.start_tiles, w.a.few = d.few;
  w.a.row_blocks = 1, w.a.rows = d.rows;
  const dim3 grid(w.a.workers, s.Hkv), block(kWaves * kWave);
  if (outgrows_cache(w.a.kb))
    hipLaunchKernelGGL((weights_kernel<D, TIn, TC, NQ, true, BLK>), grid, block, 0, st, w);
  else
    hipLaunchKernelGGL((weights_kernel<D, TIn, TC, NQ, false, BLK>), grid, block, 0, st, w);
  return hipGetLastError();
}

template <int D, typename TIn, typename TC, bool BLK>
hipError_t by_rows(const WeightsArgs& w, hipStream_t st) {
  const kda_kv_shape& s = w.a.kb.s;
  const int rows = s.T * (s.Hq / s.Hkv);
  if (rows <= 16) return run<D, TIn, TC, 1, BLK>(w, st);
  // fp32 queries need twice the registers.
  if (rows <= 32 || sizeof(TIn) == 4) return run<D, TIn, TC, 2, BLK>(w, st);
  if constexpr (sizeof(TIn) == 2) return run<D, TIn, TC, 4, BLK>(w, st);
  return hipErrorInvalidValue;
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
