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

// NQ blocks of 16 query rows at a time.  MANY: a sequence may have more.
template <int D, typename TIn, typename TC, int NQ, bool MANY, bool NT, bool BLK>
__global__ void __launch_bounds__(kWaves * kWave) weights_kernel(WeightsArgs w) {
  typedef Cache<D, TC, NT> C;
  constexpr int SUB = C::SUB, GROUPS = C::GROUPS, TILE = kWaves * SUB;
  const AttnArgs& a = w.a;
  const KvBatch& kb = a.kb;
  const int wave = uniform((int)threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 4;
  const int hk = blockIdx.y, worker = blockIdx.x, G = kb.s.Hq / kb.s.Hkv;
  Run<TILE> run(a, worker, worker == 0 && hk == 0 && wave == 0);
  float x_scale = a.scale * kLog2e;
  if (sizeof(TC) == 1 && !BLK) x_scale *= kb.pages.k_scale[hk];

  while (run.tile < run.end) {
    const Seq& s = run.s;
    const int32_t tile = run.tile, first = run.first, stop = min(run.end, first + s.tiles);
    const int R = s.n * G;
    // Rows [chunk * 16 NQ, + 16 NQ): queries by lane column, lse and the last
    // visible token by register.  A row that is not there has the first one's
    // query, an lse that makes its weights 0, and sees no token.
    typename C::Query q[NQ];
    f32x4 lse[NQ];
    int vis[NQ][4];
    auto rows = [&](int chunk) __attribute__((always_inline)) {
      const int r0 = chunk * NQ * 16;
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const int rq = r0 + 16 * n + (lane & 15), r = rq < R ? rq : r0;
        C::load_query(q[n], static_cast<const TIn*>(a.q.p) + (int64_t)(s.row0 + r / G) * a.q.stride +
                                (hk * G + r % G) * D, true);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = r0 + 16 * n + 4 * g + i, t = r / G;
          const bool live = r < R;
          lse[n][i] = live ? w.lse[(int64_t)(s.row0 + t) * kb.s.Hq + hk * G + r % G] * kLog2e : INFINITY;
          vis[n][i] = live ? (int)max(s.pos + t, (int64_t)-1) : -1;
        }
      }
    };
    const int chunks = MANY ? (R + 16 * NQ - 1) / (16 * NQ) : 1;
    if (!MANY) rows(0);

    const int base = (s.lo & ~(TILE - 1)) + wave * SUB;
    int t0 = base + (tile - first) * TILE;
    const int past = min(s.end, base - wave * SUB + (stop - first) * TILE);
    const int all_lo = a.window > 0 ? max((int)(s.pos + s.n) - a.window, 0) : 0;
    C cache;
    PageWalk walk(kb, s, run.b, hk);
    const TC* const pages = static_cast<const TC*>(kb.pages.k);
    float* const out = w.weights + ((int64_t)run.b * kb.s.Hkv + hk) * w.stride;
    // Lane group u holds the sums of tokens 16 u + (lane & 15) of the tile.
    const int mine = 16 * min(g, GROUPS - 1) + (lane & 15);
    int32_t id[GROUPS];    // page entries of the tile to be loaded next
    float k_block[GROUPS];
    bool there;            // the page of this lane's token of the tile that is loaded
    float was;             // and its sum so far
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
      was = there && j < s.pos ? out[j] : 0.f;
    };
    if (t0 < past) {
#pragma unroll
      for (int u = 0; u < GROUPS; ++u) id[u] = walk.entry(t0 + 16 * u);
      load(t0);
    }
    // One tile; PART: some row does not see some token.
    auto weigh = [&](auto part) __attribute__((always_inline)) {
      constexpr bool PART = decltype(part)::value;
      float sum[GROUPS] = {};
      const C now = cache;
      float xs[GROUPS];
#pragma unroll
      for (int u = 0; u < GROUPS; ++u) xs[u] = BLK ? x_scale * k_block[u] : x_scale;
      const bool keep = there;
      const float old = was;
      if (t0 + TILE < past) load(t0 + TILE);
      for (int chunk = 0; chunk < chunks; ++chunk) {
        if (MANY) rows(chunk);
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int u = 0; u < GROUPS; ++u) {
            const f32x4 c = now.score_t(u, q[n]);
            const int j = t0 + 16 * u + (lane & 15);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float e = exp2_(__builtin_fmaf(c[i], xs[u], -lse[n][i]));
              const bool hidden = PART && (j > vis[n][i] || (a.window > 0 && j <= vis[n][i] - a.window));
              sum[u] += hidden ? 0.f : e;
            }
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
    while (t0 < past) {
      if (t0 >= all_lo && t0 + SUB - 1 <= s.pos)
        weigh(std::false_type{});
      else
        weigh(std::true_type{});
      t0 += TILE;
    }
    if (walk.bad && lane == 0) set_err(kb.dev_err, KDA_DEV_ERR_PAGE);
    run.next(stop);
  }
}

template <int D, typename TIn, typename TC, int NQ, bool MANY, bool BLK>
hipError_t run(WeightsArgs w, hipStream_t st) {
  constexpr int kTile = kWaves * Cache<D, TC, false>::SUB;
  const kda_kv_shape& s = w.a.kb.s;
  Split d{kTile, 16 * NQ, 1, 0, 1, 1, 6};
  const int32_t page = w.a.kb.pages.page_size;
  w.a.workers = workers_of(s, 256 * 4, d, page, w.a.kb.max_pages);
  w.a.run_tiles = d.run_tiles, w.a.start_tiles = d.start_tiles, w.a.few = d.few;
  w.a.row_blocks = 1, w.a.rows = d.rows;
  const dim3 grid(w.a.workers, s.Hkv), block(kWaves * kWave);
  if (outgrows_cache(w.a.kb))
    hipLaunchKernelGGL((weights_kernel<D, TIn, TC, NQ, MANY, true, BLK>), grid, block, 0, st, w);
  else
    hipLaunchKernelGGL((weights_kernel<D, TIn, TC, NQ, MANY, false, BLK>), grid, block, 0, st, w);
  return hipGetLastError();
}

template <int D, typename TIn, typename TC, bool BLK>
hipError_t by_rows(const WeightsArgs& w, hipStream_t st) {
  const kda_kv_shape& s = w.a.kb.s;
  const int rows = s.T * (s.Hq / s.Hkv);
  if (rows <= 16) return run<D, TIn, TC, 1, false, BLK>(w, st);
  if (rows <= 32) return run<D, TIn, TC, 2, false, BLK>(w, st);
  if constexpr (sizeof(TIn) == 4) {
    return run<D, TIn, TC, 2, true, BLK>(w, st);
  } else {
    if (rows <= 64) return run<D, TIn, TC, 4, false, BLK>(w, st);
    return run<D, TIn, TC, 4, true, BLK>(w, st);
  }
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
