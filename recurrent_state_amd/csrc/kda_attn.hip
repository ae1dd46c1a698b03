// Attention of a sequence's new tokens over its paged cache, heads grouped.
//
// A workgroup of four waves takes a run of tiles (kda_attn_impl.h) of one kv
// head; each wave a quarter of every tile.  The T new tokens' G = Hq / Hkv
// query heads that share the kv head are the rows of one matrix, 16 to an
// MFMA tile, so a cached row is read once for all of them.  The work is bound
// by that read, and everything else stays out of its way: keys and values go
// from memory straight into the registers of the matrix instructions, without
// LDS, barriers or exchanges between lanes.
//
//   S^T = K Q^T    keys are the first operand: lane l holds key l & 15 of 16,
//                  the 16 bytes that its k-slot group l >> 4 needs.
//   softmax        S^T leaves the MFMA with a query row to each lane column
//                  and tokens 4 (l >> 4) + i in its registers: the row maximum
//                  is a maximum over registers and two lane swaps.
//   O^T = V^T P^T  P^T is used where it is.  The contraction index may be
//                  permuted as long as both operands agree: k-slot (g, e)
//                  stands for token 4 g + e (e < 4) or 16 + 4 g + e - 4, which
//                  is the token whose probability the lane already holds.  V^T
//                  is formed from eight row loads by byte permutations: lane l
//                  loads 8 (or 4) neighbouring values of its group's tokens,
//                  and V^T tile c takes the c-th of each.
//   epilogue       O^T has dv / 4 neighbouring outputs of one row in a lane.
//
// fp32 caches take the same paths through v_mfma_f32_16x16x4_f32 (no
// permutations: an operand is one value per lane); e4m3 values are widened to
// bf16, which holds each of them exactly, and their scales enter the softmax
// scale and the result.  Where scales go by blocks of tokens (a group of 16 lies in
// one block), a key's joins the factor of its scores and a value's its
// probabilities, before these are rounded: four numbers more to a tile and wave,
// loaded with the rows.  One sequence of 131071 tokens takes 53 us (269 MB, 5.7 TB/s
// in the kernel, 6 us the join).  16 of 500 to 8191 tokens with 1, 4, 8 and 16 new ones
// (4, 16, 32 and 64 rows to a kv head) take 26, 28, 32 and 51 us, with a scale a head
// 26, 28, 31 and 49.
//
// Measured with the join, 32 heads over 8 of 128, one new token each: one
// sequence of 131071 tokens 92 us (537 MB, 5.8 TB/s), 64 of 60 to 8191 tokens
// 80 us (446 MB, 5.6 TB/s), 32 of 4000 to 16001 tokens in e4m3 97 us (571 MB,
// 5.9 TB/s): at the rate of memory.  One sequence of 1021 tokens takes 10.3 us,
// which is two launches and the chain positions, page, keys, values.
//
// Rounding: scores, maxima, sums and outputs are fp32; for bf16 queries the
// probabilities, times their blocks' scales where there are any, are rounded to bf16
// (relative 2^-8, in the order of the result's own rounding) because the matrix
// instruction takes them so; the sum that divides the result has them unrounded.  Of
// the bf16 results' error against 64 bits, 1.8e-3 of their size for the long sequence
// above, 1.7e-3 is their own rounding.

#include <type_traits>

#include "kda_attn_cache.h"

namespace kda {
namespace {

constexpr int kWaves = 4;

// Column of the output that register i of tile c holds in lane group g.
template <int D, typename TC>
__device__ __forceinline__ int out_col(int g, int c, int i) {
  if constexpr (sizeof(TC) == 4) return 64 * (c / 4) + 4 * (4 * g + i) + c % 4;
  return D / 16 * (4 * g + i) + c;
}

// NQ blocks of 16 query rows to a workgroup.  BLK: scales by blocks of tokens.
template <int D, typename TIn, typename TC, int NQ, bool NT, bool BLK>
__global__ void __launch_bounds__(kWaves * kWave, NQ == 1 ? 3 : NQ == 2 ? 2 : 1) attn_kernel(AttnArgs a) {
  typedef Cache<D, TC, NT> C;
  constexpr int SUB = C::SUB, GROUPS = C::GROUPS, VC = C::VC, TILE = kWaves * SUB;
  constexpr int RS = D + 4;  // LDS row stride in floats
  __shared__ float lds_o[kWaves][16][RS];
  __shared__ f32x2 lds_ml[kWaves][16];

  const KvBatch& kb = a.kb;
  const int wave = uniform((int)threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int hk = blockIdx.y, rb = blockIdx.z, worker = blockIdx.x;
  const int G = kb.s.Hq / kb.s.Hkv;
  Run<TILE> run(a, worker, worker == 0 && hk == 0 && rb == 0 && wave == 0);
  float x_scale = a.scale * kLog2e;
  if (sizeof(TC) == 1 && !BLK) x_scale *= kb.pages.k_scale[hk];
  const float v_scale = sizeof(TC) == 1 && !BLK ? kb.pages.v_scale[hk] : 1.f;

  while (run.tile < run.end) {
    const Seq& s = run.s;
    const int32_t tile = run.tile, first = run.first, stop = min(run.end, first + s.tiles);
    const int R = s.n * G;
    if (rb * 16 * NQ < R) {
      // Queries, and the last visible token of the lane's row in each block.
      typename C::Query q[NQ];
      int vis[NQ];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const int r = (rb * NQ + n) * 16 + (here(lane) & 15), t = r / G;
        const bool live = r < R;
        vis[n] = live ? (int)max(s.pos + t, (int64_t)-1) : -1;
        C::load_query(q[n], static_cast<const TIn*>(a.q.p) + (int64_t)(s.row0 + t) * a.q.stride +
                                (hk * G + r % G) * D, live);
      }
      f32x4 out[NQ][VC];
      float m[NQ], l[NQ];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        m[n] = -INFINITY;
        l[n] = 0.f;
#pragma unroll
        for (int c = 0; c < VC; ++c) out[n][c] = f32x4{};
      }

      // This wave's tokens: t0, t0 + TILE, ... below `past`.
      const int base = (s.lo & ~(TILE - 1)) + wave * SUB;
      int t0 = base + (tile - first) * TILE;
      const int past = min(s.end, base - wave * SUB + (stop - first) * TILE);
      // Tokens below all_lo or past the first row's are hidden from some row.
      const int all_lo = a.window > 0 ? max((int)(s.pos + s.n) - a.window, 0) : 0;
      C cache;
      PageWalk walk(kb, s, run.b, hk);
      const TC* const pages_k = static_cast<const TC*>(kb.pages.k);
      const TC* const pages_v = static_cast<const TC*>(kb.pages.v);
      int32_t id[GROUPS];  // page entries of the tile to be loaded next
      int64_t at[GROUPS];
      // Scales of the groups' blocks (a group lies in one, and it or the one that
      // stands for it has visible tokens), of keys and values that are on their
      // way; of those being scored, times x_scale.
      float k_block[GROUPS], v_block[GROUPS], x_block[GROUPS];
      auto load_k = [&](int token) {
#pragma unroll
        for (int u = 0; u < GROUPS; ++u) {
          at[u] = walk.row(token + 16 * u, id[u]);
          cache.load_k(u, pages_k + at[u] * D);
          if constexpr (BLK) k_block[u] = block_scale(a.scales.k, a.scales.shift, at[u]);
          id[u] = walk.entry(token + TILE + 16 * u);
        }
      };
      auto load_v = [&] {
#pragma unroll
        for (int u = 0; u < GROUPS; ++u) {
          cache.load_v(u, pages_v + at[u] * D);
          if constexpr (BLK) v_block[u] = block_scale(a.scales.v, a.scales.shift, at[u]);
        }
      };
      f32x4 p[NQ][GROUPS];
      auto scores = [&] {
#pragma unroll
        for (int u = 0; u < GROUPS; ++u) {
          x_block[u] = BLK ? x_scale * k_block[u] : x_scale;
#pragma unroll
          for (int n = 0; n < NQ; ++n) p[n][u] = cache.score(u, q[n]);
        }
      };
      // O^T += V^T P^T, with blocks' scales in the probabilities (powers of two
      // there lose nothing).
      auto weigh = [&] {
        if constexpr (BLK)
#pragma unroll
          for (int u = 0; u < GROUPS; ++u)
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) p[n][u][i] *= v_block[u];
        cache.weigh(p, out);
      };
      // Scores to probabilities, and the earlier sums to the new maximum.
      // PART: some row does not see some token.
      auto softmax = [&](auto part) {
        constexpr bool PART = decltype(part)::value;
        const int g = PART ? here(lane) >> 4 : 0;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          const int low = a.window > 0 ? vis[n] - a.window : -1;
          float top = -INFINITY;
#pragma unroll
          for (int u = 0; u < GROUPS; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float x = p[n][u][i] * x_block[u];
              const int j = t0 + 16 * u + 4 * g + i;
              if (PART && (j > vis[n] || j <= low)) x = -INFINITY;
              p[n][u][i] = x;
              top = fmaxf(top, x);
            }
          const float mn = fmaxf(m[n], max_over_rows(top));
          const float mu = mn == -INFINITY ? 0.f : mn, keep = exp2_(m[n] - mu);
          m[n] = mn;
          float sum = 0.f;
#pragma unroll
          for (int u = 0; u < GROUPS; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              p[n][u][i] = exp2_(p[n][u][i] - mu);
              sum += p[n][u][i];
            }
          l[n] = l[n] * keep + sum;
#pragma unroll
          for (int c = 0; c < VC; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) out[n][c][i] *= keep;
        }
      };
      if (t0 < past) {
#pragma unroll
        for (int u = 0; u < GROUPS; ++u) id[u] = walk.entry(t0 + 16 * u);
      }
      while (t0 < past) {
        load_k(t0);
        load_v();
        // Tiles that every row sees whole, but the last: the next keys are
        // asked for before the softmax, the next values after the products.
        for (; t0 >= all_lo && t0 + SUB - 1 <= s.pos && t0 + TILE < past; t0 += TILE) {
          scores();
          load_k(t0 + TILE);
          softmax(std::false_type{});
          weigh();
          load_v();
        }
        scores();
        softmax(std::true_type{});
        // A probability of zero must meet a finite value.  Tokens that no row
        // sees count as zeros; where one that only some rows see is not finite,
        // the tokens of that kind are left to the loop below.
        const int g = here(lane) >> 4;
        uint32_t odd = 0;
#pragma unroll
        for (int e = 0; e < 4 * GROUPS; ++e) {
          const int j = t0 + 16 * (e >> 2) + 4 * g + (e & 3);
          cache.keep(e, (j >= s.lo) & (j < s.end));
          const uint32_t with = cache.peak(e, odd);
          odd = j < all_lo || j > s.pos ? with : odd;
        }
        if (__ballot(C::not_finite(odd)) != 0) {
#pragma unroll
          for (int e = 0; e < 4 * GROUPS; ++e) {
            const int j = t0 + 16 * (e >> 2) + 4 * g + (e & 3);
            cache.keep(e, (j >= all_lo) & (j <= s.pos));
          }
          // Token by token, each for the rows that see it: the probabilities
          // go through this wave's part of the LDS, [token][row].
          float* const plane = &lds_o[wave][0][0];
          const int col = here(lane) & 15;
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int e = 0; e < 4 * GROUPS; ++e)
              plane[(16 * (e >> 2) + 4 * g + (e & 3)) * 16 + col] = p[n][e >> 2][e & 3];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            for (int j = max(t0, s.lo); j < min(t0 + SUB, s.end); ++j) {
              if (j >= all_lo && j <= s.pos) continue;
              float w = plane[(j - t0) * 16 + col];
              const bool sees = j <= vis[n] && (a.window == 0 || j > vis[n] - a.window);
              const int64_t group = walk.row(j & ~15, walk.entry(j));
              if constexpr (BLK) w *= block_scale(a.scales.v, a.scales.shift, group);
              const TC* const v = pages_v + (group + (j & 15)) * D;
#pragma unroll
              for (int c = 0; c < VC; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float x = out[n][c][i] + w * widen(v[out_col<D, TC>(g, c, i)]);
                  out[n][c][i] = sees ? x : out[n][c][i];
                }
            }
          }
        }
        // Nor may a probability of zero meet a scale that is not finite: such a scale
        // goes to the rows that see its group, and the group counts as scaled.
        if constexpr (BLK)
#pragma unroll
          for (int u = 0; u < GROUPS; ++u) {
            if (fabsf(v_block[u]) < INFINITY) continue;
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
              const int low = a.window > 0 ? vis[n] - a.window : -1;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int j = t0 + 16 * u + 4 * g + i;
                if (j <= vis[n] && j > low) p[n][u][i] *= v_block[u];
              }
            }
            v_block[u] = 1.f;
          }
        weigh();
        t0 += TILE;
      }

      // The waves' results meet in LDS, 16 rows at a time.
      const int tid = here((int)threadIdx.x), col = tid & 15, g = (tid & 63) >> 4;
      const bool complete = tile == first && stop == first + s.tiles;
      const int64_t piece = piece_index(a, worker, tile > first ? 0 : 1, hk, rb);
      const bool bad = __syncthreads_or(walk.bad);
      if (bad && tid == 0) set_err(kb.dev_err, KDA_DEV_ERR_PAGE);
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float total = l[n];
        total = pair_sum32(pair_sum16(total));
        if (g == 0) lds_ml[wave][col] = (f32x2){m[n], total};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < VC; c += 4)
            *reinterpret_cast<f32x4*>(&lds_o[wave][col][out_col<D, TC>(g, c, i)]) =
                (f32x4){out[n][c][i], out[n][c + 1][i], out[n][c + 2][i], out[n][c + 3][i]};
        __syncthreads();
        constexpr int PER = D / 8;  // threads to a row
        for (int x = tid; x < 16 * PER; x += kWaves * kWave) {
          const int in = x / PER, c0 = x % PER * 8, r = (rb * NQ + n) * 16 + in;
          float M = -INFINITY, L = 0.f, o[8] = {};
#pragma unroll
          for (int w = 0; w < kWaves; ++w) M = fmaxf(M, lds_ml[w][in][0]);
#pragma unroll
          for (int w = 0; w < kWaves; ++w) {
            const f32x2 ml = lds_ml[w][in];
            const float f = ml[0] == -INFINITY ? 0.f : exp2_(ml[0] - M);
            L += ml[1] * f;
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] += lds_o[w][in][c0 + i] * f;
          }
          if (r < R) {
            if (!complete) {
              const int64_t row = piece * a.rows + 16 * n + in;
              store8(a.piece_o + row * D + c0, o);
              if (c0 == 0) a.piece_ml[row] = (f32x2){M, bad ? -1.f : L};
            } else if (!bad) {
              const float inv = s.pos + r / G < 0 ? 0.f : v_scale / L;  // 0 / 0 where every score is -inf
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] *= inv;
              const int64_t row = (int64_t)(s.row0 + r / G) * kb.s.Hq + hk * G + r % G;
              store8(static_cast<TIn*>(a.o) + row * D + c0, o);
              if (a.lse && c0 == 0) a.lse[row] = (M + __log2f(L)) * kLn2;
            }
          }
        }
        __syncthreads();
      }
    }
    run.next(stop);
  }
}

// Blocks of 16 query rows that a workgroup takes: all of them up to four (two
// in fp32, whose operands need twice the registers), so that a cached row is
// read once; more rows make more workgroups.
int query_blocks(const kda_kv_shape& s) {
  const int rows = s.T * (s.Hq / s.Hkv);
  if (rows <= 16) return 1;
  return rows <= 32 || s.in_dtype == KDA_F32 ? 2 : 4;
}

Split split_of(const kda_kv_shape& s, int32_t page_size, int32_t max_pages) {
  const int nq = query_blocks(s);
  // A sequence's beginning counted as one tile: 84.3 -> 80.5 us at 64 sequences
  // of 60 to 8191 tokens (two: 82.7).  One piece a worker from six workers to a
  // sequence on (96 to a kv head): with two, 40 of up to 8000 took 64.9 us for
  // 60.2, 24 took 48.5 for 47.2; with eight, 16 took 31.4 for 30.8.
  Split d{kWaves * (s.in_dtype == KDA_F32 ? 16 : 32), 16 * nq, 0, 0, 1, 1, 6};
  d.row_blocks = (s.T * (s.Hq / s.Hkv) + d.rows - 1) / d.rows;
  // As many workgroups as the chip's 256 CUs hold at once.
  d.workers = workers_of(s, 256 * (nq == 1 ? 3 : nq == 2 ? 2 : 1), d, page_size, max_pages);
  return d;
}

// A pool that the 256 MB Infinity Cache cannot hold is read past it with
// non-temporal loads: 105.8 -> 92.1 us at one sequence of 131071 tokens, 96 ->
// 88 at 64 of up to 8191, 116 -> 107 in e4m3.  A smaller one may still be there
// from the call before, and is then read from there: 25 us with plain loads
// against 29 for 16 sequences whose three pools of 78 MB took turns.
template <int D, typename TIn, typename TC, int NQ, bool BLK>
hipError_t run(const AttnArgs& a, hipStream_t st) {
  const dim3 grid(a.workers, a.kb.s.Hkv, a.row_blocks), block(kWaves * kWave);
  if (outgrows_cache(a.kb))
    hipLaunchKernelGGL((attn_kernel<D, TIn, TC, NQ, true, BLK>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((attn_kernel<D, TIn, TC, NQ, false, BLK>), grid, block, 0, st, a);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : run_join<D, TIn>(a, st);
}

template <typename TIn, typename TC, bool BLK = false>
hipError_t by_size(const AttnArgs& a, hipStream_t st) {
  const bool wide = a.kb.s.dk == 128;
  switch (a.rows) {
    case 16: return wide ? run<128, TIn, TC, 1, BLK>(a, st) : run<64, TIn, TC, 1, BLK>(a, st);
    case 32: return wide ? run<128, TIn, TC, 2, BLK>(a, st) : run<64, TIn, TC, 2, BLK>(a, st);
  }
  if constexpr (sizeof(TIn) == 2) return wide ? run<128, TIn, TC, 4, BLK>(a, st) : run<64, TIn, TC, 4, BLK>(a, st);
  return hipErrorInvalidValue;
}

}  // namespace

size_t attn_workspace_bytes(const kda_kv_shape& s, int32_t page_size, int32_t max_pages) {
  if (s.dk == 576) return latent_workspace_bytes(s, page_size, max_pages);
  return workspace_of(s, split_of(s, page_size, max_pages)).total;
}

hipError_t launch_attn_decode(const KvBatch& b, const BlockScales& scales, KvRows q, float scale, int32_t window,
                              void* o, float* lse, void* workspace, hipStream_t st) {
  if (b.s.dk == 576) return launch_attn_latent(b, q, scale, window, o, lse, workspace, st);
  const AttnArgs a =
      make_args(b, scales, q, scale, window, o, lse, workspace, split_of(b.s, b.pages.page_size, b.max_pages));
  if (b.s.in_dtype == KDA_F32) return by_size<float, float>(a, st);
  if (scales.k) return by_size<bf16_t, uint8_t, true>(a, st);
  if (b.s.cache_dtype == KDA_E4M3) return by_size<bf16_t, uint8_t>(a, st);
  return by_size<bf16_t, bf16_t>(a, st);
}

}  // namespace kda
