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
// scale and the result.
//
// Measured with the join, 32 heads over 8 of 128, one new token each: one
// sequence of 131071 tokens 92 us (537 MB, 5.8 TB/s), 64 of 60 to 8191 tokens
// 80 us (446 MB, 5.6 TB/s), 32 of 4000 to 16001 tokens in e4m3 97 us (571 MB,
// 5.9 TB/s): at the rate of memory.  One sequence of 1021 tokens takes 10.3 us,
// which is two launches and the chain positions, page, keys, values.
//
// Rounding: scores, maxima, sums and outputs are fp32; for bf16 queries the
// probabilities are rounded to bf16 (relative 2^-8, in the order of the
// result's own rounding) because the matrix instruction takes them so.

#include <type_traits>

#include "kda_attn_impl.h"

namespace kda {
namespace {

constexpr int kWaves = 4;

typedef __attribute__((ext_vector_type(2))) uint16_t u16x2;

__device__ __forceinline__ float widen(bf16_t x) { return __uint_as_float((uint32_t)x << 16); }
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint8_t x) { return __builtin_amdgcn_cvt_f32_fp8((int)x, 0); }
// Two e4m3 values (the low or high pair of w) as packed bf16, exactly.
template <bool HI>
__device__ __forceinline__ uint32_t widen_e4m3(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, HI));
}

// The probabilities of 32 tokens as an operand, and products with V^T tiles:
// w holds two neighbouring columns of the lane's eight tokens.
template <int NQ>
struct Weights {
  bf16x8 p[NQ];

  __device__ __forceinline__ explicit Weights(const f32x4 (&x)[NQ][2]) {
#pragma unroll
    for (int n = 0; n < NQ; ++n)
      p[n] = as_op(pack2(x[n][0][0], x[n][0][1]), pack2(x[n][0][2], x[n][0][3]), pack2(x[n][1][0], x[n][1][1]),
                   pack2(x[n][1][2], x[n][1][3]));
  }
  template <int VC>
  __device__ __forceinline__ void add(const uint32_t (&w)[8], bool high, f32x4 (&out)[NQ][VC], int c) const {
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], high ? 0x07060302u : 0x05040100u);
    const bf16x8 vt = as_op(x[0], x[1], x[2], x[3]);
#pragma unroll
    for (int n = 0; n < NQ; ++n) out[n][c] = mfma_bf16(vt, p[n], out[n][c]);
  }
};

template <bool NT, typename V, typename T>
__device__ __forceinline__ V load(const T* p) {
  const V* v = reinterpret_cast<const V*>(p);
  return NT ? __builtin_nontemporal_load(v) : *v;
}

// One wave's share of the keys and values of SUB tokens, in the layout that
// the loads give, and the operands made from it.  Token t of the share is row
// `t & 15` of group `t >> 4`; pk / pv point to each group's first row.
//
// NT: loads that leave the caches to others (see run()).
//
// bf16: 32 tokens, 32 contraction slots.
template <int D, typename TC, bool NT>
struct Cache;

template <int D, bool NT>
struct Cache<D, bf16_t, NT> {
  static constexpr int GROUPS = 2, SUB = 32;
  static constexpr int VC = D / 16;  // neighbouring values of a row in a lane
  u32x4 k[2][D / 32];
  uint32_t v[8][VC / 2];
  struct Query {
    bf16x8 q[D / 32];
  };

  static __device__ __forceinline__ void load_query(Query& q, const bf16_t* row, bool live) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int s = 0; s < D / 32; ++s)
      q.q[s] = live ? *reinterpret_cast<const bf16x8*>(row + 32 * s + 8 * g) : bf16x8{};
  }
  __device__ __forceinline__ void load_k(int u, const bf16_t* rows) {
    const int l = threadIdx.x & 63;
#pragma unroll
    for (int s = 0; s < D / 32; ++s)
      k[u][s] = load<NT, u32x4>(rows + (l & 15) * D + 32 * s + 8 * (l >> 4));
  }
  __device__ __forceinline__ void load_v(int u, const bf16_t* rows) {
    const int l = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bf16_t* p = rows + (4 * (l >> 4) + j) * D + VC * (l & 15);
      if constexpr (VC == 8) {
        const u32x4 w = load<NT, u32x4>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * u + j][i] = w[i];
      } else {
        const u32x2 w = load<NT, u32x2>(p);
        v[4 * u + j][0] = w[0];
        v[4 * u + j][1] = w[1];
      }
    }
  }
  __device__ __forceinline__ f32x4 score(int u, const Query& q) const {
    f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < D / 32; ++s) c = mfma_bf16(__builtin_bit_cast(bf16x8, k[u][s]), q.q[s], c);
    return c;
  }
  // Values of the lane's token e (of 8: group e >> 2): zero unless kept / tested.
  __device__ __forceinline__ void keep(int e, bool kept) {
#pragma unroll
    for (int i = 0; i < VC / 2; ++i) v[e][i] = kept ? v[e][i] : 0;
  }
  // What of `acc` and token e tells a value that is not finite: the largest
  // magnitude of the low and of the high halves.
  __device__ __forceinline__ uint32_t peak(int e, uint32_t acc) const {
#pragma unroll
    for (int i = 0; i < VC / 2; ++i)
      acc = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, acc),
                                                                   __builtin_bit_cast(u16x2, v[e][i] & 0x7fff7fffu)));
    return acc;
  }
  static __device__ __forceinline__ bool not_finite(uint32_t acc) {
    return (acc & 0xffffu) >= 0x7f80u || acc >= 0x7f800000u;
  }
  // out[c] += V^T tile c times the probabilities.
  template <int NQ>
  __device__ __forceinline__ void weigh(const f32x4 (&p)[NQ][2], f32x4 (&out)[NQ][VC]) const {
    const Weights<NQ> weights(p);
#pragma unroll
    for (int c = 0; c < VC; ++c) {
      uint32_t w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = v[e][c / 2];
      weights.add(w, c & 1, out, c);
    }
  }
};

// e4m3: as bf16, widened when used.  A key load of 16 bytes feeds two
// contraction steps, so the queries are laid out to match.
template <int D, bool NT>
struct Cache<D, uint8_t, NT> {
  static constexpr int GROUPS = 2, SUB = 32;
  static constexpr int VC = D / 16;
  u32x4 k[2][D / 64];
  uint32_t v[8][VC / 4];
  struct Query {
    bf16x8 q[D / 32];
  };

  static __device__ __forceinline__ void load_query(Query& q, const bf16_t* row, bool live) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int s = 0; s < D / 32; ++s)
      q.q[s] = live ? *reinterpret_cast<const bf16x8*>(row + 64 * (s / 2) + 16 * g + 8 * (s & 1)) : bf16x8{};
  }
  __device__ __forceinline__ void load_k(int u, const uint8_t* rows) {
    const int l = threadIdx.x & 63;
#pragma unroll
    for (int s = 0; s < D / 64; ++s)
      k[u][s] = load<NT, u32x4>(rows + (l & 15) * D + 64 * s + 16 * (l >> 4));
  }
  __device__ __forceinline__ void load_v(int u, const uint8_t* rows) {
    const int l = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint8_t* p = rows + (4 * (l >> 4) + j) * D + VC * (l & 15);
      if constexpr (VC == 8) {
        const u32x2 w = load<NT, u32x2>(p);
        v[4 * u + j][0] = w[0];
        v[4 * u + j][1] = w[1];
      } else {
        v[4 * u + j][0] = load<NT, uint32_t>(p);
      }
    }
  }
  __device__ __forceinline__ f32x4 score(int u, const Query& q) const {
    f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
      const uint32_t a = k[u][s / 2][2 * (s & 1)], b = k[u][s / 2][2 * (s & 1) + 1];
      c = mfma_bf16(as_op(widen_e4m3<false>(a), widen_e4m3<true>(a), widen_e4m3<false>(b), widen_e4m3<true>(b)),
                    q.q[s], c);
    }
    return c;
  }
  __device__ __forceinline__ void keep(int e, bool kept) {
#pragma unroll
    for (int i = 0; i < VC / 4; ++i) v[e][i] = kept ? v[e][i] : 0;
  }
  // The type has NaN only, all ones but the sign: adding one carries into it.
  __device__ __forceinline__ uint32_t peak(int e, uint32_t acc) const {
#pragma unroll
    for (int i = 0; i < VC / 4; ++i) acc |= (v[e][i] & 0x7f7f7f7fu) + 0x01010101u;
    return acc;
  }
  static __device__ __forceinline__ bool not_finite(uint32_t acc) { return (acc & 0x80808080u) != 0; }
  template <int NQ>
  __device__ __forceinline__ void weigh(const f32x4 (&p)[NQ][2], f32x4 (&out)[NQ][VC]) const {
    const Weights<NQ> weights(p);
#pragma unroll
    for (int c = 0; c < VC; c += 2) {
      uint32_t w[8];  // columns c and c + 1 of the lane's tokens
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = c & 2 ? widen_e4m3<true>(v[e][c / 4]) : widen_e4m3<false>(v[e][c / 4]);
      weights.add(w, false, out, c);
      weights.add(w, true, out, c + 1);
    }
  }
};

// fp32: 16 tokens; a contraction step takes four k-slots, one to each lane
// group.  V^T tile (64 h + c): columns 64 h + 4 m + c.
template <int D, bool NT>
struct Cache<D, float, NT> {
  static constexpr int GROUPS = 1, SUB = 16;
  static constexpr int VC = D / 16;
  f32x4 k[1][D / 16];
  f32x4 v[4][D / 64];
  struct Query {
    f32x4 q[D / 16];
  };

  static __device__ __forceinline__ void load_query(Query& q, const float* row, bool live) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
      q.q[s] = live ? *reinterpret_cast<const f32x4*>(row + 16 * s + 4 * g) : f32x4{};
  }
  __device__ __forceinline__ void load_k(int u, const float* rows) {
    const int l = threadIdx.x & 63;
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
      k[u][s] = load<NT, f32x4>(rows + (l & 15) * D + 16 * s + 4 * (l >> 4));
  }
  __device__ __forceinline__ void load_v(int, const float* rows) {
    const int l = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
        v[j][h] = load<NT, f32x4>(rows + (4 * (l >> 4) + j) * D + 64 * h + 4 * (l & 15));
  }
  __device__ __forceinline__ f32x4 score(int u, const Query& q) const {
    f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(k[u][s][i], q.q[s][i], c, 0, 0, 0);
    return c;
  }
  __device__ __forceinline__ void keep(int e, bool kept) {
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[e][h][i] = kept ? v[e][h][i] : 0.f;
  }
  __device__ __forceinline__ uint32_t peak(int e, uint32_t acc) const {
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc = max(acc, __float_as_uint(v[e][h][i]) & 0x7fffffffu);
    return acc;
  }
  static __device__ __forceinline__ bool not_finite(uint32_t acc) { return acc >= 0x7f800000u; }
  template <int NQ>
  __device__ __forceinline__ void weigh(const f32x4 (&p)[NQ][1], f32x4 (&out)[NQ][VC]) const {
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int n = 0; n < NQ; ++n)
            out[n][4 * h + c] =
                __builtin_amdgcn_mfma_f32_16x16x4f32(v[j][h][c], p[n][0][j], out[n][4 * h + c], 0, 0, 0);
  }
};

// Column of the output that register i of tile c holds in lane group g.
template <int D, typename TC>
__device__ __forceinline__ int out_col(int g, int c, int i) {
  if constexpr (sizeof(TC) == 4) return 64 * (c / 4) + 4 * (4 * g + i) + c % 4;
  return D / 16 * (4 * g + i) + c;
}

// NQ blocks of 16 query rows to a workgroup.
template <int D, typename TIn, typename TC, int NQ, bool NT>
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
  if (sizeof(TC) == 1) x_scale *= kb.pages.k_scale[hk];
  const float v_scale = sizeof(TC) == 1 ? kb.pages.v_scale[hk] : 1.f;

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
      auto load_k = [&](int token) {
#pragma unroll
        for (int u = 0; u < GROUPS; ++u) {
          at[u] = walk.row(token + 16 * u, id[u]);
          cache.load_k(u, pages_k + at[u] * D);
          id[u] = walk.entry(token + TILE + 16 * u);
        }
      };
      auto load_v = [&] {
#pragma unroll
        for (int u = 0; u < GROUPS; ++u) cache.load_v(u, pages_v + at[u] * D);
      };
      f32x4 p[NQ][GROUPS];
      auto scores = [&] {
#pragma unroll
        for (int u = 0; u < GROUPS; ++u)
#pragma unroll
          for (int n = 0; n < NQ; ++n) p[n][u] = cache.score(u, q[n]);
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
              float x = p[n][u][i] * x_scale;
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
          cache.weigh(p, out);
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
              const float w = plane[(j - t0) * 16 + col];
              const bool sees = j <= vis[n] && (a.window == 0 || j > vis[n] - a.window);
              const TC* const v = pages_v + (walk.row(j & ~15, walk.entry(j)) + (j & 15)) * D;
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
        cache.weigh(p, out);
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
template <int D, typename TIn, typename TC, int NQ>
hipError_t run(const AttnArgs& a, hipStream_t st) {
  const dim3 grid(a.workers, a.kb.s.Hkv, a.row_blocks), block(kWaves * kWave);
  if (outgrows_cache(a.kb))
    hipLaunchKernelGGL((attn_kernel<D, TIn, TC, NQ, true>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((attn_kernel<D, TIn, TC, NQ, false>), grid, block, 0, st, a);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : run_join<D, TIn>(a, st);
}

template <typename TIn, typename TC>
hipError_t by_size(const AttnArgs& a, hipStream_t st) {
  const bool wide = a.kb.s.dk == 128;
  switch (a.rows) {
    case 16: return wide ? run<128, TIn, TC, 1>(a, st) : run<64, TIn, TC, 1>(a, st);
    case 32: return wide ? run<128, TIn, TC, 2>(a, st) : run<64, TIn, TC, 2>(a, st);
  }
  if constexpr (sizeof(TIn) == 2) return wide ? run<128, TIn, TC, 4>(a, st) : run<64, TIn, TC, 4>(a, st);
  return hipErrorInvalidValue;
}

}  // namespace

size_t attn_workspace_bytes(const kda_kv_shape& s, int32_t page_size, int32_t max_pages) {
  if (s.dk == 576) return latent_workspace_bytes(s, page_size, max_pages);
  return workspace_of(s, split_of(s, page_size, max_pages)).total;
}

hipError_t launch_attn_decode(const KvBatch& b, KvRows q, float scale, int32_t window, void* o, float* lse,
                              void* workspace, hipStream_t st) {
  if (b.s.dk == 576) return launch_attn_latent(b, q, scale, window, o, lse, workspace, st);
  const AttnArgs a =
      make_args(b, q, scale, window, o, lse, workspace, split_of(b.s, b.pages.page_size, b.max_pages));
  if (b.s.in_dtype == KDA_F32) return by_size<float, float>(a, st);
  if (b.s.cache_dtype == KDA_E4M3) return by_size<bf16_t, uint8_t>(a, st);
  return by_size<bf16_t, bf16_t>(a, st);
}

}  // namespace kda
