// Keys and values of a grouped cache in the registers of the matrix
// instructions: what the attention (kda_attn.hip) and the sums of its weights
// (kda_weights.hip) read the pages with.
#pragma once

#include "kda_attn_impl.h"

namespace kda {
namespace {

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

// The scale of the block that holds row `row` of the pool (the same in every
// lane), through the scalar cache.
__device__ __forceinline__ float block_scale(const float* scales, int shift, int64_t row) {
  return ((const float __attribute__((address_space(4)))*)scales)[row >> shift];
}

template <bool NT, typename V, typename T>
__device__ __forceinline__ V load(const T* p) {
  const V* v = reinterpret_cast<const V*>(p);
  return NT ? __builtin_nontemporal_load(v) : *v;
}

// One wave's share of the keys and values of SUB tokens, in the layout that
// the loads give, and the operands made from it.  Token t of the share is row
// `t & 15` of group `t >> 4`; pk / pv point to each group's first row.
//
// NT: loads that leave the caches to others (see outgrows_cache()).
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
  // The keys as operands, and S = Q K^T from them, contraction step by step: a
  // token to each lane column, query rows 4 (l >> 4) + i.
  struct Keys {
    static constexpr int STEPS = D / 32;
    bf16x8 k[2][STEPS];

    __device__ __forceinline__ void add(int u, int s, const Query& q, f32x4& c) const {
      c = mfma_bf16(q.q[s], k[u][s], c);
    }
  };
  __device__ __forceinline__ Keys keys() const {
    Keys x;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int s = 0; s < D / 32; ++s) x.k[u][s] = __builtin_bit_cast(bf16x8, k[u][s]);
    return x;
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
  typedef typename Cache<D, bf16_t, NT>::Query Query;

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
  typedef typename Cache<D, bf16_t, NT>::Keys Keys;  // takes a Query of this layout too
  __device__ __forceinline__ Keys keys() const {
    Keys x;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int s = 0; s < D / 32; ++s) {
        const uint32_t a = k[u][s / 2][2 * (s & 1)], b = k[u][s / 2][2 * (s & 1) + 1];
        x.k[u][s] = as_op(widen_e4m3<false>(a), widen_e4m3<true>(a), widen_e4m3<false>(b), widen_e4m3<true>(b));
      }
    return x;
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
  struct Keys {
    static constexpr int STEPS = D / 4;
    f32x4 k[1][D / 16];

    __device__ __forceinline__ void add(int u, int s, const Query& q, f32x4& c) const {
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(q.q[s >> 2][s & 3], k[u][s >> 2][s & 3], c, 0, 0, 0);
    }
  };
  __device__ __forceinline__ Keys keys() const {
    Keys x;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) x.k[0][s] = k[0][s];
    return x;
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

}  // namespace
}  // namespace kda
