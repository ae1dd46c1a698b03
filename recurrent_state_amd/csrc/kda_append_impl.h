// What the appends to the paged cache share: loads and stores of 8 values, the
// rotation of a unit of 16, and the positions that it turns by.
#pragma once

#include <stddef.h>

#include "kda_pages.h"

namespace kda {
namespace {

typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(4))) float f32x4;

// NT: non-temporal, for calls that outgrow the caches.
template <bool NT, typename V>
__device__ __forceinline__ V get(const V* p) {
  return NT ? __builtin_nontemporal_load(p) : *p;
}
template <bool NT, typename V>
__device__ __forceinline__ void put(V* p, const V& x) {
  if (NT)
    __builtin_nontemporal_store(x, p);
  else
    *p = x;
}

// 8 values as fp32, and back.
template <bool NT>
__device__ __forceinline__ void load8(const bf16_t* p, float (&x)[8]) {
  const u32x4 w = get<NT>(reinterpret_cast<const u32x4*>(p));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}
template <bool NT>
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x4 w = get<NT>(reinterpret_cast<const f32x4*>(p) + h);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[4 * h + i] = w[i];
  }
}
template <bool NT>
__device__ __forceinline__ void store8(bf16_t* p, const float (&x)[8]) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){x[2 * i], x[2 * i + 1]}, bf16x2));
  put<NT>(reinterpret_cast<u32x4*>(p), w);
}
template <bool NT>
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  put<NT>(reinterpret_cast<f32x4*>(p), (f32x4){x[0], x[1], x[2], x[3]});
  put<NT>(reinterpret_cast<f32x4*>(p) + 1, (f32x4){x[4], x[5], x[6], x[7]});
}

// 8 values as e4m3, rounded to nearest even by the conversion.
__device__ __forceinline__ u32x2 e4m3_of(const float (&y)[8]) {  // of values in range
  int w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i], y[4 * i + 1], w[i], false);
    w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2], y[4 * i + 3], w[i], true);
  }
  return (u32x2){(uint32_t)w[0], (uint32_t)w[1]};
}
// x / scale so; the division is the IEEE one, so the stored bits are those of the
// formula.
template <bool NT>
__device__ __forceinline__ void store8_e4m3(uint8_t* p, const float (&x)[8], float scale) {
  int w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(to_range(x[4 * i] / scale), to_range(x[4 * i + 1] / scale), w[i], false);
    w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(to_range(x[4 * i + 2] / scale), to_range(x[4 * i + 3] / scale), w[i], true);
  }
  put<NT>(reinterpret_cast<u32x2*>(p), (u32x2){(uint32_t)w[0], (uint32_t)w[1]});
}

// The first values of the two chunks of 8 of unit w of a head: rotated units
// (n_rot of them) come first, chunks dim / 2 apart or neighbours.
struct Chunks {
  int c0, c1;
};
__device__ __forceinline__ Chunks chunks_of(const kda_rotation& rot, int n_rot, int w) {
  if (w < n_rot) {
    const int c0 = rot.start + (rot.pairs ? 16 * w : 8 * w);
    return Chunks{c0, c0 + (rot.pairs ? 8 : rot.dim >> 1)};
  }
  int c0 = 16 * (w - n_rot);
  if (n_rot > 0 && c0 >= rot.start) c0 += rot.dim;
  return Chunks{c0, c0 + 8};
}

// x holds the first members of 8 pairs and y the second, or, with `pairs`, pairs
// 0 to 3 and 4 to 7 interleaved.
__device__ __forceinline__ void rotate(float (&x)[8], float (&y)[8], const float (&c)[8], const float (&s)[8],
                                       bool pairs) {
  if (pairs) {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const float x0 = x[2 * n], x1 = x[2 * n + 1], y0 = y[2 * n], y1 = y[2 * n + 1];
      x[2 * n] = x0 * c[n] - x1 * s[n];
      x[2 * n + 1] = x1 * c[n] + x0 * s[n];
      y[2 * n] = y0 * c[4 + n] - y1 * s[4 + n];
      y[2 * n + 1] = y1 * c[4 + n] + y0 * s[4 + n];
    }
  } else {
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const float x0 = x[n], y0 = y[n];
      x[n] = x0 * c[n] - y0 * s[n];
      y[n] = y0 * c[n] + x0 * s[n];
    }
  }
}

// Cosines and sines of the 8 pairs of unit w at position p.
__device__ __forceinline__ void angles(const kda_rotation& rot, int64_t p, int w, float (&c)[8], float (&s)[8]) {
  const float* cs = rot.cos_sin + p * rot.dim + 8 * w;
  load8<false>(cs, c);
  load8<false>(cs + (rot.dim >> 1), s);
}

// A token's positions on the axes; bad: one is not in the table.
struct AxisPos {
  int32_t p0, p1, p2, p3;
  bool bad;

  // Selected by value: chosen by address, they would live in memory.
  __device__ __forceinline__ int32_t of(uint32_t a) const {
    const int32_t x0 = p0, x1 = p1, x2 = p2, x3 = p3;
    const int32_t lo = a & 1 ? x1 : x0, hi = a & 1 ? x3 : x2;
    return a & 2 ? hi : lo;
  }
};
__device__ __forceinline__ AxisPos axis_positions(const Axes& axes, const kda_rotation& rot, int64_t row) {
  const int64_t* p = axes.pos + row;
  // All are asked for at once; an axis that is not there stands for the first.
  const int64_t x0 = p[0], x1 = p[axes.n > 1 ? axes.stride : 0], x2 = p[axes.n > 2 ? 2 * axes.stride : 0],
                x3 = p[axes.n > 3 ? 3 * axes.stride : 0];
  const auto out = [&](int64_t x) { return x < 0 || x >= rot.max_pos; };
  return AxisPos{(int32_t)x0, (int32_t)x1, (int32_t)x2, (int32_t)x3, out(x0) || out(x1) || out(x2) || out(x3)};
}
// As angles(), each pair at its axis's position.  `of`: two bits for each pair.
// Units of one axis (of contiguous sections, most) read whole rows.
__device__ __forceinline__ void angles(const kda_rotation& rot, const AxisPos& at, uint32_t of, int w, float (&c)[8],
                                       float (&s)[8]) {
  if (of == (of & 3) * 0x5555u) {
    angles(rot, at.of(of & 3), w, c, s);
    return;
  }
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    const float* cs = rot.cos_sin + (int64_t)at.of(of >> 2 * n & 3) * rot.dim + 8 * w + n;
    c[n] = cs[0];
    s[n] = cs[rot.dim >> 1];
  }
}
// The axes of the pairs of unit w, from the kernel's arguments in memory (indexed
// as a parameter, the array would be copied to scratch).
template <typename Args>
__device__ __forceinline__ uint32_t axes_of_unit(int w) {
  typedef const char __attribute__((address_space(4))) * bytes;
  typedef const uint16_t __attribute__((address_space(4))) * words;
  return ((words)((bytes)__builtin_amdgcn_kernarg_segment_ptr() + offsetof(Args, axes) + offsetof(Axes, of)))[w];
}

}  // namespace
}  // namespace kda
