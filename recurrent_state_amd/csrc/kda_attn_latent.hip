// Attention of a sequence's new tokens over a latent cache: one row of 576
// values per token is the key of every query head, its first 512 values the
// value.
//
// With R = T Hq query rows a cached row of 1152 bytes meets 2176 R flops:
// bound by memory up to about 64 rows, by the matrix units and the LDS beyond.
// So unlike the grouped kernel this one stages rows in the LDS, once for all
// its waves and for both uses.  A workgroup of eight waves takes up to 128
// query rows and walks its run in tiles of 32 tokens:
//
//   scores   S^T = K Q^T.  A wave has 16 or 32 query rows, half of the
//            contraction (every other 32 values) and, with few rows, half of
//            the tokens; its queries stay in registers (36 or 72).  The halves
//            go to the LDS as they leave the MFMA.
//   softmax  a wave takes 16 rows: sums the halves, moves the maximum and
//            leaves the probabilities in the LDS as an MFMA operand.
//   output   O^T += V^T P^T.  A wave has 64 of the 512 columns of all rows (32
//            to 128 registers), so a value is read from the LDS once.  V^T
//            comes from ds_read_b64_tr_b16, which hands lane l column l & 15
//            of four rows.
//
// Scores of tile i + 1 and output of tile i are one phase between barriers,
// the softmax the other; later tiles are on their way meanwhile (LDS-direct
// loads, 16 bytes a lane).  The split by contraction and columns is what keeps
// a wave within 256 registers, two waves to a SIMD; waves with 32 whole rows
// each (256 + 144 registers) spilled.
//
// LDS layout: 16-byte chunk c of row r lies at chunk (c & ~7) | ((c ^ f(r)) &
// 7) of its row, f(r) = 2 (r / 2 % 4) + r / 8 % 2: the key reads (16 rows, one
// chunk) and the transposed value reads (8 rows, two neighbouring chunks) both
// touch every bank once.
//
// The outputs are scaled only when a row's maximum has grown past 2^8 times
// the one in use: probabilities stay below 2^8 and their roundings are
// relative, so nothing is lost.  Rounding as in the grouped kernel: everything
// fp32, probabilities bf16.

#include "kda_attn_impl.h"

namespace kda {
namespace {

constexpr int kDk = 576, kDv = 512;
constexpr int kWaves = 8, kTile = 32;       // tokens
constexpr int kRowBytes = kDk * 2;          // 72 chunks of 16 bytes
constexpr int kBufBytes = kTile * kRowBytes;
constexpr int kHalf = 16 * kRowBytes;       // 16 rows
constexpr int kSteps = kDk / 64;            // contraction steps of a wave
constexpr int kCols = kDv / kWaves / 16;    // column tiles of a wave
constexpr int kLoads = 9;                   // LDS-direct loads of a loading wave and tile

typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(1))) void global_void;

__device__ __forceinline__ int swizzle(int row) { return (row >> 1 & 3) << 1 | (row >> 3 & 1); }

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

// RB blocks of 16 query rows.
template <int RB>
__global__ void __launch_bounds__(kWaves * kWave, 2) latent_kernel(AttnArgs a) {
  // Tiles in the LDS: one being scored, one being weighed, the others on
  // their way (what the scores and probabilities leave room for).
  constexpr int BUFS = RB == 2 ? 4 : 3, AHEAD = BUFS - 1;
  constexpr int QB = RB == 8 ? 2 : 1;   // row blocks whose scores a wave makes
  constexpr int US = RB == 2 ? 1 : 2;   // 16-token groups of them
  __shared__ __attribute__((aligned(1024))) unsigned char lds[BUFS * kBufBytes];
  __shared__ f32x4 lds_s[2][RB][2][kWave];     // scores: [contraction half][row block][16 tokens]
  __shared__ u32x4 lds_p[RB][kWave];           // probabilities
  __shared__ float lds_keep[RB][16];           // factor of the sums so far
  __shared__ f32x2 lds_ml[RB][16];             // at the end: maximum, sum

  const KvBatch& kb = a.kb;
  const int wave = uniform((int)threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int rb = blockIdx.y, worker = blockIdx.x, Hq = kb.s.Hq;
  const Run run = find_run<kTile>(a, worker, worker == 0 && rb == 0 && wave == 0);
  const float x_scale = a.scale * kLog2e;
  // The wave's part of the scores.
  const int half = wave & 1, qb = (RB == 2 ? wave >> 2 : wave >> 1) * QB, us = RB == 2 ? wave >> 1 & 1 : 0;

  // Byte offsets in a tile: key chunk 4 half + g of row `col` (of the wave's
  // tokens), and the wave's value chunks of row 4 g + col / 4.  Computed where
  // they are used (here()), as most lane constants below: registers are short.
  auto k_at = [&] {
    const int lane = here((int)threadIdx.x & 63), row = lane & 15;
    return us * kHalf + row * kRowBytes + (((4 * half + (lane >> 4)) ^ swizzle(row)) & 7) * 16;
  };
  auto v_at = [&](int lane) {
    const int row = 4 * (lane >> 4) + (lane >> 2 & 3);
    return wave * 128 + row * kRowBytes + ((lane >> 1 & 1) ^ swizzle(row)) * 16 + (lane & 1) * 8;
  };

  int64_t tile = run.tile, first = run.first;
  for (int b = run.b; tile < run.end && b < kb.s.B; ++b) {
    const Seq s = uniform_seq<kTile>(a, b);
    if (s.tiles == 0) continue;
    const int64_t stop = min(run.end, first + s.tiles);
    const int R = s.n * Hq, row0 = rb * RB * 16;
    if (row0 < R) {
      bf16x8 q[QB][kSteps];
#pragma unroll
      for (int n = 0; n < QB; ++n) {
        const int r = row0 + 16 * (qb + n) + (here(lane) & 15);
        const bf16_t* p = static_cast<const bf16_t*>(a.q.p) + (int64_t)(s.row0 + r / Hq) * a.q.stride + r % Hq * kDk +
                          32 * half + 8 * (here(lane) >> 4);
#pragma unroll
        for (int k = 0; k < kSteps; ++k) q[n][k] = r < R ? *reinterpret_cast<const bf16x8*>(p + 64 * k) : bf16x8{};
      }
      f32x4 out[RB][kCols];
#pragma unroll
      for (int n = 0; n < RB; ++n)
#pragma unroll
        for (int c = 0; c < kCols; ++c) out[n][c] = f32x4{};
      float m = -INFINITY, l = 0.f;  // of the rows whose softmax the wave makes
      const int my_row = row0 + 16 * wave + (here(lane) & 15);
      const int vis = my_row < R ? (int)max(s.pos + my_row / Hq, (int64_t)-1) : -1;  // the last token it sees

      const int n_tiles = s.end > 0 ? (int)(stop - tile) : 0;
      const int tok0 = (s.lo & ~(kTile - 1)) + (int)(tile - first) * kTile;
      const int all_lo = a.window > 0 ? max((int)(s.pos + s.n) - a.window, 0) : 0;
      auto whole = [&](int t0) { return t0 >= all_lo && t0 + kTile - 1 <= s.pos; };
      PageWalk walk(kb, s, b, 0);

      // Tile i into buffer i % BUFS.  Rows outside the visible tokens get a
      // copy of the nearest visible one, so that a probability of zero meets
      // what some row sees anyway.
      const int t16 = 16 * (wave >> 1 & 1);
      int32_t id = n_tiles > 0 ? walk.entry(tok0 + t16) : 0;  // of the tile to be loaded next
      auto load = [&](int i) {
        if (wave >= 4) return;
        const int tok = tok0 + i * kTile, at = tok + t16;
        const unsigned char* base = static_cast<const unsigned char*>(kb.pages.k) + walk.row(at, id) * kRowBytes;
        unsigned char* dst = lds + i % BUFS * kBufBytes + wave * (8 * kRowBytes);
        const int from = min(max(at, walk.lo), walk.hi);  // the token of the base row
        // Load k of a wave's 8 rows writes 64 chunks from chunk 64 k on; this
        // lane's comes from row k - (lane < 8 k) of them.
        const int lane_ = here(lane), r8 = 8 * (wave & 1);
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const int r = r8 + k - (lane_ < 8 * k), c = lane_ - 8 * k + (lane_ < 8 * k ? 72 : 0);
          const int row = min(max(from + r, s.lo), s.end - 1) - from;
          const uint32_t off = row * kRowBytes + ((c & ~7) | ((c ^ swizzle(r)) & 7)) * 16;
          __builtin_amdgcn_global_load_lds((global_void*)(base + off), (lds_void*)(dst + k * 1024), 16, 0, 0);
        }
        id = walk.entry(at + kTile);
      };
      // Waits until tile i has landed; tiles up to `issued` are on their way.
      auto landed = [&](int i, int issued) {
        if (BUFS == 4 && issued - i >= 2)
          wait_loads<2 * kLoads>();
        else if (issued - i >= 1)
          wait_loads<kLoads>();
        else
          wait_loads<0>();
      };

      auto scores = [&](int i) {
        const unsigned char* buf = lds + i % BUFS * kBufBytes + k_at();
        f32x4 x[QB][US];
#pragma unroll
        for (int n = 0; n < QB; ++n)
#pragma unroll
          for (int u = 0; u < US; ++u) x[n][u] = f32x4{};
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
#pragma unroll
          for (int u = 0; u < US; ++u) {
            const bf16x8 key = *reinterpret_cast<const bf16x8*>(buf + k * 128 + u * kHalf);
#pragma unroll
            for (int n = 0; n < QB; ++n) x[n][u] = mfma_bf16(key, q[n][k], x[n][u]);
          }
#pragma unroll
        for (int n = 0; n < QB; ++n)
#pragma unroll
          for (int u = 0; u < US; ++u) lds_s[half][qb + n][us + u][lane] = x[n][u];
      };

      auto softmax = [&](int i) {
        if (wave >= RB) return;
        const int t0 = tok0 + i * kTile, lane = here((int)threadIdx.x & 63), g = lane >> 4;
        f32x4 p[2];
        float top = -INFINITY;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const f32x4 x = lds_s[0][wave][u][lane], y = lds_s[1][wave][u][lane];
#pragma unroll
          for (int j = 0; j < 4; ++j) p[u][j] = (x[j] + y[j]) * x_scale;
        }
        if (!whole(t0)) {
          const int low = a.window > 0 ? vis - a.window : -1;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int tok = t0 + 16 * u + 4 * g + j;
              p[u][j] = tok <= vis && tok > low ? p[u][j] : -INFINITY;
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) top = fmaxf(top, p[u][j]);
        top = max_over_rows(top);
        float keep = 1.f;
        if (top > m + 8.f) {
          keep = exp2_(m - top);
          m = top;
          l *= keep;
        }
        const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            p[u][j] = exp2_(p[u][j] - mu);
            l += p[u][j];
          }
        lds_p[wave][lane] = (u32x4){pack2(p[0][0], p[0][1]), pack2(p[0][2], p[0][3]), pack2(p[1][0], p[1][1]),
                                    pack2(p[1][2], p[1][3])};
        if (g == 0) lds_keep[wave][lane] = keep;
      };

      auto output = [&](int i) {
        const int t0 = tok0 + i * kTile, lane = here((int)threadIdx.x & 63);
        const unsigned char* buf = lds + i % BUFS * kBufBytes;
#pragma unroll
        for (int n = 0; n < RB; ++n) {
          const float keep = lds_keep[n][lane & 15];
          if (__ballot(keep != 1.f) != 0) {
#pragma unroll
            for (int c = 0; c < kCols; ++c)
#pragma unroll
              for (int j = 0; j < 4; ++j) out[n][c][j] *= keep;
          }
        }
        // A probability of zero must meet a finite value: look at the tokens
        // that only some rows see, in this wave's columns.
        bool odd = false;
        if (!whole(t0)) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int j = t0 + 8 * x + (lane >> 3);
            const u32x4 v = *reinterpret_cast<const u32x4*>(buf + (j - t0) * kRowBytes + wave * 128 + (lane & 7) * 16);
            uint32_t peak = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) peak = max(peak, max(v[e] << 16 & 0x7fff0000u, v[e] & 0x7fff0000u));
            odd |= (peak >= 0x7f800000u) & (j >= s.lo) & (j < s.end) & ((j < all_lo) | (j > s.pos));
          }
        }
        u32x4 vt[kCols];
        const int v0 = v_at(lane);
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const unsigned char* at = buf + (v0 ^ c * 32);
          const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at));
          const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + kHalf)));
          vt[c] = (u32x4){x[0], x[1], y[0], y[1]};
        }
        if (__ballot(odd) != 0) {
          // Such tokens count here, for the rows that see them, and not below.
          u32x4 keep;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = t0 + 16 * (i >> 1) + 4 * (here(lane) >> 4) + 2 * (i & 1);
            keep[i] = (j >= all_lo && j <= s.pos ? 0xffffu : 0u) | (j + 1 >= all_lo && j < s.pos ? 0xffff0000u : 0u);
          }
#pragma unroll
          for (int c = 0; c < kCols; ++c) vt[c] &= keep;
          for (int j = max(t0, s.lo); j < min(t0 + kTile, s.end); ++j) {
            if (j >= all_lo && j <= s.pos) continue;
            const int at = j - t0, e = (at & 3) + (at >> 4) * 4, lane_ = here(lane);
            // The rows that see token j: those of new tokens j - pos and on,
            // up to the one whose window ends with it.
            const int r_from = max(j - (int)s.pos, 0) * Hq - row0;
            const int r_to = a.window > 0 ? (int)min((int64_t)s.n, j - s.pos + a.window) * Hq - row0 : R - row0;
            const unsigned char* row = buf + at * kRowBytes + wave * 128 + (lane_ >> 4 & 1) * 8;
#pragma unroll
            for (int n = 0; n < RB; ++n) {
              const int r = 16 * n + (lane_ & 15);
              const bool sees = r >= r_from && r < r_to;
              __builtin_amdgcn_sched_barrier(0);  // one block's terms at a time: registers
              const float x = bf16_lo(reinterpret_cast<const uint16_t*>(&lds_p[n][4 * (at & 12) + (lane_ & 15)])[e]);
#pragma unroll
              for (int c = 0; c < kCols; ++c) {
                const u32x2 v = *reinterpret_cast<const u32x2*>(row + ((2 * c + (lane_ >> 5)) ^ swizzle(at & 15)) * 16);
                const float y[4] = {bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]), bf16_hi(v[1])};
#pragma unroll
                for (int k = 0; k < 4; ++k) out[n][c][k] = sees ? out[n][c][k] + x * y[k] : out[n][c][k];
              }
            }
          }
        }
#pragma unroll
        for (int n = 0; n < RB; ++n) {
          const bf16x8 w = __builtin_bit_cast(bf16x8, lds_p[n][lane]);
#pragma unroll
          for (int c = 0; c < kCols; ++c) out[n][c] = mfma_bf16(__builtin_bit_cast(bf16x8, vt[c]), w, out[n][c]);
        }
      };

      // Tile i is being weighed while tile i + 1 is scored; the buffer that a
      // new tile goes to was weighed before the last barrier but one.
      int issued = -1;
      for (; issued + 1 < min(AHEAD, n_tiles);) load(++issued);
      for (int i = -1; i < n_tiles; ++i) {
        if (i + 1 < n_tiles) landed(i + 1, issued);
        lds_barrier();
        if (i >= 0) {
          if (i + AHEAD < n_tiles) load(++issued);
          output(i);
        }
        if (i + 1 < n_tiles) {
          scores(i + 1);
          lds_barrier();
          softmax(i + 1);
        }
      }

      // Sums to the rows' own lanes, and out.
      const bool complete = tile == first && stop == first + s.tiles;
      const int64_t piece = piece_index(a, worker, tile > first ? 0 : 1, 0, rb);
      const bool bad = __syncthreads_or(walk.bad);
      if (threadIdx.x == 0) {
        if (bad) set_err(kb.dev_err, KDA_DEV_ERR_PAGE);
        if (!complete) a.piece_bad[piece] = bad;
      }
      if (wave < RB) {
        const float sum = pair_sum32(pair_sum16(l));
        if (lane < 16) lds_ml[wave][lane] = (f32x2){m, sum};
      }
      __syncthreads();
      const int c0 = wave * (16 * kCols) + 4 * (here(lane) >> 4);
#pragma unroll
      for (int n = 0; n < RB; ++n) {
        const int in = 16 * n + (here(lane) & 15), r = row0 + in;
        if (r >= R) continue;
        const f32x2 ml = lds_ml[n][in & 15];
        if (!complete) {
          const int64_t row = piece * a.rows + in;
#pragma unroll
          for (int c = 0; c < kCols; ++c) store4(a.piece_o + row * kDv + c0 + 16 * c, out[n][c]);
          if (c0 == 0) a.piece_ml[row] = ml;
        } else if (!bad) {
          const float inv = ml[1] == 0.f ? 0.f : 1.f / ml[1];
          const int64_t row = (int64_t)(s.row0 + r / Hq) * Hq + r % Hq;
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            f32x4 x = out[n][c];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] *= inv;
            store4(static_cast<bf16_t*>(a.o) + row * kDv + c0 + 16 * c, x);
          }
          if (a.lse && c0 == 0) a.lse[row] = (ml[0] + __log2f(ml[1])) * kLn2;
        }
      }
      __syncthreads();
    }
    first += s.tiles;
    tile = stop;
  }
}

Split split_of(const kda_kv_shape& s, int32_t page_size, int32_t max_pages) {
  const int rows = s.T * s.Hq;
  Split d{kTile, rows <= 32 ? 32 : rows <= 64 ? 64 : 128, 0, 0, 4};
  d.row_blocks = (rows + d.rows - 1) / d.rows;
  d.workers = workers_of(s, 256, d, page_size, max_pages);  // one workgroup to a CU: its LDS is full
  return d;
}

template <int RB>
hipError_t run(const AttnArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((latent_kernel<RB>), dim3(a.workers, a.row_blocks), dim3(kWaves * kWave), 0, st, a);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : run_join<kDv, bf16_t>(a, st);
}

}  // namespace

size_t latent_workspace_bytes(const kda_kv_shape& s, int32_t page_size, int32_t max_pages) {
  return workspace_of(s, split_of(s, page_size, max_pages)).total;
}

hipError_t launch_attn_latent(const KvBatch& b, KvRows q, float scale, int32_t window, void* o, float* lse,
                              void* workspace, hipStream_t st) {
  const Split d = split_of(b.s, b.pages.page_size, b.max_pages);
  const AttnArgs a = make_args(b, q, scale, window, o, lse, workspace, d);
  return d.rows == 32 ? run<2>(a, st) : d.rows == 64 ? run<4>(a, st) : run<8>(a, st);
}

}  // namespace kda
