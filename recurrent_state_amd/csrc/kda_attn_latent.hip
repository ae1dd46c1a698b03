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
//   scores   S^T = K Q^T and their softmax.  One wave for each 16 query rows,
//            whose queries it holds (72 registers): the rows' maxima and sums
//            stay in its registers, and the probabilities go to the LDS as an
//            MFMA operand.
//   output   O^T += V^T P^T.  A wave has 64 of the 512 columns of all rows, or
//            128 where the other four waves make the scores (up to 64 rows; 64
//            or 128 registers), so a value is read from the LDS once.  V^T comes
//            from ds_read_b64_tr_b16, which hands lane l column l & 15 of four
//            rows.
//
// Between two barriers the waves score tile i + 1 and weigh tile i, while later
// tiles are on their way (LDS-direct loads, 16 bytes a lane).  So the two waves
// of a SIMD fill each other's waits: a form with the scores' contraction split
// over pairs of waves, which halves the key reads but needs a second barrier
// and an exchange in the LDS for every tile, took 3.2 us a tile of 128 rows.
//
// Measured: a tile of 128 rows takes 2.7 us on every CU (840 TFLOP/s; the MFMAs
// are busy for a third of it, and neither deeper LDS read-ahead nor loads
// spread over the products shortened it).  64 sequences of 4000 to 16000 tokens
// are read at 5.1 TB/s with 16 rows (126 us), 5.0 with 32 and 4.7 with 64; with
// 128 rows they take 212 us (730 TFLOP/s).
//
// LDS layout of a tile: 32 rows of 64 16-byte chunks (the values), then 32 rows
// of the last 8.  Chunk c of row r lies at c ^ f(r) in the first part, with
// f(r) = 2 r mod 16, xor 9 from row 8 on, and at c ^ (r / 2 % 8) in the second.
// A 16-byte read serves 16 lanes at a time, but not neighbours: lanes 0-3, 12-15
// and 20-27, then the other 16 of the half wave (counted as conflicts: with f(r)
// the bits of r rotated left, right for neighbours, 1024 cycles a tile).  So
// the key reads (eight rows of one chunk, the other eight of the next) and
// the transposed value reads (8 rows, two neighbouring chunks) touch every bank
// once, and a row's first part is one load of a wave, whose addresses are the
// row's and a constant of the lane.
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
constexpr int kRowBytes = kDk * 2;          // in the pages: 72 chunks of 16 bytes
constexpr int kMain = kDv * 2, kTail = kRowBytes - kMain;  // in the LDS: see above
constexpr int kTailAt = kTile * kMain, kBufBytes = kTile * kRowBytes;
constexpr int kSteps = kDk / 32;            // contraction steps

typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(1))) void global_void;

// By row of 16.
__device__ __forceinline__ int swizzle(int row) { return (row << 1 & 14) ^ (row >> 3 & 1) * 9; }
__device__ __forceinline__ int swizzle_tail(int row) { return row >> 1 & 7; }

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
  // their way (what the probabilities leave room for).
  constexpr int BUFS = RB == 8 ? 3 : 4, AHEAD = BUFS - 1;
  constexpr int kDepth = RB == 8 ? 4 : 12;
  constexpr int OUT = RB == 8 ? 8 : 4;      // waves that make the output: the last ones
  constexpr int kCols = kDv / OUT / 16;     // column tiles of such a wave
  __shared__ __attribute__((aligned(1024))) unsigned char lds[BUFS * kBufBytes];
  __shared__ u32x4 lds_p[2][RB][kWave];        // probabilities, of even and odd tiles
  __shared__ float lds_keep[2][RB][16];        // factors of the sums so far,
  __shared__ int32_t lds_grown[2][RB];         // where some are not one
  __shared__ f32x2 lds_ml[RB][16];             // at the end: maximum, sum

  const KvBatch& kb = a.kb;
  const int wave = uniform((int)threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int rb = blockIdx.y, worker = blockIdx.x, Hq = kb.s.Hq;
  Run<kTile> run(a, worker, worker == 0 && rb == 0 && wave == 0);
  const float x_scale = a.scale * kLog2e;

  // Byte offset in a tile of chunk c (below 16) of row `row`; this wave's
  // columns begin at chunk v_chunk after v_col bytes.  Lane constants are
  // computed where they are used (here()): registers are short.
  auto chunk_at = [](int row, int c) { return row * kMain + ((c ^ swizzle(row & 15)) << 4); };
  const int ow = wave - (kWaves - OUT);
  const int v_col = (OUT == 8 ? ow >> 1 : ow) * 256, v_chunk = OUT == 8 ? 8 * (ow & 1) : 0;

  while (run.tile < run.end) {
    const Seq& s = run.s;
    const int32_t tile = run.tile, first = run.first, stop = min(run.end, first + s.tiles);
    const int R = s.n * Hq, row0 = rb * RB * 16;
    if (row0 < R) {
      // The outputs [row block][column tile], and the queries: after them where a
      // wave holds both, else in the same registers.
      constexpr int Q0 = OUT == kWaves ? RB * kCols : 0;
      constexpr int HELD = RB * kCols > Q0 + kSteps ? RB * kCols : Q0 + kSteps;
      f32x4 held[HELD];
#pragma unroll
      for (int x = 0; x < HELD; ++x) held[x] = f32x4{};
      float m = -INFINITY, l = 0.f;  // of the rows that the wave scores
      const int my_row = row0 + 16 * wave + (here(lane) & 15);
      const int vis = my_row < R ? (int)max(s.pos + my_row / Hq, (int64_t)-1) : -1;  // the last token it sees

      const int n_tiles = s.end > 0 ? stop - tile : 0;
      const int tok0 = (s.lo & ~(kTile - 1)) + (tile - first) * kTile;
      const int all_lo = a.window > 0 ? max((int)(s.pos + s.n) - a.window, 0) : 0;
      auto whole = [&](int t0) { return t0 >= all_lo && t0 + kTile - 1 <= s.pos; };
      PageWalk walk(kb, s, run.b, 0);

      // Tile i into buffer i % BUFS: four rows of a group of 16 to a wave, and
      // eight of its rows' last chunks to two waves of each group.  Where some
      // row is outside the visible tokens, it gets a copy of the nearest visible
      // one, so that a probability of zero meets what some row sees anyway.
      const int t16 = 16 * (wave >> 2);
      const bool tails = (wave & 2) == 0;
      int32_t id = 0;  // the page entry of the tile to be loaded next
      if (n_tiles > 0) id = walk.entry(tok0 + t16);
      auto load = [&](int i) {
        const int tok = tok0 + i * kTile + t16, lane = here((int)threadIdx.x & 63);
        unsigned char* dst = lds + i % BUFS * kBufBytes;
        const unsigned char* base = static_cast<const unsigned char*>(kb.pages.k) + walk.row(tok, id) * kRowBytes;
        const uint32_t at = (lane ^ (8 * ((wave ^ wave >> 1) & 1) | (wave >> 1 & 1))) * 16;
        const int r = 8 * (wave & 1) + (lane >> 3);  // of the tails
        const uint32_t tail_at = kMain + ((lane & 7) ^ swizzle_tail(r)) * 16;
        auto get = [&](uint32_t offset, unsigned char* to) {
          __builtin_amdgcn_global_load_lds((global_void*)(base + offset), (lds_void*)to, 16, 0, 0);
        };
        unsigned char* rows = dst + wave * 4 * kMain;
        unsigned char* tail = dst + kTailAt + (2 * (wave >> 2) + (wave & 1)) * 8 * kTail;
        if (tok >= s.lo && tok + 16 <= s.end) {
          const uint32_t row = 4 * (wave & 3) * kRowBytes;
#pragma unroll
          for (int x = 0; x < 4; ++x) get((at ^ 32 * x) + (row + x * kRowBytes), rows + x * kMain);
          if (tails) get(r * kRowBytes + tail_at, tail);
        } else {
          const int from = min(max(tok, walk.lo), walk.hi);  // the token of the base row
          auto near = [&](int row) { return (uint32_t)(min(max(from + row, s.lo), s.end - 1) - from); };  // 0 to 15
#pragma unroll
          for (int x = 0; x < 4; ++x) get((at ^ 32 * x) + near(4 * (wave & 3) + x) * kRowBytes, rows + x * kMain);
          if (tails) get(near(r) * kRowBytes + tail_at, tail);
        }
        id = walk.entry(tok + kTile);
      };
      // Waits until tile i has landed; tiles up to `issued` are on their way.
      auto landed = [&](int i, int issued) {
        const int behind = issued - i;
        if (tails) {
          if (BUFS == 4 && behind >= 2)
            wait_loads<10>();
          else if (behind >= 1)
            wait_loads<5>();
          else
            wait_loads<0>();
        } else {
          if (BUFS == 4 && behind >= 2)
            wait_loads<8>();
          else if (behind >= 1)
            wait_loads<4>();
          else
            wait_loads<0>();
        }
      };

      // Scores and probabilities of tile i, for the waves that have rows.
      auto scores = [&](int i) {
        if (wave >= RB) return;
        const int t0 = tok0 + i * kTile, lane = here((int)threadIdx.x & 63), g = lane >> 4, row = lane & 15;
        const unsigned char* buf = lds + i % BUFS * kBufBytes;
        f32x4 p[2] = {f32x4{}, f32x4{}};
        // Key chunk 4 k + g of token group u; kDepth reads are ahead of their
        // products.  The order is fixed: the compiler's own has every product
        // wait for its read.
        auto key = [&](int n) {
          const int k = n >> 1, u = n & 1;
          const unsigned char* at =
              k < 16 ? buf + chunk_at(row, 4 * (k & 3) + g) + (k >> 2) * 256 + u * 16 * kMain
                     : buf + kTailAt + (16 * u + row) * kTail + ((4 * (k & 1) + g ^ swizzle_tail(row)) << 4);
          return *reinterpret_cast<const bf16x8*>(at);
        };
        bf16x8 keys[kDepth];
#pragma unroll
        for (int n = 0; n < kDepth; ++n) keys[n] = key(n);
#pragma unroll
        for (int n = 0; n < 2 * kSteps; ++n) {
          __builtin_amdgcn_sched_barrier(0);
          p[n & 1] = mfma_bf16(keys[n % kDepth], __builtin_bit_cast(bf16x8, held[Q0 + (n >> 1)]), p[n & 1]);
          if (n + kDepth < 2 * kSteps) keys[n % kDepth] = key(n + kDepth);
        }
        __builtin_amdgcn_sched_barrier(0);
        float top = -INFINITY;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) p[u][j] *= x_scale;
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
        lds_p[i & 1][wave][lane] = (u32x4){pack2(p[0][0], p[0][1]), pack2(p[0][2], p[0][3]), pack2(p[1][0], p[1][1]),
                                           pack2(p[1][2], p[1][3])};
        const bool grown = __ballot(keep != 1.f) != 0;
        if (grown && g == 0) lds_keep[i & 1][wave][lane] = keep;
        if (lane == 0) lds_grown[i & 1][wave] = grown;
      };

      auto output = [&](int i) {
        if (OUT < kWaves && ow < 0) return;
        const int t0 = tok0 + i * kTile, lane = here((int)threadIdx.x & 63);
        const unsigned char* buf = lds + i % BUFS * kBufBytes;
        const uint64_t grown = __ballot(lane < RB && lds_grown[i & 1][lane % RB] != 0);
        if (grown != 0) {
#pragma unroll
          for (int n = 0; n < RB; ++n)
            if (grown >> n & 1) {
              const float keep = lds_keep[i & 1][n][lane & 15];
#pragma unroll
              for (int c = 0; c < kCols; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j) held[n * kCols + c][j] *= keep;
            }
        }
        // A probability of zero must meet a finite value: look at the tokens
        // that only some rows see, in this wave's columns.
        bool odd = false;
        if (!whole(t0)) {
#pragma unroll
          for (int x = 0; x < kCols; ++x) {
            const int c = x * kWave + lane, j = t0 + c / (2 * kCols);
            const u32x4 v =
                *reinterpret_cast<const u32x4*>(buf + v_col + chunk_at(j - t0, v_chunk + c % (2 * kCols)));
            uint32_t peak = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) peak = max(peak, max(v[e] << 16 & 0x7fff0000u, v[e] & 0x7fff0000u));
            odd |= (peak >= 0x7f800000u) & (j >= s.lo) & (j < s.end) & ((j < all_lo) | (j > s.pos));
          }
        }
        u32x4 vt[kCols];
        const int v0 = v_col + chunk_at(4 * (lane >> 4) + (lane >> 2 & 3), v_chunk + (lane >> 1 & 1)) + (lane & 1) * 8;
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const unsigned char* at = buf + (v0 ^ c * 32);
          const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at));
          const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 16 * kMain)));
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
            const unsigned char* row = buf + v_col + (lane_ >> 4 & 1) * 8;
#pragma unroll
            for (int n = 0; n < RB; ++n) {
              const int r = 16 * n + (lane_ & 15);
              const bool sees = r >= r_from && r < r_to;
              __builtin_amdgcn_sched_barrier(0);  // one block's terms at a time: registers
              const float x = bf16_lo(reinterpret_cast<const uint16_t*>(&lds_p[i & 1][n][4 * (at & 12) + (lane_ & 15)])[e]);
#pragma unroll
              for (int c = 0; c < kCols; ++c) {
                const u32x2 v = *reinterpret_cast<const u32x2*>(row + chunk_at(at, v_chunk + 2 * c + (lane_ >> 5)));
                const float y[4] = {bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]), bf16_hi(v[1])};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const float o = held[n * kCols + c][k];
                  held[n * kCols + c][k] = sees ? o + x * y[k] : o;
                }
              }
            }
          }
        }
        auto weights = [&](int n) { return __builtin_bit_cast(bf16x8, lds_p[i & 1][n][lane]); };
        bf16x8 w[2] = {weights(0), bf16x8{}};
        if constexpr (RB > 1) w[1] = weights(1);
#pragma unroll
        for (int n = 0; n < RB; ++n) {
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            held[n * kCols + c] = mfma_bf16(__builtin_bit_cast(bf16x8, vt[c]), w[n & 1], held[n * kCols + c]);
          if (n + 2 < RB) w[n & 1] = weights(n + 2);
        }
      };

      // Tile i is weighed while tile i + 1 is scored; the buffer that a new
      // tile goes to was weighed before the barrier.
      int issued = -1;
      for (; issued + 1 < min(AHEAD, n_tiles);) load(++issued);
      // The queries, behind the first tiles' loads.
      const int q_row = row0 + 16 * wave + (here(lane) & 15);
      const bf16_t* q_at = static_cast<const bf16_t*>(a.q.p) + (int64_t)(s.row0 + q_row / Hq) * a.q.stride +
                           q_row % Hq * kDk + 8 * (here(lane) >> 4);
      if (wave < RB && q_row < R) {
#pragma unroll
        for (int k = 0; k < kSteps; ++k) held[Q0 + k] = *reinterpret_cast<const f32x4*>(q_at + 32 * k);
      }
      for (int i = -1; i < n_tiles; ++i) {
        if (i + 1 < n_tiles) landed(i + 1, issued);
        lds_barrier();
        // With 128 rows every wave does both: half of them (one of each SIMD)
        // begin with the scores, which are bound by LDS reads, the others with
        // the output, bound by the MFMAs.
        if (wave < 4 && i + 1 < n_tiles) scores(i + 1);
        if (i >= 0) {
          if (i + AHEAD < n_tiles) load(++issued);
          output(i);
        }
        if (wave >= 4 && i + 1 < n_tiles) scores(i + 1);
      }

      // Sums to the rows' own lanes, and out.
      const bool complete = tile == first && stop == first + s.tiles;
      const int64_t piece = piece_index(a, worker, tile > first ? 0 : 1, 0, rb);
      const bool bad = __syncthreads_or(walk.bad);
      if (bad && threadIdx.x == 0) set_err(kb.dev_err, KDA_DEV_ERR_PAGE);
      if (wave < RB) {
        const float sum = pair_sum32(pair_sum16(l));
        if (lane < 16) lds_ml[wave][lane] = (f32x2){m, sum};
      }
      __syncthreads();
      const int c0 = ow * (16 * kCols) + 4 * (here(lane) >> 4);
#pragma unroll
      for (int n = 0; n < RB; ++n) {
        const int in = 16 * n + (here(lane) & 15), r = row0 + in;
        if (r >= R || ow < 0) continue;
        const f32x2 ml = lds_ml[n][in & 15];
        if (!complete) {
          const int64_t row = piece * a.rows + in;
#pragma unroll
          for (int c = 0; c < kCols; ++c) store4(a.piece_o + row * kDv + c0 + 16 * c, held[n * kCols + c]);
          if (c0 == 0) a.piece_ml[row] = (f32x2){ml[0], bad ? -1.f : ml[1]};
        } else if (!bad) {
          const float inv = s.pos + r / Hq < 0 ? 0.f : 1.f / ml[1];  // 0 / 0 where every score is -inf
          const int64_t row = (int64_t)(s.row0 + r / Hq) * Hq + r % Hq;
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            f32x4 x = held[n * kCols + c];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] *= inv;
            store4(static_cast<bf16_t*>(a.o) + row * kDv + c0 + 16 * c, x);
          }
          if (a.lse && c0 == 0) a.lse[row] = (ml[0] + __log2f(ml[1])) * kLn2;
        }
      }
      lds_barrier();
    }
    run.next(stop);
  }
}

// Rows of a workgroup.  Large blocks read a cached row from the LDS and from
// memory once for more rows; small ones bring more workgroups to a short cache,
// begin sooner and leave less to write and join.  So the block grows by two
// with every factor of four in rows x tokens (of the longest caches that the
// page table has room for), and further while there would be more than 64
// blocks of sequences, which leaves each fewer than four workgroups.  Measured
// in us with 16 / 32 / 64 / 128 rows, 128 rows in all: one sequence of 500
// tokens 17.2 / 19.2 / 22.7 / 31.3, of 32000 34.6 / 30.6 / 36.8 / 43.5; 8 of
// 8000 77 / 52 / 45 / 55; 64 of 2000 151 / 100 / 81 / 73.  Up to 16 rows a
// block of 16 is 1-5% ahead of one of 32 everywhere.
Split split_of(const kda_kv_shape& s, int32_t page_size, int32_t max_pages) {
  const int rows = s.T * s.Hq;
  const int64_t work = (int64_t)s.B * max_pages * page_size * rows;
  // A piece more costs much here, so one a worker from two workers to a sequence
  // on: 64 of up to 2000 tokens with 128 rows in 68.6 us, where the list of
  // tiles takes 71.6, and 81.1 with a beginning counted as three tiles, not eight.
  Split d{kTile, 16, 0, 0, 4, 8, 2};
  for (int64_t most = (int64_t)1 << 20; d.rows < 128 && d.rows < rows; d.rows *= 2, most *= 4) {
    d.row_blocks = (rows + d.rows - 1) / d.rows;
    if (work <= most && (int64_t)d.row_blocks * s.B <= 64) break;
  }
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
  return d.rows == 16   ? run<1>(a, st)
         : d.rows == 32 ? run<2>(a, st)
         : d.rows == 64 ? run<4>(a, st)
                        : run<8>(a, st);
}

}  // namespace kda
