// Appending to e4m3 pages whose scales go by blocks of tokens.
//
// A block's new scale needs the largest of all its new values before the first
// is stored, so the work is cut along the blocks: a workgroup takes a block's
// new tokens ("item") for one head of keys, values or queries ("kind"; queries
// are only rotated), or for several where few tokens make few rows.  A group of
// W waves holds 16 W rows of a head in registers, 16 values to a lane, laid out
// as in kda_pages.hip; the maximum is exchanged by lane swaps and, for W > 1,
// through the LDS.  Calls that bring more than 256 tokens to a block read them
// twice.
//
// The host knows neither lengths nor positions: the grid has an item for every
// block that well-formed ranges can touch, each finds its sequence by a scan of
// the sequences' block counts, 64 at a time, and those past the last end there.

#include "kda_append_impl.h"
#include "kda_blocks.h"

namespace kda {
namespace {

struct BlocksArgs {
  KvBatch kb;
  BlockScales scales;
  KvRows k, v, q;
  void* q_out;
  int64_t q_out_stride;
  kda_rotation rot;
  int32_t kinds;  // kv heads of keys, then of values, then query heads
  Axes axes;
};

// The new tokens of a sequence that have places: row0 + i at place pos + i for
// places [first, end), and the blocks that these touch.
struct Places {
  int32_t row0;
  int64_t pos;
  int32_t first, end, blocks;
  int32_t err;
};
__device__ __forceinline__ Places places_of(const BlocksArgs& a, int b) {
  const KvBatch& kb = a.kb;
  const int64_t pos = kb.pos[b];  // asked for together with the token range
  const SeqRows sr = seq_rows(kb, b);
  Places s{sr.row0, pos, 0, 0, 0, sr.bad ? KDA_DEV_ERR_TOKENS : 0};
  if (sr.n == 0) return s;
  // Outside of +-2^30 no token of the sequence has a place.
  const int64_t p = min(max(pos, -((int64_t)1 << 31)), (int64_t)1 << 31), past = p + sr.n;
  int64_t end = past;
  if (a.rot.cos_sin && !a.axes.n) end = min(end, max((int64_t)a.rot.max_pos, p));
  if (p < 0 || end < past) s.err |= KDA_DEV_ERR_POS;
  const int64_t limit = (int64_t)kb.max_pages << kb.page_shift;
  if (end > limit && end > p) s.err |= KDA_DEV_ERR_PAGE;
  end = min(end, limit);
  s.first = (int32_t)min(max(p, (int64_t)0), limit);
  if (end <= s.first) return s;
  s.end = (int32_t)end;
  s.blocks = ((s.end - 1) >> a.scales.shift) - (s.first >> a.scales.shift) + 1;
  return s;
}

// One block's part of a sequence: places [lo, hi), whose block begins at `begin`.
struct Item {
  int b;
  int32_t row0, lo, hi, begin;
  int64_t pos;
};
// Called by a whole wave; false: there is no item `item`.
__device__ __forceinline__ bool find_item(const BlocksArgs& a, int item, Item& it) {
  const int lane = threadIdx.x & 63, B = a.kb.s.B;
  int before = 0;
  for (int c = 0; c < B; c += kWave) {
    const Places s = c + lane < B ? places_of(a, c + lane) : Places{};
    const int upto = wave_scan(s.blocks), sum = __builtin_amdgcn_readlane(upto, kWave - 1);
    if (before + sum > item) {
      const int at = __ffsll((unsigned long long)__ballot(before + upto > item)) - 1;
      const int nth = item - before - __builtin_amdgcn_readlane(upto - s.blocks, at);
      const int first = __builtin_amdgcn_readlane(s.first, at), end = __builtin_amdgcn_readlane(s.end, at);
      it.b = c + at;
      it.row0 = __builtin_amdgcn_readlane(s.row0, at);
      it.pos = (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(s.pos >> 32), at) << 32 |
                         (uint32_t)__builtin_amdgcn_readlane((int)s.pos, at));
      it.begin = ((first >> a.scales.shift) + nth) << a.scales.shift;
      it.lo = max(first, it.begin);
      it.hi = min(end, it.begin + (1 << a.scales.shift));
      return true;
    }
    before += sum;
  }
  return false;
}

// W waves to a (block, head); NW waves to a workgroup.
template <int D, int W, bool NT, bool AXES>
__global__ void __launch_bounds__(64 * (W > 4 ? W : 4)) append_blocks_kernel(BlocksArgs a) {
  constexpr int NW = W > 4 ? W : 4;
  constexpr int LPR = D / 16, RPP = kWave / LPR, PASSES = 16 / RPP;  // lanes to a row, rows of a wave's pass
  __shared__ uint32_t lds_max[NW];
  const KvBatch& kb = a.kb;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int part = wave % W, kind = blockIdx.y * (NW / W) + wave / W;
  const bool is_key = kind < kb.s.Hkv, is_value = !is_key && kind < 2 * kb.s.Hkv;
  const bool idle = kind >= a.kinds;
  const int h = is_key ? kind : is_value ? kind - kb.s.Hkv : kind - 2 * kb.s.Hkv;
  const int w = lane % LPR, n_rot = a.rot.cos_sin ? a.rot.dim >> 4 : 0;
  const bool turn = !is_value && w < n_rot;
  const Chunks c = is_value ? Chunks{16 * w, 16 * w + 8} : chunks_of(a.rot, n_rot, w);
  const KvRows& rows = is_key ? a.k : is_value ? a.v : a.q;
  const bf16_t* const src = static_cast<const bf16_t*>(rows.p) + h * D;
  const bool names = blockIdx.y == 0 && wave < W;  // of the waves of an item's rows, those that name errors

  if (names && wave == 0 && blockIdx.x == 0)
    for (int b = lane; b < kb.s.B; b += kWave) {
      const int err = places_of(a, b).err;
      if (err) set_err(kb.dev_err, err);
    }
  // The grid covers all items but where ranges overlap.
  Item it;
  for (int item = blockIdx.x; find_item(a, item, it); item += gridDim.x) {
    const int32_t page = kb.table[(int64_t)it.b * kb.max_pages + (it.begin >> kb.page_shift)];
    const int chunks = W < 16 ? 1 : (it.hi - it.lo + 16 * W - 1) / (16 * W);  // see by_rows()
    uint32_t m = 0;
    float x[PASSES][8], y[PASSES][8];
    bool live[PASSES];
    auto row_of = [&](int chunk, int pass) { return it.lo + (chunk * W + part) * 16 + pass * RPP + lane / LPR; };
    auto load = [&](int chunk) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const int p = row_of(chunk, i);
        live[i] = p < it.hi && !idle;
        if (!live[i]) continue;
        const int64_t row = it.row0 + (p - it.pos);
        load8<NT>(src + row * rows.stride + c.c0, x[i]);
        load8<NT>(src + row * rows.stride + c.c1, y[i]);
        float cc[8], ss[8];
        if constexpr (AXES) {
          const AxisPos at = axis_positions(a.axes, a.rot, row);
          if (at.bad) {
            if (names && w == 0) set_err(kb.dev_err, KDA_DEV_ERR_POS);
            live[i] = false;
            continue;
          }
          if (turn) angles(a.rot, at, axes_of_unit<BlocksArgs>(w), w, cc, ss);
        } else if (turn) {
          angles(a.rot, p, w, cc, ss);
        }
        if (turn) rotate(x[i], y[i], cc, ss, a.rot.pairs);
      }
    };
    const bool bad = page < 0 || page >= kb.pages.n_pages;
    if (bad && names && lane == 0) set_err(kb.dev_err, KDA_DEV_ERR_PAGE);
    if (bad) continue;  // the whole workgroup agrees
    const bool stored = is_key || is_value;
    const int64_t head = (int64_t)page * kb.s.Hkv + h;
    float* const scale =
        (is_key ? a.scales.k : a.scales.v) + (head << (kb.page_shift - a.scales.shift)) +
        ((it.begin & (kb.pages.page_size - 1)) >> a.scales.shift);
    uint8_t* const dst = static_cast<uint8_t*>(is_key ? kb.pages.k : kb.pages.v) +
                         ((head << kb.page_shift) + (it.begin & (kb.pages.page_size - 1))) * D;
    const bool joins = stored && !idle && it.lo > it.begin;
    const float old = joins ? *scale : 0.f;
    for (int chunk = 0; chunk < chunks && (stored || chunks == 1); ++chunk) {
      load(chunk);
#pragma unroll
      for (int i = 0; i < PASSES; ++i)
        if (live[i])
#pragma unroll
          for (int n = 0; n < 8; ++n) m = max(m, max(finite_bits(x[i][n]), finite_bits(y[i][n])));
    }
    m = wave_max(m);
    if (W > 1) {
      __syncthreads();  // the item before has been read
      if (lane == 0) lds_max[wave] = m;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < W; ++i) m = max(m, lds_max[wave - part + i]);
    }
    uint32_t s = scale_for(m);
    if (joins) {
      s = max(s, power_of_two(old));
      if (s != __float_as_uint(old)) {
        const float f = old * inverse(s);
        for (int r = part * RPP + lane / LPR; r < it.lo - it.begin; r += W * RPP) {
          codes16* const at = reinterpret_cast<codes16*>(dst + r * D + 16 * w);
          *at = rescaled(*at, f);
        }
      }
    }
    const float inv = inverse(s);
    if (stored && !idle && part == 0 && lane == 0) *scale = __uint_as_float(s);
    for (int chunk = 0; chunk < chunks; ++chunk) {
      if (chunks > 1) load(chunk);
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        if (!live[i]) continue;
        const int p = row_of(chunk, i);
        if (stored) {
#pragma unroll
          for (int n = 0; n < 8; ++n) x[i][n] *= inv, y[i][n] *= inv;
          uint8_t* const to = dst + (p - it.begin) * D;
          store8_e4m3<NT>(to + c.c0, x[i]);
          store8_e4m3<NT>(to + c.c1, y[i]);
        } else {
          bf16_t* const to = static_cast<bf16_t*>(a.q_out) + (it.row0 + (p - it.pos)) * a.q_out_stride + h * D;
          store8<NT>(to + c.c0, x[i]);
          store8<NT>(to + c.c1, y[i]);
        }
      }
    }
  }
}

template <int D, int W, bool NT>
hipError_t run(const BlocksArgs& a, hipStream_t st) {
  constexpr int NW = W > 4 ? W : 4;
  const int64_t N = a.kb.n_tokens, B = a.kb.s.B;
  int64_t items = (N >> a.scales.shift) + 2 * B;
  if (items > N) items = N;
  const unsigned y = (a.kinds + NW / W - 1) / (NW / W);
  const int64_t most = (((int64_t)1 << 32) - 1) / ((int64_t)y * NW * kWave);  // threads of a launch
  if (items > most) items = most;
  const dim3 grid((unsigned)items, y), block(NW * kWave);
  if (a.axes.n)
    hipLaunchKernelGGL((append_blocks_kernel<D, W, NT, true>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((append_blocks_kernel<D, W, NT, false>), grid, block, 0, st, a);
  return hipGetLastError();
}

template <int D, bool NT>
hipError_t by_rows(const BlocksArgs& a, hipStream_t st) {
  // Waves enough for the rows that a call can bring to a block, up to 16.
  const int block = 1 << a.scales.shift, rows = a.kb.s.T < block ? a.kb.s.T : block;
  if (rows <= 16) return run<D, 1, NT>(a, st);
  if (rows <= 32) return run<D, 2, NT>(a, st);
  if (rows <= 64) return run<D, 4, NT>(a, st);
  if (rows <= 128) return run<D, 8, NT>(a, st);
  return run<D, 16, NT>(a, st);
}

}  // namespace

hipError_t launch_kv_append_blocks(const KvBatch& b, const BlockScales& scales, KvRows k, KvRows v, KvRows q,
                                   void* q_out, int64_t q_out_stride, const kda_rotation& rot, const Axes& axes,
                                   hipStream_t st) {
  const BlocksArgs a{b, scales, k, v, q, q_out, q_out_stride, rot, 2 * b.s.Hkv + (q.p ? b.s.Hq : 0), axes};
  return b.s.dk == 128 ? by_rows<128, false>(a, st) : by_rows<64, false>(a, st);
}

}  // namespace kda
