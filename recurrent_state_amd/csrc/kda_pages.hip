// Appending to the paged attention cache: new keys are rotated by their
// positions and stored in their pages with the values, and the queries of the
// same tokens are rotated, in one launch.
//
// A thread takes one unit of 16 values of one head row: two chunks of 8 that
// hold both members of 8 rotation pairs (chunks `dim / 2` apart for pairs
// (n, dim / 2 + n), neighbours for (2n, 2n + 1) and for values that are not
// rotated), so nothing is exchanged between lanes and q_out may be q itself.
// A token's units are numbered queries, keys, values; consecutive threads take
// consecutive units, so a wave covers whole 128-byte lines of a head row.  With
// positions on several axes the cosines and sines of a unit may come from as many
// rows of the table, pair by pair; in large calls a thread reads them once for
// the same unit of four heads.
//
// Bound by memory for prompts, and by the chain of dependent loads (token range,
// position, page) for a few tokens: the unit's values depend on none of these
// and are asked for first.  Measured, the kernel by itself, 32 query and 8 kv
// heads of 128: eight prompts of 8192 tokens in bf16 285 us (1.64 GB, 5.8 TB/s),
// into e4m3 286 (5.3 TB/s), four in f32 338 (4.8 TB/s), four latent ones 504
// (2.50 GB, 5.0 TB/s); one token 2.6 us, 256 tokens of a latent cache 6.6 us.  A
// call of one token among others takes 4.2 us, which is the host's part.  With three
// axes: four prompts of 5000 tokens in bf16 104 us (502 MB, 4.8 TB/s), one token 3.4.

#include "kda_append_impl.h"

namespace kda {
namespace {

constexpr int kThreads = 256;

struct AppendArgs {
  KvBatch kb;
  KvRows k, v, q;
  void* q_out;
  int64_t q_out_stride;
  kda_rotation rot;
  int32_t units_q, units_k, units;  // threads of a token: for queries; and keys; and values
  Axes axes;
};

// A sequence with packed row `row` in its range, and which of its tokens that
// row is; b = -1 for a row of no sequence.
struct Owner {
  int b, token;
  bool more;  // a later sequence's range holds the row too
};
// The first such sequence from `from` on (`begin`: the wave's smallest, or less).
// Every range counts by itself, so that one that does not fit the launch takes
// nothing from the others, wherever its ends point.  They are looked at until
// every lane that looks has met two: a lane takes four of 256 neighbours (the rest
// 64 at a time), and the few that meet the wave's rows, which ascend with the
// lanes, are held against each lane's.
__device__ __forceinline__ Owner owner_of(const KvBatch& kb, int row, int from, int begin) {
  const int lane = here((int)threadIdx.x & 63), B = kb.s.B;
  const int first = __builtin_amdgcn_readfirstlane(row), last = __builtin_amdgcn_readlane(row, kWave - 1);
  Owner o{-1, 0, false};
  auto meet = [&](int c, int step, int32_t start, int32_t end) {  // of sequence c + step * lane
    for (uint64_t near = __ballot(start <= last && end > first); near != 0; near &= near - 1) {
      const int at = __ffsll((unsigned long long)near) - 1, b = c + step * at;
      const int r0 = __builtin_amdgcn_readlane(start, at), r1 = __builtin_amdgcn_readlane(end, at);
      if (!fits(kb, r0, r1) || row < r0 || row >= r1 || b < from) continue;
      o.more |= o.b >= 0;
      if (o.b < 0 || b < o.b) o.b = b, o.token = row - r0;
    }
  };
  int c = begin & ~(4 * kWave - 1);
  for (; c + 4 * kWave <= B; c += 4 * kWave) {
    const int32_t* p = kb.tok_start + c + 4 * lane;
    int32_t at[5];
#pragma unroll
    for (int j = 0; j < 5; ++j) at[j] = p[j];
    bool any = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) any |= (at[j] <= last) & (at[j + 1] > first);
    if (__ballot(any) == 0) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) meet(c + j, 4, at[j], at[j + 1]);
    if (__ballot(from < B && !o.more) == 0) return o;
  }
  for (; c < B; c += kWave) {
    const int b = min(c + lane, B - 1);
    meet(c, 1, kb.tok_start[b], c + lane < B ? kb.tok_start[b + 1] : INT32_MIN);
  }
  return o;
}

// Unit e, of HEADS heads, to its place for the first sequence from `from` on that has its row
// (`begin`: see owner_of).
// Returns where a search for a further one begins, B if there is none.
template <int DK, int DV, typename TIn, typename TC, bool NT, bool AXES, int HEADS>
__device__ __forceinline__ int append_unit(const AppendArgs& a, uint32_t e, int from, int begin) {
  constexpr bool kE4m3 = sizeof(TC) == 1;
  const KvBatch& kb = a.kb;
  // Row and unit of this thread; the threads past the last unit take part in
  // owner_of with that one's row.
  const uint32_t total = (uint32_t)kb.n_tokens * (uint32_t)a.units;  // fits: checked on the host
  const bool live = e < total;
  const uint32_t unit = live ? e : total - 1;
  const int row = (int)(unit / (uint32_t)a.units), u = (int)(unit - (uint32_t)row * (uint32_t)a.units);

  // What the unit is, and its two chunks: rotated units of a head come first.
  const bool is_value = u >= a.units_k, is_key = !is_value && u >= a.units_q;
  const bool rotates = a.rot.cos_sin != nullptr;
  const int n_rot = rotates ? a.rot.dim >> 4 : 0;
  int h, w = 0;
  Chunks c;
  const TIn* src;
  if (is_value) {
    const int at = u - a.units_k;
    h = at / (DV / 16) * HEADS;
    c.c0 = at % (DV / 16) * 16;
    c.c1 = c.c0 + 8;
    src = static_cast<const TIn*>(a.v.p) + row * a.v.stride + h * DV;
  } else {
    const int at = is_key ? u - a.units_q : u;
    h = at / (DK / 16) * HEADS;
    w = at % (DK / 16);
    c = chunks_of(a.rot, n_rot, w);
    src = is_key ? static_cast<const TIn*>(a.k.p) + row * a.k.stride + h * DK
                 : static_cast<const TIn*>(a.q.p) + row * a.q.stride + h * DK;
  }
  const int width = is_value ? DV : DK, heads = HEADS == 1 ? 1 : min(HEADS, (is_key || is_value ? kb.s.Hkv : kb.s.Hq) - h);
  float x[HEADS][8], y[HEADS][8];
#pragma unroll
  for (int i = 0; i < HEADS; ++i)
    if (i < heads) {
      load8<NT>(src + i * width + c.c0, x[i]);
      load8<NT>(src + i * width + c.c1, y[i]);
    }

  Owner o;
  if (kb.tok_start)
    o = owner_of(kb, row, from, begin);
  else
    o.b = row / kb.s.T, o.token = row - o.b * kb.s.T, o.more = false;
  const int b = o.b, next = o.more && (is_key || is_value) ? b + 1 : kb.s.B;
  auto append = [&] {
    const int64_t p = kb.pos[b] + o.token;
    bool off = p < 0;
    AxisPos axis_pos;
    if constexpr (AXES)
      axis_pos = axis_positions(a.axes, a.rot, row), off |= axis_pos.bad;
    else
      off |= rotates && p >= a.rot.max_pos;
    if (off) {
      if (u == a.units_q) set_err(kb.dev_err, KDA_DEV_ERR_POS);
      return;
    }
    const int64_t at = p >> kb.page_shift;
    const int32_t page = at < kb.max_pages ? kb.table[(int64_t)b * kb.max_pages + at] : -1;
    float cc[8], ss[8];
    const bool turn = !is_value && w < n_rot;
    if (turn) {
      if constexpr (AXES)
        angles(a.rot, axis_pos, axes_of_unit<AppendArgs>(w), w, cc, ss);
      else
        angles(a.rot, p, w, cc, ss);
    }
    if (page < 0 || page >= kb.pages.n_pages) {
      if (u == a.units_q) set_err(kb.dev_err, KDA_DEV_ERR_PAGE);
      return;
    }

#pragma unroll
    for (int i = 0; i < HEADS; ++i)
      if (turn && i < heads) rotate(x[i], y[i], cc, ss, a.rot.pairs);
    if (!is_value && !is_key) {
      TIn* dst = static_cast<TIn*>(a.q_out) + row * a.q_out_stride + h * DK;
#pragma unroll
      for (int i = 0; i < HEADS; ++i)
        if (i < heads) {
          store8<NT>(dst + i * DK + c.c0, x[i]);
          store8<NT>(dst + i * DK + c.c1, y[i]);
        }
      return;
    }
    const int64_t place = (((int64_t)page * kb.s.Hkv + h) << kb.page_shift) + ((int)p & (kb.pages.page_size - 1));
    TC* dst = is_value ? static_cast<TC*>(kb.pages.v) + place * DV : static_cast<TC*>(kb.pages.k) + place * DK;
    const int64_t next_head = (int64_t)width << kb.page_shift;
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
      if (i >= heads) continue;
      if constexpr (kE4m3) {
        const float scale = (is_value ? kb.pages.v_scale : kb.pages.k_scale)[h + i];
        store8_e4m3<NT>(dst + i * next_head + c.c0, x[i], scale);
        store8_e4m3<NT>(dst + i * next_head + c.c1, y[i], scale);
      } else {
        store8<NT>(dst + i * next_head + c.c0, x[i]);
        store8<NT>(dst + i * next_head + c.c1, y[i]);
      }
    }
  };
  if (live && b >= 0) append();
  return next;
}

template <int DK, int DV, typename TIn, typename TC, bool NT, bool AXES, int HEADS>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendArgs a) {
  const KvBatch& kb = a.kb;
  // Ranges that do not fit the launch are named by the first block, whether
  // or not they hold a row.
  if (blockIdx.x == 0 && kb.tok_start)
    for (int b = threadIdx.x; b < kb.s.B; b += kThreads)
      if (seq_rows(kb, b).bad) set_err(kb.dev_err, KDA_DEV_ERR_TOKENS);
  // A second turn only for keys or values that several ranges hold: one of them
  // begins before a range that runs backwards.  here(), also in owner_of: what a
  // turn computes is not kept for the next, which took 20 registers (8 prompts of
  // 8192 tokens to e4m3 364 us, now 285).
  for (int from = 0, begin = 0;;) {
    from = append_unit<DK, DV, TIn, TC, NT, AXES, HEADS>(
        a, here((int)(blockIdx.x * kThreads + threadIdx.x)), from, begin);
    if (__ballot(from < kb.s.B) == 0) return;
    begin = from;
#pragma unroll
    for (int i = 1; i < kWave; i *= 2) begin = min(begin, __shfl_xor(begin, i));
    begin = __builtin_amdgcn_readfirstlane(begin);
  }
}

// Calls that touch more than the 256 MB Infinity Cache go past it: 65536 tokens
// of 32 + 8 heads of 128 in 282 us for 292 with plain accesses, into e4m3 283 for
// 300; with pairs dealt to three axes 314 for 343 and 435 for 454.  The rule goes by
// bytes alone, and f32 and latent prompts lose by it: 16384 f32 tokens 173 us for
// 146, with axes 184 for 167; 32768 latent ones 500 for 445, with axes 567 for 493.
// What smaller calls write stays there for the attention that reads it next.
template <int DK, int DV, typename TIn, typename TC, bool NT, bool AXES, int HEADS>
hipError_t run(AppendArgs a, hipStream_t st) {
  const kda_kv_shape& s = a.kb.s;
  const auto groups = [](int32_t heads) { return (heads + HEADS - 1) / HEADS; };
  a.units_q = a.q.p ? groups(s.Hq) * (DK / 16) : 0;
  a.units_k = a.units_q + groups(s.Hkv) * (DK / 16);
  a.units = a.units_k + (a.v.p ? groups(s.Hkv) * (DV / 16) : 0);
  const int64_t blocks = ((int64_t)a.kb.n_tokens * a.units + kThreads - 1) / kThreads;
  hipLaunchKernelGGL((append_kernel<DK, DV, TIn, TC, NT, AXES, HEADS>), dim3((unsigned)blocks), dim3(kThreads), 0, st,
                     a);
  return hipGetLastError();
}

// With axes a thread takes four heads (two into e4m3) from 2^24 values on, 2730 tokens
// of 32 + 8 heads of 128, so that the pairs' angle rows are read once for them.  us
// with one head to a thread, two and four, pairs dealt to three axes:
//           2^22 values        2^23               2^24               2^26
//   bf16     8.5  7.4  7.5     14.3 11.9 10.6     23.0 19.2 17.1     81   64   59
//   e4m3     8.8  9.0 10.6     14.7 15.2 18.1     23.2 21.5 26.4     86   83  101
//   f32     11.9 11.1 10.9     18.2 17.2 17.8     37.0 35.4 38.2    140  124  125
//   latent   6.5  7.0  7.2     10.8 10.8 11.6     17.0 16.8 17.7     67   63   68
// and by sections, where units of one axis read whole rows of angles in any case:
//   bf16     5.8  6.0  6.8      9.7  9.4  9.4     15.4 15.7 16.1     57   55   57
//   e4m3     6.3  7.6 10.0     10.6 13.1 17.2     16.3 18.7 25.3     62   73   96
// Fewer values leave the chip without threads (one token 3.5 -> 4.8 with four).  The
// rule is made for dealt pairs; sections into e4m3 lose by it.
template <int DK, int DV, typename TIn, typename TC>
hipError_t run(const AppendArgs& a, hipStream_t st) {
  const kda_kv_shape& s = a.kb.s;
  const int64_t values = a.kb.n_tokens * ((int64_t)s.Hkv * (DK + (a.v.p ? DV : 0)) + (a.q.p ? (int64_t)s.Hq * DK : 0));
  const bool large = values * (int64_t)(sizeof(TIn) + sizeof(TC)) > (int64_t)256 << 20;
  constexpr int kMost = sizeof(TC) == 1 ? 2 : 4;  // the divisions by a scale take registers
  if (a.axes.n) {
    if (large) return run<DK, DV, TIn, TC, true, true, kMost>(a, st);
    if (values >= (int64_t)1 << 24) return run<DK, DV, TIn, TC, false, true, kMost>(a, st);
    return run<DK, DV, TIn, TC, false, true, 1>(a, st);
  }
  return large ? run<DK, DV, TIn, TC, true, false, 1>(a, st) : run<DK, DV, TIn, TC, false, false, 1>(a, st);
}

}  // namespace

hipError_t launch_kv_append(const KvBatch& b, KvRows k, KvRows v, KvRows q, void* q_out, int64_t q_out_stride,
                            const kda_rotation& rot, const Axes& axes, hipStream_t st) {
  const AppendArgs a{b, k, v, q, q_out, q_out_stride, rot, 0, 0, 0, axes};
  if (b.s.dk == 576) return run<576, 512, bf16_t, bf16_t>(a, st);
  const bool wide = b.s.dk == 128;
  if (b.s.in_dtype == KDA_F32)
    return wide ? run<128, 128, float, float>(a, st) : run<64, 64, float, float>(a, st);
  if (b.s.cache_dtype == KDA_E4M3)
    return wide ? run<128, 128, bf16_t, uint8_t>(a, st) : run<64, 64, bf16_t, uint8_t>(a, st);
  return wide ? run<128, 128, bf16_t, bf16_t>(a, st) : run<64, 64, bf16_t, bf16_t>(a, st);
}

}  // namespace kda
