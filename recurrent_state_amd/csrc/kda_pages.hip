// Appending to the paged attention cache: new keys are rotated by their
// positions and stored in their pages with the values, and the queries of the
// same tokens are rotated, in one launch.
//
// A thread takes one unit of 16 values of one head row: two chunks of 8 that
// hold both members of 8 rotation pairs (chunks `dim / 2` apart for pairs
// (n, dim / 2 + n), neighbours for (2n, 2n + 1) and for values that are not
// rotated), so nothing is exchanged between lanes and q_out may be q itself.
// A token's units are numbered queries, keys, values; consecutive threads take
// consecutive units, so a wave covers whole 128-byte lines of a head row.
//
// Bound by memory for prompts, and by the chain of dependent loads (token range,
// position, page) for a few tokens: the unit's values depend on none of these
// and are asked for first.  Measured, the kernel by itself, 32 query and 8 kv
// heads of 128: eight prompts of 8192 tokens in bf16 285 us (1.64 GB, 5.8 TB/s),
// into e4m3 286 (5.3 TB/s), four in f32 338 (4.8 TB/s), four latent ones 504
// (2.50 GB, 5.0 TB/s); one token 2.6 us, 256 tokens of a latent cache 6.6 us.  A
// call of one token among others takes 4.2 us, which is the host's part.

#include "kda_pages.h"

namespace kda {
namespace {

constexpr int kThreads = 256;

struct AppendArgs {
  KvBatch kb;
  KvRows k, v, q;
  void* q_out;
  int64_t q_out_stride;
  kda_rotation rot;
  int32_t units_q, units_k, units;  // units of a token: queries; and keys; and values
};

typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(4))) float f32x4;

// NT: non-temporal, for calls that outgrow the caches (see run()).
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

// e4m3 of x / scale: clamped to the type's largest value (it has no infinity),
// rounded to nearest even by the conversion.  The division is the IEEE one, so
// the stored bits are those of the formula.
__device__ __forceinline__ float to_range(float x, float scale) {
  const float y = x / scale;
  return y != y ? y : fminf(fmaxf(y, -448.f), 448.f);
}
template <bool NT>
__device__ __forceinline__ void store8_e4m3(uint8_t* p, const float (&x)[8], float scale) {
  int w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(to_range(x[4 * i], scale), to_range(x[4 * i + 1], scale), w[i], false);
    w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(to_range(x[4 * i + 2], scale), to_range(x[4 * i + 3], scale), w[i], true);
  }
  put<NT>(reinterpret_cast<u32x2*>(p), (u32x2){(uint32_t)w[0], (uint32_t)w[1]});
}

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

// Unit e to its place for the first sequence from `from` on that has its row
// (`begin`: see owner_of).
// Returns where a search for a further one begins, B if there is none.
template <int DK, int DV, typename TIn, typename TC, bool NT>
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
  int h, w = 0, c0, c1;
  const TIn* src;
  if (is_value) {
    const int at = u - a.units_k;
    h = at / (DV / 16);
    c0 = at % (DV / 16) * 16;
    c1 = c0 + 8;
    src = static_cast<const TIn*>(a.v.p) + row * a.v.stride + h * DV;
  } else {
    const int at = is_key ? u - a.units_q : u;
    h = at / (DK / 16);
    w = at % (DK / 16);
    if (w < n_rot) {
      c0 = a.rot.start + (a.rot.pairs ? 16 * w : 8 * w);
      c1 = c0 + (a.rot.pairs ? 8 : a.rot.dim >> 1);
    } else {
      c0 = 16 * (w - n_rot);
      if (rotates && c0 >= a.rot.start) c0 += a.rot.dim;
      c1 = c0 + 8;
    }
    src = is_key ? static_cast<const TIn*>(a.k.p) + row * a.k.stride + h * DK
                 : static_cast<const TIn*>(a.q.p) + row * a.q.stride + h * DK;
  }
  float x[8], y[8];
  load8<NT>(src + c0, x);
  load8<NT>(src + c1, y);

  Owner o;
  if (kb.tok_start)
    o = owner_of(kb, row, from, begin);
  else
    o.b = row / kb.s.T, o.token = row - o.b * kb.s.T, o.more = false;
  const int b = o.b, next = o.more && (is_key || is_value) ? b + 1 : kb.s.B;
  auto append = [&] {
    const int64_t p = kb.pos[b] + o.token;
    if (p < 0 || (rotates && p >= a.rot.max_pos)) {
      if (u == a.units_q) set_err(kb.dev_err, KDA_DEV_ERR_POS);
      return;
    }
    const int64_t at = p >> kb.page_shift;
    const int32_t page = at < kb.max_pages ? kb.table[(int64_t)b * kb.max_pages + at] : -1;
    float cc[8], ss[8];
    const bool turn = !is_value && w < n_rot;
    if (turn) {
      const float* cs = a.rot.cos_sin + p * a.rot.dim + 8 * w;
      load8<false>(cs, cc);
      load8<false>(cs + (a.rot.dim >> 1), ss);
    }
    if (page < 0 || page >= kb.pages.n_pages) {
      if (u == a.units_q) set_err(kb.dev_err, KDA_DEV_ERR_PAGE);
      return;
    }

    if (turn) {
      if (a.rot.pairs) {
        // x holds pairs 0..3 interleaved, y pairs 4..7.
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const float x0 = x[2 * n], x1 = x[2 * n + 1], y0 = y[2 * n], y1 = y[2 * n + 1];
          x[2 * n] = x0 * cc[n] - x1 * ss[n];
          x[2 * n + 1] = x1 * cc[n] + x0 * ss[n];
          y[2 * n] = y0 * cc[4 + n] - y1 * ss[4 + n];
          y[2 * n + 1] = y1 * cc[4 + n] + y0 * ss[4 + n];
        }
      } else {
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const float x0 = x[n], y0 = y[n];
          x[n] = x0 * cc[n] - y0 * ss[n];
          y[n] = y0 * cc[n] + x0 * ss[n];
        }
      }
    }
    if (!is_value && !is_key) {
      TIn* dst = static_cast<TIn*>(a.q_out) + row * a.q_out_stride + h * DK;
      store8<NT>(dst + c0, x);
      store8<NT>(dst + c1, y);
      return;
    }
    const int64_t place = (((int64_t)page * kb.s.Hkv + h) << kb.page_shift) + ((int)p & (kb.pages.page_size - 1));
    TC* dst = is_value ? static_cast<TC*>(kb.pages.v) + place * DV : static_cast<TC*>(kb.pages.k) + place * DK;
    if constexpr (kE4m3) {
      const float scale = (is_value ? kb.pages.v_scale : kb.pages.k_scale)[h];
      store8_e4m3<NT>(dst + c0, x, scale);
      store8_e4m3<NT>(dst + c1, y, scale);
    } else {
      store8<NT>(dst + c0, x);
      store8<NT>(dst + c1, y);
    }
  };
  if (live && b >= 0) append();
  return next;
}

template <int DK, int DV, typename TIn, typename TC, bool NT>
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
    from = append_unit<DK, DV, TIn, TC, NT>(a, here((int)(blockIdx.x * kThreads + threadIdx.x)), from, begin);
    if (__ballot(from < kb.s.B) == 0) return;
    begin = from;
#pragma unroll
    for (int i = 1; i < kWave; i *= 2) begin = min(begin, __shfl_xor(begin, i));
    begin = __builtin_amdgcn_readfirstlane(begin);
  }
}

// Calls that touch more than the 256 MB Infinity Cache go past it: 65536 tokens
// of 32 + 8 heads of 128 in 284 us for 288 with plain accesses, into e4m3 285 for
// 303.  f32 and latent prompts lose by it (16384 f32 tokens 170 us for 147, 32768
// latent ones 503 for 444).  What smaller calls write stays there for the
// attention that reads it next.
template <int DK, int DV, typename TIn, typename TC>
hipError_t run(const AppendArgs& a, hipStream_t st) {
  const int64_t units = (int64_t)a.kb.n_tokens * a.units, blocks = (units + kThreads - 1) / kThreads;
  if (units * 16 * (int64_t)(sizeof(TIn) + sizeof(TC)) > (int64_t)256 << 20)
    hipLaunchKernelGGL((append_kernel<DK, DV, TIn, TC, true>), dim3((unsigned)blocks), dim3(kThreads), 0, st, a);
  else
    hipLaunchKernelGGL((append_kernel<DK, DV, TIn, TC, false>), dim3((unsigned)blocks), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const KvBatch& b, KvRows k, KvRows v, KvRows q, void* q_out, int64_t q_out_stride,
                            const kda_rotation& rot, hipStream_t st) {
  AppendArgs a{b, k, v, q, q_out, q_out_stride, rot, 0, 0, 0};
  a.units_q = q.p ? b.s.Hq * (b.s.dk / 16) : 0;
  a.units_k = a.units_q + b.s.Hkv * (b.s.dk / 16);
  a.units = a.units_k + (v.p ? b.s.Hkv * (b.s.dv / 16) : 0);
  if (b.s.dk == 576) return run<576, 512, bf16_t, bf16_t>(a, st);
  const bool wide = b.s.dk == 128;
  if (b.s.in_dtype == KDA_F32)
    return wide ? run<128, 128, float, float>(a, st) : run<64, 64, float, float>(a, st);
  if (b.s.cache_dtype == KDA_E4M3)
    return wide ? run<128, 128, bf16_t, uint8_t>(a, st) : run<64, 64, bf16_t, uint8_t>(a, st);
  return wide ? run<128, 128, bf16_t, bf16_t>(a, st) : run<64, 64, bf16_t, bf16_t>(a, st);
}

}  // namespace kda
