// Head norms and rotary positions: forward, gradient, and the form that
// appends the new tokens of a batch to a paged cache.
//
//   y = R(p) (x r w),  r = rsqrt(mean(x^2) + eps)          (x: one head's d values)
//   z = R(p)^T dy,  h = x r:   dw = sum z h,  dx = r (z w - h mean(z w h))
//
// Bound by HBM: 2 bytes in and 2 out for each value, the cos | sin row of a
// token read once for 16 (d 128) or 32 (d 64) of its heads.  Seven warps of a
// CTA work, each on its own units (up to 4 KB of one token's heads, which are
// contiguous) and from its own ring of them in shared memory; the eighth finds
// the places of the units, four lanes a ring so that four look-ups are under
// way, and fills the rings by bulk copies that run ahead.  The reads in flight
// then do not depend on registers, and what a unit costs in instructions beside
// its arithmetic is spent once for seven of them.  Units are dealt one to each
// warp of the grid in turn: at any time the grid reads one run of memory, and
// padding, which costs less, is spread evenly.  Small calls, and tokens of so few
// heads that units would be small, go row by row straight from memory instead
// (fwd_rows_kernel, bwd_rows_kernel; the choice is use_rows()'s).
//
// A row of d values is held by d / 16 lanes, each with two 16-byte pieces whose
// pairs of the rotation are both in the lane: pieces l and l + rot/16 where
// halves are paired, pieces 2l and 2l + 1 where neighbours are, so the rotation
// needs no exchange and the norm only 3 shuffles (2 for d 64).  All pieces of a
// lane use cos and sin values [8l, 8l + 8) of the token.  The arithmetic is in
// packed pairs of fp32 (f32x2), which halves its instructions; these, not the
// reads, bound a form with plain fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "device_common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace {

__device__ unsigned int g_status_rope = 0;

// A CTA: seven warps that work and one that loads.  (One CTA an SM with 13 + 3
// warps was within 3 % either way; a second loading warp leaves 96 registers a
// thread and took 236 instead of 195 us on the 64K-token tree.)
constexpr int kWarps = 7;
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kBatch = 4;  // lanes of the loading warp for each ring: units looked up together
constexpr int kCtas = 2;   // CTAs an SM

struct Rope {
  const float* table;
  const void* wq;
  const void* wk;
  int32_t table_rows, rot, interleaved, w_bf16;
  float eps;
};

// [rows, heads, d] with contiguous heads
struct Rows {
  const uint8_t* p;
  int64_t stride;  // bytes
};
struct RowsOut {
  uint8_t* p;
  int64_t stride;
};

template <int D>
struct Geo {
  static constexpr int LPR = D / 16;    // lanes of a row
  static constexpr int RPW = 32 / LPR;  // rows of a warp
};

// The two 16-byte pieces of a row that lane l of its LPR lanes holds.
template <int D>
__device__ __forceinline__ void pieces(int l, int rot, bool interleaved, int& a, int& b) {
  const int nr = rot >> 4;
  if (!interleaved && l < nr) {
    a = l;
    b = l + nr;
  } else {
    a = 2 * l;
    b = 2 * l + 1;
  }
}

using tc::add2;
using tc::f2;
using tc::fma2;
using tc::mul2;
using tc::unf2;

// A lane's 16 values of a row: the first and the second of its 8 pairs, packed by two.
struct Vals {
  uint64_t a[4], b[4];
};

// bf16 words of the lane's two pieces <-> pairs.  Where neighbours are paired, a
// word holds a pair: the words are re-sorted into firsts and seconds.
__device__ __forceinline__ uint64_t widen(uint32_t w) {
  return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ Vals unpack16(const uint4& x, const uint4& y, bool inter) {
  uint32_t u[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  if (inter) {
    uint32_t t[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t[i] = __byte_perm(u[2 * i], u[2 * i + 1], 0x5410);
      t[4 + i] = __byte_perm(u[2 * i], u[2 * i + 1], 0x7632);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = t[i];
  }
  Vals v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v.a[i] = widen(u[i]);
    v.b[i] = widen(u[4 + i]);
  }
  return v;
}
__device__ __forceinline__ uint32_t narrow(uint64_t v) {
  float lo, hi;
  unf2(v, lo, hi);
  return tc::pack_bf16(lo, hi);
}
__device__ __forceinline__ void pack16(const Vals& v, bool inter, uint4& x, uint4& y) {
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    u[i] = narrow(v.a[i]);
    u[4 + i] = narrow(v.b[i]);
  }
  if (inter) {
    uint32_t t[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t[2 * i] = __byte_perm(u[i], u[4 + i], 0x5410);
      t[2 * i + 1] = __byte_perm(u[i], u[4 + i], 0x7632);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = t[i];
  }
  x = make_uint4(u[0], u[1], u[2], u[3]);
  y = make_uint4(u[4], u[5], u[6], u[7]);
}

// 8 consecutive floats as 4 packed pairs
__device__ __forceinline__ void load_p4(const float* p, uint64_t* x) {
  const ulonglong2 a = reinterpret_cast<const ulonglong2*>(p)[0], b = reinterpret_cast<const ulonglong2*>(p)[1];
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}

// Both weights as fp32 into shared memory, by the working warps, in the order in
// which the lanes hold a row: 16 l + j is the first of lane l's pair j, 16 l + 8 + j the second.
template <int D>
__device__ __forceinline__ void stage_weights(const Rope& r, float* w) {
  for (int i = threadIdx.x; i < 2 * D; i += 32 * kWarps) {
    const void* src = i < D ? r.wq : r.wk;
    const int e = i % D, l = e >> 4, j = e & 7, second = (e >> 3) & 1, nr = r.rot >> 4;
    int at;
    if (r.interleaved) at = 16 * l + 2 * j + second;
    else if (l < nr) at = 8 * (l + second * nr) + j;
    else at = 16 * l + 8 * second + j;
    w[i] = r.w_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(src)[at]) : static_cast<const float*>(src)[at];
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float sum2(uint64_t v) {
  float lo, hi;
  unf2(v, lo, hi);
  return lo + hi;
}
__device__ __forceinline__ uint64_t neg2(uint64_t v) { return v ^ 0x8000000080000000ull; }

template <int D>
__device__ __forceinline__ float rstd(const Vals& v, float eps) {
  uint64_t s = mul2(v.a[0], v.a[0]), t = mul2(v.b[0], v.b[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    s = fma2(v.a[i], v.a[i], s);
    t = fma2(v.b[i], v.b[i], t);
  }
  return rsqrtf(row_sum<Geo<D>::LPR>(sum2(add2(s, t))) * (1.f / D) + eps);
}

// A lane's two 16-byte pieces of a bf16 row.  Where they are neighbours they
// may leave as one 32-byte store, a whole sector (`one`).
__device__ __forceinline__ void store_pieces(uint8_t* row, int pa, int pb, const uint4& x, const uint4& y, bool one) {
  if (one) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(row + 16 * pa), "r"(x.x), "r"(x.y),
                 "r"(x.z), "r"(x.w), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w)
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(row)[pa] = x;
    reinterpret_cast<uint4*>(row)[pb] = y;
  }
}

// What a lane's pairs are multiplied by, the weights with it:
// first' = r (ca first - sb second), second' = r (cb second + sa first), sb held negative.
struct Coefs {
  uint64_t ca[4], cb[4], sa[4], sb[4];

  // From the cosines and sines in ca and sa, where `turns` (the lane's pairs are among those turned), and the weights.
  template <bool NORM>
  __device__ __forceinline__ void weigh(bool turns, const uint64_t (&wa)[4], const uint64_t (&wb)[4]) {
    if (turns) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        cb[j] = ca[j];
        sb[j] = sa[j];
      }
    }
    if constexpr (NORM) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ca[j] = turns ? mul2(ca[j], wa[j]) : wa[j];
        cb[j] = turns ? mul2(cb[j], wb[j]) : wb[j];
        sa[j] = mul2(sa[j], wa[j]);
        sb[j] = mul2(sb[j], wb[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) sb[j] = neg2(sb[j]);
  }

  template <int D, bool NORM>
  __device__ __forceinline__ Vals apply(const Vals& x, bool turns, float eps) const {
    Vals y = x;
    if (turns) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y.a[j] = fma2(x.a[j], ca[j], mul2(x.b[j], sb[j]));
        y.b[j] = fma2(x.b[j], cb[j], mul2(x.a[j], sa[j]));
      }
    } else if constexpr (NORM) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y.a[j] = mul2(x.a[j], ca[j]);
        y.b[j] = mul2(x.b[j], cb[j]);
      }
    }
    if constexpr (NORM) {
      const float rs = rstd<D>(x, eps);
      const uint64_t r2 = f2(rs, rs);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y.a[j] = mul2(y.a[j], r2);
        y.b[j] = mul2(y.b[j], r2);
      }
    }
    return y;
  }
};

// ------------------------------------------------------------------ the warps' rings


// One unit: rows of one token from head h on.  Its first `turned` rows are
// queries or keys, the others (append) values from head 0 on, or h when there are no keys with them.
struct Unit {
  int32_t kind, h, rows, turned, state, token;  // kind 0: queries, 1: keys and values
  int64_t slot;                                 // append: row of (page, head 0, slot) in the cache
};
enum { kUse = 0, kPad = 1, kSkip = 2 };

template <int D, uint32_t DATA>
struct Ring {
  static constexpr uint32_t TABLE = D * 4;
  static constexpr uint32_t STAGE = DATA + TABLE + uint32_t(sizeof(Unit));
  // Three stages where the rings of two CTAs fit beside each other (20K tokens appended: 42.8 us, with two 47.5;
  // the 64K-token tree 194.5 and 196.5 us).
  static constexpr int NST = kCtas * (3 * kWarps * STAGE + 2048) <= 227 * 1024 ? 3 : 2;
  static constexpr uint32_t WARP = NST * STAGE;
  static constexpr uint32_t OFF_FULL = kWarps * WARP;
  static constexpr uint32_t OFF_EMPTY = OFF_FULL + kWarps * NST * 8;
  static constexpr uint32_t OFF_FLAG = OFF_EMPTY + kWarps * NST * 8;
  static constexpr uint32_t OFF_W = OFF_FLAG + 16;
  static constexpr uint32_t BYTES = OFF_W + 2 * D * 4;
  static_assert(sizeof(Unit) == 32 && NST <= kBatch && STAGE % 16 == 0 && OFF_W % 16 == 0 &&
                    kCtas * (BYTES + 1024) <= 228 * 1024,
                "ring");
};

// Barriers of the rings: set w is that of working warp w and of the four lanes of the loading warp that fill its ring.
template <class R>
struct Bars {
  uint8_t* ring;
  uint64_t* full;
  uint64_t* empty;
  volatile int* abort_flag;
  __device__ __forceinline__ Bars(uint8_t* smem, int w)
      : ring(smem + w * R::WARP),
        full(reinterpret_cast<uint64_t*>(smem + R::OFF_FULL) + w * R::NST),
        empty(reinterpret_cast<uint64_t*>(smem + R::OFF_EMPTY) + w * R::NST),
        abort_flag(reinterpret_cast<volatile int*>(smem + R::OFF_FLAG)) {}
  __device__ __forceinline__ void init() const {  // one thread of each ring
    for (int s = 0; s < R::NST; ++s) {
      tc::mbar_init(full + s, 1);
      tc::mbar_init(empty + s, 1);
    }
    tc::fence_mbar_init();
  }
  // Lets the copies already issued land, after a wait that ran out.
  __device__ inline void drain(int issued) const {
    volatile int never = 0;
    for (int j = issued > R::NST ? issued - R::NST : 0; j < issued; ++j)
      tc::mbar_wait(full + j % R::NST, (j / R::NST) & 1, &never, &g_status_rope, 100000000ull);
  }
};

// The loading warp arrives and goes on; the others wait until the barriers (and
// their own weights) are there.
__device__ __forceinline__ void ready_arrive() { asm volatile("bar.arrive 1, %0;" ::"n"(kThreads) : "memory"); }
__device__ __forceinline__ void ready_wait() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }

// The units of global warp `me` of n: one of each run of n, the next one in the
// next run, so that a warp's units are of all kinds where a token's number of
// units divides n.
__device__ __forceinline__ int64_t unit_of(int64_t me, int64_t n, int i) { return i * n + (me + i) % n; }
__device__ __forceinline__ int units_for(int64_t units, int64_t me, int64_t n) {
  const int runs = int(units / n);
  return runs + (unit_of(me, n, runs) < units ? 1 : 0);
}

// A stage and the parity of its phase, one after another.
template <int NST>
struct Turn {
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++s == NST) {
      s = 0;
      phase ^= 1;
    }
  }
};

// A unit's token and part of it, and the token's place.
struct Place {
  int32_t tok, part, pos, state;
  int64_t slot;
};

// The loop of a loading warp: `look(i)` finds the place of this ring's unit i
// (kBatch lanes look up as many of them together), `issue(place, i, stage)`
// starts its copies.  The rings go on in step.  (Each at its own pace, polling
// the stages instead of waiting for them, took 201 instead of 190 us on the
// 64K-token tree: the polls take issue slots from the warps that work.)
template <class R, bool SLOT, class Look, class Issue>
__device__ __forceinline__ void run_loader(const Bars<R>& bar, int w, int mine, Look look, Issue issue) {
  const int lane = threadIdx.x & 31, j = lane % kBatch;
  Turn<R::NST> turn;
  int most = mine, issued = 0;
  bool dead = false;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  for (int i0 = 0; i0 < most; i0 += kBatch) {
    Place own{0, 0, 0, kSkip, 0};
    if (i0 + j < mine) own = look(i0 + j);
    for (int k = 0; k < kBatch && i0 + k < most; ++k) {
      const int from = lane - j + k;
      Place p;
      p.tok = __shfl_sync(0xffffffffu, own.tok, from);
      p.part = __shfl_sync(0xffffffffu, own.part, from);
      p.pos = __shfl_sync(0xffffffffu, own.pos, from);
      p.state = __shfl_sync(0xffffffffu, own.state, from);
      p.slot = SLOT ? __shfl_sync(0xffffffffu, own.slot, from) : 0;
      if (j == 0 && i0 + k < mine && !dead) {
        if (tc::mbar_wait(bar.empty + turn.s, turn.phase ^ 1, bar.abort_flag, &g_status_rope)) {
          issue(p, i0 + k, turn.s);
          turn.next();
          ++issued;
        } else {
          dead = true;
        }
      }
      __syncwarp();
    }
  }
  if (j == 0 && w < kWarps && *bar.abort_flag) bar.drain(issued);
  __syncwarp();
}

// A row's place in the rope table, and whether it is padding.
__device__ __forceinline__ void plain_place(const int32_t* positions, const int32_t* n_tokens, int t_pad, int rows,
                                            int tok, int& pos, int& state) {
  pos = __ldg(positions + tok);
  state = pos < 0 ? kPad : kUse;
  if (n_tokens) {
    const int b = tok / t_pad;
    if (tok - b * t_pad >= __ldg(n_tokens + b)) state = kPad;
  }
  if (state == kUse && pos >= rows) {
    atomicOr(&g_status_rope, TPA_DEV_BAD_INPUT);
    state = kPad;
  }
}

// ------------------------------------------------------------------ forward

struct FwdParams {
  Rope rope;
  const int32_t* positions;
  const int32_t* n_tokens;
  int64_t n_rows;
  int32_t t_pad, hq, hkv;
  int32_t sq, sk, sv;  // units of a token: of queries, of keys (with the values where sv is 0), of values
  Rows q, k, v;
  RowsOut qo, ko;
  tpa_paged_view cache;  // append
  int32_t wide;          // the rows written are 32-byte aligned
};

// Number of entries of the sorted array a[0..n) that are <= v: seven probes a
// round, which are under way together.  Ends for any contents.
__device__ __forceinline__ int count_le(const int32_t* a, int n, int v) {
  int lo = 0, len = n;
  while (len > 0) {
    const int step = (len + 7) >> 3;
    int below = 0;
#pragma unroll
    for (int k = 1; k <= 7; ++k) {
      const int at = k * step - 1;
      below += at < len && __ldg(a + lo + at) <= v;
    }
    const int done = below * step;
    lo += done;
    len = min(below < 7 ? step - 1 : len - done, len - done);
  }
  return lo;
}

// Append: position and cache row of new token `tok`.
__device__ __forceinline__ void paged_place(const FwdParams& p, int tok, int& pos, int& state, int64_t& slot) {
  const tpa_paged_view& c = p.cache;
  pos = 0;
  slot = 0;
  state = kSkip;
  const int s = count_le(c.offsets + 1, c.n_seqs, tok);
  if (s >= c.n_seqs) return;  // rows behind the last sequence
  const int first = __ldg(c.offsets + s), last = __ldg(c.offsets + s + 1), kv = __ldg(c.kv_lens + s);
  // in 64 bits: nothing here is known to be in range yet
  const int64_t at = int64_t(kv) - last + tok;
  bool ok = first >= 0 && tok >= first && tok < last && last <= p.n_rows && at >= 0 &&
            at < int64_t(c.max_pages) * c.page_size && (!p.rope.table || at < p.rope.table_rows);
  if (ok) {
    const int page = __ldg(c.pages + int64_t(s) * c.page_stride + int(at) / c.page_size);
    ok = page >= 0 && page < c.n_pages;
    pos = int(at);
    slot = int64_t(page) * c.n_heads_kv * c.page_size + pos % c.page_size;
  }
  if (ok)
    state = kUse;
  else
    atomicOr(&g_status_rope, TPA_DEV_BAD_INPUT);
}

// Append: the numbers of sequence s, the attention's conditions on them.  The tokens' own look-ups do not meet all: a
// search of offsets out of order may pass over them, and a sequence without new tokens is nobody's.
struct SeqNumbers {
  int32_t o0 = 0, o1 = 0, kv = 0;
  __device__ __forceinline__ void load(const tpa_paged_view& c, int64_t s) {
    o0 = __ldg(c.offsets + s);
    o1 = __ldg(c.offsets + s + 1);
    kv = __ldg(c.kv_lens + s);
  }
  __device__ __forceinline__ void check(const FwdParams& p, int64_t s) const {
    if (o0 < 0 || o1 < o0 || o1 > p.n_rows || (s == 0 && o0 != 0) || kv < 0 ||
        kv > int64_t(p.cache.max_pages) * p.cache.page_size)
      atomicOr(&g_status_rope, TPA_DEV_BAD_INPUT);
  }
};
// Sequences s, s + step, ... of the batch.
__device__ __forceinline__ void check_seqs(const FwdParams& p, int64_t s, int64_t step) {
  for (; s < p.cache.n_seqs; s += step) {
    SeqNumbers q;
    q.load(p.cache, s);
    q.check(p, s);
  }
}

template <int D, bool NORM, bool APPEND>
__global__ void __launch_bounds__(kThreads, kCtas) fwd_kernel(const FwdParams p) {
  using G = Geo<D>;
  constexpr int UROWS = 4096 / (D * 2);  // rows of a unit
  using R = Ring<D, 4096>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool loads = warp == kWarps;
  const int w = loads ? lane / kBatch : warp;  // whose ring; lanes past the last ring have no units
  const Bars<R> bar(smem, min(w, kWarps - 1));
  float* w_s = reinterpret_cast<float*>(smem + R::OFF_W);

  const int per_token = p.sq + p.sk + p.sv;
  const int64_t units = p.n_rows * per_token, n_warps = int64_t(gridDim.x) * kWarps;
  const int64_t me = int64_t(w) * gridDim.x + blockIdx.x;
  const int mine = w < kWarps ? units_for(units, me, n_warps) : 0;
  const uint32_t table_bytes = p.rope.rot * 4;
  if (loads) {
    const int j = lane % kBatch;
    if (threadIdx.x == 32 * kWarps) *bar.abort_flag = 0;
    if (j == 0 && w < kWarps) bar.init();
    __syncwarp();
    ready_arrive();
    // the rows of unit (tok, part) and the copies that bring them
    auto describe = [&](int tok, int part, int& more) {
      Unit u{0, 0, 0, 0, kUse, tok, 0};
      more = 0;  // value rows behind the keys
      if (part < p.sq) {
        u.h = part * UROWS;
        u.turned = u.rows = min(p.hq - u.h, UROWS);
      } else if (part < p.sq + p.sk) {
        u.kind = 1;
        u.h = (part - p.sq) * UROWS;
        u.turned = u.rows = min(p.hkv - u.h, UROWS);
        if (APPEND && p.sv == 0) {
          more = p.hkv;
          u.rows += more;
        }
      } else {
        u.kind = 1;
        u.h = (part - p.sq - p.sk) * UROWS;
        u.rows = min(p.hkv - u.h, UROWS);
      }
      return u;
    };
    auto copy_rows = [&](const Unit& u, int more, int s) {
      const Rows& src = u.kind == 0 ? p.q : u.turned ? p.k : p.v;
      uint8_t* st = bar.ring + s * R::STAGE;
      const int first = u.rows - more;
      tc::bulk_load(st, src.p + u.token * src.stride + int64_t(u.h) * (D * 2), first * (D * 2), bar.full + s);
      if (APPEND && more) tc::bulk_load(st + first * (D * 2), p.v.p + u.token * p.v.stride, more * (D * 2), bar.full + s);
    };
    // the rows of the first units are on their way before their places are known
    auto where = [&](int i) {
      const int64_t u_at = unit_of(me, n_warps, i);
      Place at{int(u_at / per_token), 0, 0, kSkip, 0};
      at.part = int(u_at - int64_t(at.tok) * per_token);
      return at;
    };
    int more;
    if (j < R::NST && j < mine) {
      const Place at = where(j);
      copy_rows(describe(at.tok, at.part, more), more, j);
    }
    run_loader<R, APPEND>(
        bar, w, mine,
        [&](int i) {
          Place at = where(i);
          if constexpr (APPEND) paged_place(p, at.tok, at.pos, at.state, at.slot);
          else plain_place(p.positions, p.n_tokens, p.t_pad, p.rope.table_rows, at.tok, at.pos, at.state);
          return at;
        },
        [&](const Place& at, int i, int stage) {
          const bool early = i < R::NST;
          uint8_t* st = bar.ring + stage * R::STAGE;
          uint64_t* fb = bar.full + stage;
          Unit u = describe(at.tok, at.part, more);
          u.state = at.state;
          u.slot = at.slot;
          *reinterpret_cast<Unit*>(st + 4096 + R::TABLE) = u;
          const bool angles = at.state == kUse && u.turned > 0 && table_bytes > 0;
          if (at.state == kUse && !early) copy_rows(u, more, stage);
          if (angles) tc::bulk_load(st + 4096, p.rope.table + int64_t(at.pos) * p.rope.rot, table_bytes, fb);
          tc::mbar_arrive_expect_tx(fb, (early || at.state == kUse ? u.rows * (D * 2) : 0) + (angles ? table_bytes : 0));
        });
    return;
  }
  if constexpr (NORM) stage_weights<D>(p.rope, w_s);
  ready_wait();
  // beside the first units' way here
  if constexpr (APPEND) check_seqs(p, int64_t(blockIdx.x) * (32 * kWarps) + threadIdx.x, int64_t(gridDim.x) * (32 * kWarps));

  const int l = lane % G::LPR, sub = lane / G::LPR;
  const bool inter = p.rope.interleaved != 0, turns = l < (p.rope.rot >> 4);
  int pa, pb;
  pieces<D>(l, p.rope.rot, inter, pa, pb);
  const bool one = p.wide && pb == pa + 1;
  Turn<R::NST> turn;
  for (int i = 0; i < mine; ++i, turn.next()) {
    if (!__all_sync(0xffffffffu, tc::mbar_wait(bar.full + turn.s, turn.phase, bar.abort_flag, &g_status_rope))) break;
    const uint8_t* st = bar.ring + turn.s * R::STAGE;
    const Unit u = *reinterpret_cast<const Unit*>(st + 4096 + R::TABLE);
    if (u.state != kSkip) {
      Coefs c;
      if (u.turned > 0 && u.state == kUse) {
        uint64_t wa[4], wb[4];
        if (turns) {
          const float* row = reinterpret_cast<const float*>(st + 4096) + 8 * l;
          load_p4(row, c.ca);
          load_p4(row + (p.rope.rot >> 1), c.sa);
        }
        if constexpr (NORM) {
          load_p4(w_s + u.kind * D + 16 * l, wa);
          load_p4(w_s + u.kind * D + 16 * l + 8, wb);
        }
        c.weigh<NORM>(turns, wa, wb);
      }
      int64_t pitch = D * 2;
      uint8_t* out;
      uint8_t* vout = nullptr;
      if (APPEND && u.kind == 1) {
        pitch = int64_t(p.cache.page_size) * (D * 2);
        const int64_t at = u.slot * (D * 2);
        out = static_cast<uint8_t*>(p.cache.k_cache) + at + u.h * pitch;
        vout = static_cast<uint8_t*>(p.cache.v_cache) + at + (u.turned ? -int64_t(u.turned) : int64_t(u.h)) * pitch;
      } else {
        const RowsOut& o = u.kind == 0 ? p.qo : p.ko;
        out = o.p + u.token * o.stride + int64_t(u.h) * (D * 2);
      }
#pragma unroll 4
      for (int r0 = 0; r0 < u.rows; r0 += G::RPW) {
        const int r = r0 + sub;
        uint4 oa = make_uint4(0, 0, 0, 0), ob = oa;
        if (u.state == kUse) {
          // rows past the unit read what an earlier one left there, and are not written
          const uint4* src = reinterpret_cast<const uint4*>(st + r * (D * 2));
          oa = src[pa];
          ob = src[pb];
          if ((NORM || p.rope.rot > 0) && r0 < u.turned) {
            const Vals y = c.apply<D, NORM>(unpack16(oa, ob, inter), turns, p.rope.eps);
            if (r < u.turned) pack16(y, inter, oa, ob);
          }
        }
        if (r < u.rows) {
          store_pieces((APPEND && r >= u.turned ? vout : out) + r * pitch, pa, pb, oa, ob, one);
        }
      }
    }
    __syncwarp();  // every lane has read the stage
    if (lane == 0) tc::mbar_arrive(bar.empty + turn.s);
  }
}

// The same with every d / 16 lanes taking a row by themselves, straight from
// memory: 24 warps an SM hide the way from position to angles to results.  What
// a row costs is nearly the same whatever its token has, where a ring's unit costs the
// most of 4 KB even if it has 256 bytes: see use_rows().
constexpr int kRowThreads = 256, kRowCtas = 3;

template <int D, bool NORM, bool APPEND>
__global__ void __launch_bounds__(kRowThreads, kRowCtas) fwd_rows_kernel(const FwdParams p) {
  using G = Geo<D>;
  constexpr int ROWS = kRowThreads / G::LPR;  // of a CTA at a time
  __shared__ __align__(16) float w_s[2 * D];
  // one sequence a thread is loaded here and looked at behind the rows, which do not wait for it
  const int64_t seq = int64_t(blockIdx.x) * kRowThreads + threadIdx.x;
  SeqNumbers numbers;
  if (APPEND && seq < p.cache.n_seqs) numbers.load(p.cache, seq);
  if constexpr (NORM) {
    stage_weights<D>(p.rope, w_s);
    __syncthreads();
  }
  const int l = threadIdx.x % G::LPR, sub = threadIdx.x / G::LPR, heads = p.hq + (APPEND ? 2 : 1) * p.hkv;
  const bool inter = p.rope.interleaved != 0, turns = l < (p.rope.rot >> 4);
  int pa, pb;
  pieces<D>(l, p.rope.rot, inter, pa, pb);
  const bool one = p.wide && pb == pa + 1;
  // the CTA's first row as token and head, and what a step adds to them
  const int64_t base = int64_t(blockIdx.x) * ROWS, step = int64_t(gridDim.x) * ROWS;
  int64_t tok0 = base / heads;
  const int64_t d_tok = step / heads;
  int h0 = int(base - tok0 * heads);
  const int d_h = int(step - d_tok * heads);
  for (; tok0 < p.n_rows; tok0 += d_tok) {
    const unsigned at = unsigned(h0 + sub), over = at / unsigned(heads);
    const int64_t tok = tok0 + over;
    int h = int(at - over * unsigned(heads));
    int pos = 0, state = kSkip;
    int64_t slot = 0;
    if (tok < p.n_rows) {
      if constexpr (APPEND) paged_place(p, int(tok), pos, state, slot);
      else plain_place(p.positions, p.n_tokens, p.t_pad, p.rope.table_rows, int(tok), pos, state);
    }
    const Rows* src = &p.q;
    int kind = 0;  // 0: queries, 1: keys, 2: values
    if (h >= p.hq) {
      h -= p.hq;
      kind = 1;
      src = &p.k;
      if (APPEND && h >= p.hkv) {
        h -= p.hkv;
        kind = 2;
        src = &p.v;
      }
    }
    uint4 oa = make_uint4(0, 0, 0, 0), ob = oa;
    if (state == kUse) {
      const uint4* x = reinterpret_cast<const uint4*>(src->p + tok * src->stride + int64_t(h) * (D * 2));
      oa = x[pa];
      ob = x[pb];
    }
    if (NORM || p.rope.rot > 0) {
      // the lanes of a row agree; those of rows without one take part in the sums with zeros
      Coefs c;
      uint64_t wa[4], wb[4];
      if (turns) {
        const float* row = p.rope.table + int64_t(state == kUse ? pos : 0) * p.rope.rot + 8 * l;
        load_p4(row, c.ca);
        load_p4(row + (p.rope.rot >> 1), c.sa);
      }
      if constexpr (NORM) {
        load_p4(w_s + (kind ? D : 0) + 16 * l, wa);
        load_p4(w_s + (kind ? D : 0) + 16 * l + 8, wb);
      }
      c.weigh<NORM>(turns, wa, wb);
      const Vals y = c.apply<D, NORM>(unpack16(oa, ob, inter), turns, p.rope.eps);
      if (state == kUse && kind < 2) pack16(y, inter, oa, ob);
    }
    if (state != kSkip) {
      uint8_t* to;
      if (APPEND && kind) {
        to = static_cast<uint8_t*>(kind == 1 ? p.cache.k_cache : p.cache.v_cache) +
             (slot + int64_t(h) * p.cache.page_size) * (D * 2);
      } else {
        const RowsOut& dst = kind ? p.ko : p.qo;
        to = dst.p + tok * dst.stride + int64_t(h) * (D * 2);
      }
      store_pieces(to, pa, pb, oa, ob, one);
    }
    h0 += d_h;
    if (h0 >= heads) {
      h0 -= heads;
      ++tok0;
    }
  }
  if constexpr (APPEND) {
    if (seq < p.cache.n_seqs) numbers.check(p, seq);
    check_seqs(p, seq + int64_t(gridDim.x) * kRowThreads, int64_t(gridDim.x) * kRowThreads);
  }
}

// ------------------------------------------------------------------ gradient

struct BwdParams {
  Rope rope;
  const int32_t* positions;
  const int32_t* n_tokens;
  int64_t n_rows;
  int32_t t_pad, hq, hkv;
  Rows gq, gk, q, k;
  RowsOut dq, dk;
  float* partial;  // [grid][2][D]
  int32_t wide;    // dq and dk rows are 32-byte aligned
};

constexpr int kBwdMaxGrid = 608;  // CTAs: bounds the partial sums

// 16 values of a lane from a row in shared memory
template <bool F32>
__device__ __forceinline__ Vals load16(const uint8_t* row, int pa, int pb, bool inter) {
  if constexpr (F32) {
    Vals v;
    load_p4(reinterpret_cast<const float*>(row) + 8 * pa, v.a);
    load_p4(reinterpret_cast<const float*>(row) + 8 * pb, v.b);
    if (inter) {
      uint64_t t[8] = {v.a[0], v.a[1], v.a[2], v.a[3], v.b[0], v.b[1], v.b[2], v.b[3]};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a0, b0, a1, b1;
        unf2(t[2 * i], a0, b0);
        unf2(t[2 * i + 1], a1, b1);
        v.a[i] = f2(a0, a1);
        v.b[i] = f2(b0, b1);
      }
    }
    return v;
  } else {
    return unpack16(reinterpret_cast<const uint4*>(row)[pa], reinterpret_cast<const uint4*>(row)[pb], inter);
  }
}

// 32 bytes, one whole sector, in a store
__device__ __forceinline__ void store32(uint8_t* at, uint64_t a, uint64_t b, uint64_t c, uint64_t d) {
  asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(at), "l"(a), "l"(b), "l"(c), "l"(d) : "memory");
}

// `wide`: rows are 32-byte aligned.  Where a lane's 16-byte pieces lie two and
// two together they then leave as one store; as two, each would touch half a sector.
template <bool F32>
__device__ __forceinline__ void store16(uint8_t* row, int pa, int pb, const Vals& v, bool inter, bool wide) {
  if constexpr (F32) {
    uint64_t t[8] = {v.a[0], v.a[1], v.a[2], v.a[3], v.b[0], v.b[1], v.b[2], v.b[3]};
    if (inter) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a0, a1, b0, b1;
        unf2(v.a[i], a0, a1);
        unf2(v.b[i], b0, b1);
        t[2 * i] = f2(a0, b0);
        t[2 * i + 1] = f2(a1, b1);
      }
    }
    if (wide) {
      store32(row + 32 * pa, t[0], t[1], t[2], t[3]);
      store32(row + 32 * pb, t[4], t[5], t[6], t[7]);
      return;
    }
    ulonglong2* a = reinterpret_cast<ulonglong2*>(row + 32 * pa);
    ulonglong2* b = reinterpret_cast<ulonglong2*>(row + 32 * pb);
    a[0] = make_ulonglong2(t[0], t[1]);
    a[1] = make_ulonglong2(t[2], t[3]);
    b[0] = make_ulonglong2(t[4], t[5]);
    b[1] = make_ulonglong2(t[6], t[7]);
  } else {
    uint4 x, y;
    pack16(v, inter, x, y);
    store_pieces(row, pa, pb, x, y, wide && pb == pa + 1);
  }
}

// Where in a row the first value of a lane's packed pair j is (0..3: firsts, 4..7: seconds); the other is 1 further, or
// 2 where neighbours are paired.
__device__ __forceinline__ int weight_at(int j, int l, int pa, int pb, bool inter) {
  const int i = 2 * (j & 3), second = j >> 2;
  return inter ? 16 * l + 2 * i + second : 8 * (second ? pb : pa) + i;
}

// The gradient of a row, in z from that of its result: R(p)^T first, then with y = r z w: dw += (r z) x (`add`),
// dx = y - x (r^2 mean(y x)).
template <int D, bool NORM, class Add>
__device__ __forceinline__ void grad_row(Vals& z, const Vals& x, const uint64_t (&c)[4], const uint64_t (&sn)[4],
                                         const Vals& w, bool turns, bool live, float eps, Add add) {
  if (turns) {
    const Vals g = z;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      z.a[j] = fma2(g.a[j], c[j], mul2(g.b[j], sn[j]));
      z.b[j] = fma2(g.b[j], c[j], neg2(mul2(g.a[j], sn[j])));
    }
  }
  if constexpr (NORM) {
    const float rs = rstd<D>(x, eps);
    const uint64_t r2 = live ? f2(rs, rs) : 0;  // eps may be 0, and rs of a row of zeros infinite
    uint64_t dot[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      z.a[j] = mul2(z.a[j], r2);
      z.b[j] = mul2(z.b[j], r2);
    }
    add(z, x);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      z.a[j] = mul2(z.a[j], w.a[j]);
      z.b[j] = mul2(z.b[j], w.b[j]);
      dot[0] = fma2(z.a[j], x.a[j], dot[0]);
      dot[1] = fma2(z.b[j], x.b[j], dot[1]);
    }
    const float m = row_sum<Geo<D>::LPR>(sum2(add2(dot[0], dot[1]))) * (-1.f / D) * (live ? rs * rs : 0.f);
    const uint64_t m2 = f2(m, m);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      z.a[j] = fma2(x.a[j], m2, z.a[j]);
      z.b[j] = fma2(x.b[j], m2, z.b[j]);
    }
  }
}

// Row by row, as fwd_rows_kernel; a lane holds the sums of both weights.
constexpr int kBwdRowCtas = 2;

template <int D, bool NORM, bool GIN32, bool GOUT32>
__global__ void __launch_bounds__(kRowThreads, kBwdRowCtas) bwd_rows_kernel(const BwdParams p) {
  using G = Geo<D>;
  constexpr int GB = GIN32 ? 4 : 2, OB = GOUT32 ? 4 : 2, ROWS = kRowThreads / G::LPR;
  __shared__ __align__(16) float w_s[NORM ? 2 * D : 4];
  __shared__ float sum_s[NORM ? kRowThreads / 32 : 1][2 * D];
  if constexpr (NORM) {
    stage_weights<D>(p.rope, w_s);
    __syncthreads();
  }
  const int l = threadIdx.x % G::LPR, sub = threadIdx.x / G::LPR, heads = p.hq + p.hkv;
  const bool inter = p.rope.interleaved != 0, turns = l < (p.rope.rot >> 4);
  int pa, pb;
  pieces<D>(l, p.rope.rot, inter, pa, pb);
  const int64_t base = int64_t(blockIdx.x) * ROWS, step = int64_t(gridDim.x) * ROWS;
  int64_t tok0 = base / heads;
  const int64_t d_tok = step / heads;
  int h0 = int(base - tok0 * heads);
  const int d_h = int(step - d_tok * heads);
  Vals acc[2];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[0].a[j] = acc[0].b[j] = acc[1].a[j] = acc[1].b[j] = 0;
  for (; tok0 < p.n_rows; tok0 += d_tok) {
    const unsigned at = unsigned(h0 + sub), over = at / unsigned(heads);
    const int64_t tok = tok0 + over;
    const int head = int(at - over * unsigned(heads)), kind = head < p.hq ? 0 : 1, h = kind ? head - p.hq : head;
    int pos = 0, state = kSkip;
    if (tok < p.n_rows) plain_place(p.positions, p.n_tokens, p.t_pad, p.rope.table_rows, int(tok), pos, state);
    const bool live = state == kUse;
    Vals z, x, w;
#pragma unroll
    for (int j = 0; j < 4; ++j) z.a[j] = z.b[j] = x.a[j] = x.b[j] = 0;
    uint64_t c[4], sn[4];
    if (live) {
      const Rows& g = kind ? p.gk : p.gq;
      z = load16<GIN32>(g.p + tok * g.stride + int64_t(h) * (D * GB), pa, pb, inter);
      if constexpr (NORM) {
        const Rows& src = kind ? p.k : p.q;
        x = load16<false>(src.p + tok * src.stride + int64_t(h) * (D * 2), pa, pb, inter);
      }
    }
    if (turns) {
      const float* row = p.rope.table + int64_t(live ? pos : 0) * p.rope.rot + 8 * l;
      load_p4(row, c);
      load_p4(row + (p.rope.rot >> 1), sn);
    }
    if constexpr (NORM) {
      load_p4(w_s + kind * D + 16 * l, w.a);
      load_p4(w_s + kind * D + 16 * l + 8, w.b);
    }
    grad_row<D, NORM>(z, x, c, sn, w, turns, live, p.rope.eps, [&](const Vals& zx, const Vals& x_) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t a = mul2(zx.a[j], x_.a[j]), b = mul2(zx.b[j], x_.b[j]);
        acc[0].a[j] = add2(acc[0].a[j], kind == 0 ? a : 0);
        acc[0].b[j] = add2(acc[0].b[j], kind == 0 ? b : 0);
        acc[1].a[j] = add2(acc[1].a[j], kind == 1 ? a : 0);
        acc[1].b[j] = add2(acc[1].b[j], kind == 1 ? b : 0);
      }
    });
    if (state != kSkip) {
      const RowsOut& o = kind ? p.dk : p.dq;
      store16<GOUT32>(o.p + tok * o.stride + int64_t(h) * (D * OB), pa, pb, z, inter, p.wide);
    }
    h0 += d_h;
    if (h0 >= heads) {
      h0 -= heads;
      ++tok0;
    }
  }
  if constexpr (NORM) {
    // rows of the warp, then warps of the CTA, in a fixed order
#pragma unroll
    for (int kind = 0; kind < 2; ++kind)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float lo, hi;
        unf2(j < 4 ? acc[kind].a[j] : acc[kind].b[j - 4], lo, hi);
#pragma unroll
        for (int o_ = G::LPR; o_ < 32; o_ <<= 1) {
          lo += __shfl_xor_sync(0xffffffffu, lo, o_);
          hi += __shfl_xor_sync(0xffffffffu, hi, o_);
        }
        if ((threadIdx.x & 31) < G::LPR) {
          const int at = weight_at(j, l, pa, pb, inter);
          sum_s[threadIdx.x >> 5][kind * D + at] = lo;
          sum_s[threadIdx.x >> 5][kind * D + at + (inter ? 2 : 1)] = hi;
        }
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kRowThreads) {
      float t = 0.f;
#pragma unroll
      for (int j = 0; j < kRowThreads / 32; ++j) t += sum_s[j][i];
      p.partial[int64_t(blockIdx.x) * 2 * D + i] = t;
    }
  }
  tc::grid_launch_dependents();
}

// Units of 2 KB of x and as many gradients (2 or 4 KB).  A warp takes queries
// or keys, not both, so that it holds one weight's sums (16 registers); the
// warps are divided as the units are.
template <int D, bool NORM, bool GIN32, bool GOUT32>
__global__ void __launch_bounds__(kThreads, kCtas) bwd_kernel(const BwdParams p) {
  using G = Geo<D>;
  constexpr int GB = GIN32 ? 4 : 2, OB = GOUT32 ? 4 : 2;
  constexpr int UROWS = 2048 / (D * 2);
  constexpr uint32_t XOFF = UROWS * D * GB, DATA = XOFF + 2048;
  using R = Ring<D, DATA>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool loads = warp == kWarps;
  const int wi = loads ? lane / kBatch : warp;  // whose ring; lanes past the last ring have no units
  const Bars<R> bar(smem, min(wi, kWarps - 1));
  float* w_s = reinterpret_cast<float*>(smem + R::OFF_W);

  const int sq = (p.hq + UROWS - 1) / UROWS, skv = (p.hkv + UROWS - 1) / UROWS;
  const int n_warps = gridDim.x * kWarps, n_q = min(max(int(int64_t(n_warps) * sq / (sq + skv)), 1), n_warps - 1);
  auto kind_of = [&](int w_) { return w_ * int(gridDim.x) + int(blockIdx.x) < n_q ? 0 : 1; };
  const int kind = kind_of(wi), per_token = kind == 0 ? sq : skv, heads = kind == 0 ? p.hq : p.hkv;
  const int me = wi * gridDim.x + blockIdx.x - (kind == 0 ? 0 : n_q), of = kind == 0 ? n_q : n_warps - n_q;
  const int64_t units = p.n_rows * per_token;
  const int mine = wi < kWarps ? units_for(units, me, of) : 0;
  const uint32_t table_bytes = p.rope.rot * 4;
  const int l = lane % G::LPR, sub = lane / G::LPR;
  const bool inter = p.rope.interleaved != 0, turns = l < (p.rope.rot >> 4);
  int pa, pb;
  pieces<D>(l, p.rope.rot, inter, pa, pb);

  if (loads) {
    const int j = lane % kBatch;
    if (threadIdx.x == 32 * kWarps) *bar.abort_flag = 0;
    if (j == 0 && wi < kWarps) bar.init();
    __syncwarp();
    ready_arrive();
    const Rows g_in = kind == 0 ? p.gq : p.gk, x_in = kind == 0 ? p.q : p.k;
    run_loader<R, false>(
        bar, wi, mine,
        [&](int i) {
          const int64_t u_at = unit_of(me, of, i);
          Place at{int(u_at / per_token), 0, 0, kPad, 0};
          at.part = int(u_at - int64_t(at.tok) * per_token);
          plain_place(p.positions, p.n_tokens, p.t_pad, p.rope.table_rows, at.tok, at.pos, at.state);
          return at;
        },
        [&](const Place& at, int, int stage) {
          uint8_t* st = bar.ring + stage * R::STAGE;
          uint64_t* fb = bar.full + stage;
          const int h = at.part * UROWS, rows = min(heads - h, UROWS);
          *reinterpret_cast<Unit*>(st + DATA + R::TABLE) = Unit{kind, h, rows, rows, at.state, at.tok, 0};
          if (at.state == kUse) {
            tc::mbar_arrive_expect_tx(fb, rows * (D * (GB + (NORM ? 2 : 0))) + table_bytes);
            tc::bulk_load(st, g_in.p + at.tok * g_in.stride + int64_t(h) * (D * GB), rows * (D * GB), fb);
            if constexpr (NORM)
              tc::bulk_load(st + XOFF, x_in.p + at.tok * x_in.stride + int64_t(h) * (D * 2), rows * (D * 2), fb);
            tc::bulk_load(st + DATA, p.rope.table + int64_t(at.pos) * p.rope.rot, table_bytes, fb);
          } else {
            tc::mbar_arrive(fb);
          }
        });
  } else {
  if constexpr (NORM) stage_weights<D>(p.rope, w_s);
  ready_wait();
  Vals w, acc;
#pragma unroll
  for (int j = 0; j < 4; ++j) acc.a[j] = acc.b[j] = 0;
  if constexpr (NORM) {
    load_p4(w_s + kind * D + 16 * l, w.a);
    load_p4(w_s + kind * D + 16 * l + 8, w.b);
  }
  const RowsOut o = kind == 0 ? p.dq : p.dk;
  Turn<R::NST> turn;
  for (int i = 0; i < mine; ++i, turn.next()) {
    if (!__all_sync(0xffffffffu, tc::mbar_wait(bar.full + turn.s, turn.phase, bar.abort_flag, &g_status_rope))) break;
    const uint8_t* st = bar.ring + turn.s * R::STAGE;
    const Unit u = *reinterpret_cast<const Unit*>(st + DATA + R::TABLE);
    uint64_t c[4], sn[4];
    if (turns && u.state == kUse) {
      const float* row = reinterpret_cast<const float*>(st + DATA) + 8 * l;
      load_p4(row, c);
      load_p4(row + (p.rope.rot >> 1), sn);
    }
    uint8_t* out = o.p + u.token * o.stride + int64_t(u.h) * (D * OB);
#pragma unroll 1
    for (int r0 = 0; r0 < u.rows; r0 += G::RPW) {
      const int r = r0 + sub;
      const bool live = r < u.rows;
      Vals z;
#pragma unroll
      for (int j = 0; j < 4; ++j) z.a[j] = z.b[j] = 0;
      if (u.state == kUse) {
        if (live) z = load16<GIN32>(st + r * (D * GB), pa, pb, inter);
        Vals x;
        if constexpr (NORM) {
#pragma unroll
          for (int j = 0; j < 4; ++j) x.a[j] = x.b[j] = 0;
          if (live) x = load16<false>(st + XOFF + r * (D * 2), pa, pb, inter);
        }
        grad_row<D, NORM>(z, x, c, sn, w, turns, live, p.rope.eps, [&](const Vals& zx, const Vals& x_) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc.a[j] = fma2(zx.a[j], x_.a[j], acc.a[j]);
            acc.b[j] = fma2(zx.b[j], x_.b[j], acc.b[j]);
          }
        });
      }
      if (live) store16<GOUT32>(out + r * (D * OB), pa, pb, z, inter, p.wide);
    }
    __syncwarp();  // every lane has read the stage
    if (lane == 0) tc::mbar_arrive(bar.empty + turn.s);
  }
  if constexpr (NORM) {
    // rows of the warp, then warps of the CTA, in a fixed order; a warp's ring is its own and no longer in use
    float* mine_s = reinterpret_cast<float*>(bar.ring);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float lo, hi;
      unf2(j < 4 ? acc.a[j] : acc.b[j - 4], lo, hi);
#pragma unroll
      for (int o_ = G::LPR; o_ < 32; o_ <<= 1) {
        lo += __shfl_xor_sync(0xffffffffu, lo, o_);
        hi += __shfl_xor_sync(0xffffffffu, hi, o_);
      }
      if (sub == 0) {
        const int at = weight_at(j, l, pa, pb, inter);
        mine_s[at] = lo;
        mine_s[at + (inter ? 2 : 1)] = hi;
      }
    }
  }
  }
  if constexpr (NORM) {
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
      float t = 0.f;
#pragma unroll
      for (int j = 0; j < kWarps; ++j)
        if (kind_of(j) == i / D) t += reinterpret_cast<const float*>(smem + j * R::WARP)[i % D];
      p.partial[int64_t(blockIdx.x) * 2 * D + i] = t;
    }
  }
  tc::grid_launch_dependents();
}

// Adds the CTAs' partial sums of a column in a fixed order: 32 columns a CTA.
__global__ void __launch_bounds__(1024) bwd_sum_kernel(const float* partial, int n, int d, float* dwq, float* dwk) {
  __shared__ float s[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, col = blockIdx.x * 32 + tx;
  tc::grid_wait_prior();
  float t = 0.f;
  for (int i = ty; i < n; i += 32) t += partial[int64_t(i) * 2 * d + col];
  s[ty][tx] = t;
  __syncthreads();
  if (ty == 0) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += s[i][tx];
    if (col < d) dwq[col] = sum;
    else dwk[col - d] = sum;
  }
}

// ------------------------------------------------------------------ table

struct Freqs {
  double f[64];
};

__global__ void __launch_bounds__(256) table_kernel(float* table, int64_t n, int half, double scale, const Freqs fr) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n * half) return;
  const int64_t pos = i / half;
  const int j = int(i - pos * half);
  double s, c;
  sincos(double(pos) * fr.f[j], &s, &c);
  table[pos * 2 * half + j] = float(scale * c);
  table[pos * 2 * half + half + j] = float(scale * s);
}

// ------------------------------------------------------------------ host side

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

bool aligned32(const void* p, int64_t stride) { return ((reinterpret_cast<uintptr_t>(p) | uintptr_t(stride)) & 31) == 0; }

bool rows_ok(const void* p, int64_t stride, int heads, int d, int elem) {
  // the largest strides in use are those of fused projections; 2^40 elements keep all byte offsets in 64 bits
  return p && aligned16(p) && stride >= int64_t(heads) * d && stride < (int64_t(1) << 40) && (stride * elem) % 16 == 0;
}

bool rope_ok(const tpa_rope_params* r, int d, bool need_table) {
  if (!r || (!r->q_weight) != (!r->k_weight) || !(r->eps >= 0.f) || std::isinf(r->eps)) return false;
  if (r->q_weight && (!aligned16(r->q_weight) || !aligned16(r->k_weight))) return false;
  if (r->weight_type != TPA_WEIGHT_F32 && r->weight_type != TPA_WEIGHT_BF16) return false;
  if (!r->table) return !need_table;
  return aligned16(r->table) && r->table_rows >= 1 && r->rot_dim >= 16 && r->rot_dim <= d && r->rot_dim % 16 == 0;
}

Rope make_rope(const tpa_rope_params* r) {
  Rope o;
  o.table = r->table;
  o.wq = r->q_weight;
  o.wk = r->k_weight;
  o.table_rows = r->table_rows;
  o.rot = r->table ? r->rot_dim : 0;
  o.interleaved = r->interleaved != 0;
  o.w_bf16 = r->weight_type == TPA_WEIGHT_BF16;
  o.eps = r->eps;
  return o;
}

int units_of(int heads, int d) {
  const int rows = 4096 / (d * 2);
  return (heads + rows - 1) / rows;
}

int num_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return 148;
  }
  return sms;
}

// Row by row instead of through rings: tokens of few heads, whose units would be small (16384 of which 14000 real, d 128:
// 2/1 heads 9.0 us instead of 21.4, 4/4 21.2 and 22.6, 8/8 39.0 and 29.7; 16000 appended: 2/1 heads 16.7 instead of
// 26.0, 4/2 30.3 and 26.5, d 64 8/2 22.0 and 24.4), and calls of one pass over the grid, where the rings' start
// counts (32/8 heads: 100 tokens 3.3 us instead of 4.3, 200 3.9 and 4.65, 300 4.5 and 4.85, 400 5.55 and 5.05; one
// appended token 3.7 and 4.75, 200 5.3 and 5.9, 250 6.2 and 6.15, 400 8.15 and 6.4; 16/2 heads, 400 appended 5.45
// and 6.1, 600 6.6 both, 800 8.2 and 7.3): up to 3 MB.
bool use_rows(const FwdParams& p, int d, bool append) {
  const int64_t token = int64_t(p.hq + (append ? 2 : 1) * p.hkv) * d * 2;
  return token <= (append ? 1536 : 2048) || token * p.n_rows <= (3 << 20);
}

// Two CTAs an SM, or one for every unit where there are fewer.
int grid_of(int64_t units) {
  const int64_t most = kCtas * int64_t(num_sms());
  const int64_t n = units < most ? units : most;
  return int(n < 1 ? 1 : n < kBwdMaxGrid ? n : kBwdMaxGrid);
}

template <int D, bool NORM, bool APPEND>
int launch_fwd_as(const FwdParams& p, cudaStream_t st) {
  if (use_rows(p, D, APPEND)) {
    constexpr int rows = kRowThreads / Geo<D>::LPR;
    const int64_t n = (p.n_rows * (p.hq + (APPEND ? 2 : 1) * p.hkv) + rows - 1) / rows, most = kRowCtas * int64_t(num_sms());
    fwd_rows_kernel<D, NORM, APPEND><<<unsigned(n < most ? n : most), kRowThreads, 0, st>>>(p);
    TPA_CUDA_TRY(cudaGetLastError());
    return TPA_OK;
  }
  using R = Ring<D, 4096>;
  const int per_token = p.sq + p.sk + p.sv;
  TPA_CUDA_TRY(cudaFuncSetAttribute(fwd_kernel<D, NORM, APPEND>, cudaFuncAttributeMaxDynamicSharedMemorySize, R::BYTES));
  fwd_kernel<D, NORM, APPEND><<<grid_of(p.n_rows * per_token), kThreads, R::BYTES, st>>>(p);
  TPA_CUDA_TRY(cudaGetLastError());
  return TPA_OK;
}

template <int D, bool APPEND>
int launch_fwd(const FwdParams& p, bool norm, cudaStream_t st) {
  return norm ? launch_fwd_as<D, true, APPEND>(p, st) : launch_fwd_as<D, false, APPEND>(p, st);
}

// As use_rows(), by the values of a token and of the call whatever the gradients' type, since the borders are the same
// (bf16 and fp32): 16384 rows, d 128 2/1 heads 13.9 us instead of 22.3 and 19.2 instead of 24.4, 4/2 27.5 (rings 23.5)
// and 31.0 (28.0), d 64 4/2 12.7 instead of 21.4 and 17.7 instead of 23.0, 8/2 22.1 (22.4) and 26.2 (25.4); 32/8
// heads: 100 rows 5.55 instead of 6.8 and 5.65 instead of 6.9, 200 7.2 (7.5) and 7.5 (7.6), 250 7.7 (7.65) and 8.0
// (7.7), 400 8.7 (8.0) and 8.95 (8.45).  Beyond 2 MB of bf16 values rings.
bool use_bwd_rows(const BwdParams& p, int d) {
  const int64_t token = int64_t(p.hq + p.hkv) * d * 2;
  return token <= 1024 || token * p.n_rows <= (2 << 20);
}

template <int D, bool NORM, bool GIN32, bool GOUT32>
int launch_bwd_as(const BwdParams& p, float* dwq, float* dwk, cudaStream_t st) {
  constexpr int UROWS = 2048 / (D * 2);
  using R = Ring<D, UROWS * D * (GIN32 ? 4 : 2) + 2048>;
  const int64_t units = p.n_rows * ((p.hq + UROWS - 1) / UROWS + (p.hkv + UROWS - 1) / UROWS);
  int grid = grid_of(units);
  if (use_bwd_rows(p, D)) {
    constexpr int rows = kRowThreads / Geo<D>::LPR;
    const int64_t n = (p.n_rows * (p.hq + p.hkv) + rows - 1) / rows, most = kBwdRowCtas * int64_t(num_sms());
    grid = int(n < 1 ? 1 : n < most ? n : most);
    if (grid > kBwdMaxGrid) grid = kBwdMaxGrid;
    bwd_rows_kernel<D, NORM, GIN32, GOUT32><<<grid, kRowThreads, 0, st>>>(p);
  } else {
    TPA_CUDA_TRY(cudaFuncSetAttribute(bwd_kernel<D, NORM, GIN32, GOUT32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      R::BYTES));
    bwd_kernel<D, NORM, GIN32, GOUT32><<<grid, kThreads, R::BYTES, st>>>(p);
  }
  TPA_CUDA_TRY(cudaGetLastError());
  if (!NORM) return TPA_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * D / 32);
  cfg.blockDim = dim3(1024);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  TPA_CUDA_TRY(cudaLaunchKernelEx(&cfg, bwd_sum_kernel, static_cast<const float*>(p.partial), grid, D, dwq, dwk));
  return TPA_OK;
}

template <int D, bool GIN32, bool GOUT32>
int launch_bwd(const BwdParams& p, bool norm, float* dwq, float* dwk, cudaStream_t st) {
  return norm ? launch_bwd_as<D, true, GIN32, GOUT32>(p, dwq, dwk, st)
              : launch_bwd_as<D, false, GIN32, GOUT32>(p, dwq, dwk, st);
}

}  // namespace

TPA_DEFINE_STATUS_READER(tpa_internal_status_rope, g_status_rope)

extern "C" int tpa_rope_table(float* table, int32_t n_positions, int32_t rot_dim, double base,
                              const double* inv_freq, double scale, void* stream) {
  TPA_NVTX_RANGE("tpa_rope_table");
  if (!table || !aligned16(table) || n_positions < 1 || rot_dim < 16 || rot_dim > 128 || rot_dim % 16 ||
      !std::isfinite(scale))
    return TPA_ERR_INVALID_ARG;
  if (!inv_freq && !(base > 0.0 && std::isfinite(base))) return TPA_ERR_INVALID_ARG;
  Freqs fr = {};
  for (int j = 0; j < rot_dim / 2; ++j) {
    fr.f[j] = inv_freq ? inv_freq[j] : std::pow(base, -2.0 * j / rot_dim);
    if (!std::isfinite(fr.f[j])) return TPA_ERR_INVALID_ARG;
  }
  const int64_t n = int64_t(n_positions) * (rot_dim / 2);
  if ((n + 255) / 256 > 0x7fffffff) return TPA_ERR_INVALID_ARG;
  table_kernel<<<unsigned((n + 255) / 256), 256, 0, static_cast<cudaStream_t>(stream)>>>(table, n_positions,
                                                                                        rot_dim / 2, scale, fr);
  TPA_CUDA_TRY(cudaGetLastError());
  return TPA_OK;
}

extern "C" int tpa_qk_norm_rope_fwd(const int32_t* positions, const int32_t* n_tokens, int32_t t_pad, int64_t n_rows,
                                    const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                    const tpa_rope_params* rope, void* q_out, int64_t q_out_stride, void* k_out,
                                    int64_t k_out_stride, int32_t n_heads_q, int32_t n_heads_kv, int32_t head_dim,
                                    void* stream) {
  TPA_NVTX_RANGE("tpa_qk_norm_rope_fwd");
  const int d = head_dim;
  if ((d != 64 && d != 128) || n_rows < 0 || n_rows > 0x7fffffff || n_heads_q < 1 || n_heads_kv < 1 ||
      n_heads_q > 65535 || n_heads_kv > 65535 || !rope_ok(rope, d, true))
    return TPA_ERR_INVALID_ARG;
  if (n_tokens && (t_pad < 1 || n_rows % t_pad)) return TPA_ERR_INVALID_ARG;
  if (n_rows == 0) return TPA_OK;
  if (!positions || !rows_ok(q, q_stride, n_heads_q, d, 2) || !rows_ok(k, k_stride, n_heads_kv, d, 2) ||
      !rows_ok(q_out, q_out_stride, n_heads_q, d, 2) || !rows_ok(k_out, k_out_stride, n_heads_kv, d, 2))
    return TPA_ERR_INVALID_ARG;
  FwdParams p = {};
  p.rope = make_rope(rope);
  p.positions = positions;
  p.n_tokens = n_tokens;
  p.t_pad = t_pad;
  p.n_rows = n_rows;
  p.hq = n_heads_q;
  p.hkv = n_heads_kv;
  p.sq = units_of(n_heads_q, d);
  p.sk = units_of(n_heads_kv, d);
  p.q = {static_cast<const uint8_t*>(q), q_stride * 2};
  p.k = {static_cast<const uint8_t*>(k), k_stride * 2};
  p.qo = {static_cast<uint8_t*>(q_out), q_out_stride * 2};
  p.ko = {static_cast<uint8_t*>(k_out), k_out_stride * 2};
  p.wide = aligned32(q_out, p.qo.stride) && aligned32(k_out, p.ko.stride);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d == 128 ? launch_fwd<128, false>(p, rope->q_weight, st) : launch_fwd<64, false>(p, rope->q_weight, st);
}

extern "C" uint64_t tpa_qk_norm_rope_bwd_workspace_bytes(int32_t head_dim) {
  if (head_dim != 64 && head_dim != 128) return 0;
  return uint64_t(kBwdMaxGrid) * 2 * head_dim * sizeof(float);
}

extern "C" int tpa_qk_norm_rope_bwd(const int32_t* positions, const int32_t* n_tokens, int32_t t_pad, int64_t n_rows,
                                    const void* dq_out, int64_t dq_out_stride, const void* dk_out,
                                    int64_t dk_out_stride, int32_t grad_in, const void* q, int64_t q_stride,
                                    const void* k, int64_t k_stride, const tpa_rope_params* rope, void* dq,
                                    int64_t dq_stride, void* dk, int64_t dk_stride, int32_t grad_out,
                                    float* dq_weight, float* dk_weight, void* workspace, uint64_t workspace_bytes,
                                    int32_t n_heads_q, int32_t n_heads_kv, int32_t head_dim, void* stream) {
  TPA_NVTX_RANGE("tpa_qk_norm_rope_bwd");
  const int d = head_dim;
  if ((d != 64 && d != 128) || n_rows < 0 || n_rows > 0x7fffffff || n_heads_q < 1 || n_heads_kv < 1 ||
      n_heads_q > 65535 || n_heads_kv > 65535 || !rope_ok(rope, d, true))
    return TPA_ERR_INVALID_ARG;
  if (n_tokens && (t_pad < 1 || n_rows % t_pad)) return TPA_ERR_INVALID_ARG;
  if ((grad_in != TPA_GRAD_F32 && grad_in != TPA_GRAD_BF16) || (grad_out != TPA_GRAD_F32 && grad_out != TPA_GRAD_BF16))
    return TPA_ERR_INVALID_ARG;
  const bool norm = rope->q_weight != nullptr;
  if (norm) {
    if (!dq_weight || !dk_weight || !workspace || !aligned16(workspace) ||
        (reinterpret_cast<uintptr_t>(dq_weight) & 3) || (reinterpret_cast<uintptr_t>(dk_weight) & 3))
      return TPA_ERR_INVALID_ARG;
    if (workspace_bytes < tpa_qk_norm_rope_bwd_workspace_bytes(d)) return TPA_ERR_BUFFER_TOO_SMALL;
  }
  const int gi = grad_in == TPA_GRAD_F32 ? 4 : 2, go = grad_out == TPA_GRAD_F32 ? 4 : 2;
  if (n_rows > 0) {
    if (!positions || !rows_ok(dq_out, dq_out_stride, n_heads_q, d, gi) ||
        !rows_ok(dk_out, dk_out_stride, n_heads_kv, d, gi) || !rows_ok(dq, dq_stride, n_heads_q, d, go) ||
        !rows_ok(dk, dk_stride, n_heads_kv, d, go))
      return TPA_ERR_INVALID_ARG;
    if (norm && (!rows_ok(q, q_stride, n_heads_q, d, 2) || !rows_ok(k, k_stride, n_heads_kv, d, 2)))
      return TPA_ERR_INVALID_ARG;
  } else if (!norm) {
    return TPA_OK;
  }
  BwdParams p = {};
  p.rope = make_rope(rope);
  p.positions = positions;
  p.n_tokens = n_tokens;
  p.t_pad = t_pad;
  p.n_rows = n_rows;
  p.hq = n_heads_q;
  p.hkv = n_heads_kv;
  p.gq = {static_cast<const uint8_t*>(dq_out), dq_out_stride * gi};
  p.gk = {static_cast<const uint8_t*>(dk_out), dk_out_stride * gi};
  p.q = {static_cast<const uint8_t*>(q), q_stride * 2};
  p.k = {static_cast<const uint8_t*>(k), k_stride * 2};
  p.dq = {static_cast<uint8_t*>(dq), dq_stride * go};
  p.dk = {static_cast<uint8_t*>(dk), dk_stride * go};
  p.partial = static_cast<float*>(workspace);
  p.wide = aligned32(dq, p.dq.stride) && aligned32(dk, p.dk.stride);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto run = [&](auto gin, auto gout) {
    constexpr bool A = decltype(gin)::value, B = decltype(gout)::value;
    return d == 128 ? launch_bwd<128, A, B>(p, norm, dq_weight, dk_weight, st)
                    : launch_bwd<64, A, B>(p, norm, dq_weight, dk_weight, st);
  };
  using T = std::true_type;
  using F = std::false_type;
  if (gi == 4) return go == 4 ? run(T{}, T{}) : run(T{}, F{});
  return go == 4 ? run(F{}, T{}) : run(F{}, F{});
}

int tpa_internal_check_paged(const tpa_paged_view* c) {
  if (!c || !c->k_cache || !c->v_cache || !c->offsets) return TPA_ERR_INVALID_ARG;
  if (!aligned16(c->k_cache) || !aligned16(c->v_cache)) return TPA_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return TPA_ERR_INVALID_ARG;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return TPA_ERR_INVALID_ARG;
  // a batch of no sequences has no rows; its arrays of one entry a sequence may be anything
  const bool none = c->n_seqs == 0 && c->n_rows == 0;
  if (!none && (c->n_seqs < 1 || !c->pages || !c->kv_lens)) return TPA_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->max_pages < (none ? 0 : 1) || c->page_stride < c->max_pages || c->n_rows < 0 ||
      c->n_rows >= (1 << 30) || c->n_heads_kv < 1 || c->n_heads_kv > 65535)
    return TPA_ERR_INVALID_ARG;
  if (int64_t(c->n_pages) * c->n_heads_kv >= (int64_t(1) << 31) / c->page_size) return TPA_ERR_INVALID_ARG;
  // positions, and differences of them and of rows, are held in 32 bits
  if (int64_t(c->max_pages) * c->page_size >= (int64_t(1) << 30)) return TPA_ERR_INVALID_ARG;
  return TPA_OK;
}

extern "C" int tpa_paged_append(const tpa_paged_view* cache, const void* k, int64_t k_stride, const void* v,
                                int64_t v_stride, const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
                                int32_t n_heads_q, const tpa_rope_params* rope, void* stream) {
  TPA_NVTX_RANGE("tpa_paged_append");
  const int rc = tpa_internal_check_paged(cache);
  if (rc != TPA_OK) return rc;
  const int d = cache->head_dim;
  if (n_heads_q < 0 || n_heads_q > 65535 || !rope_ok(rope, d, false)) return TPA_ERR_INVALID_ARG;
  if (cache->n_rows == 0) return TPA_OK;
  if (!rows_ok(k, k_stride, cache->n_heads_kv, d, 2) || !rows_ok(v, v_stride, cache->n_heads_kv, d, 2))
    return TPA_ERR_INVALID_ARG;
  if (n_heads_q > 0 && (!rows_ok(q, q_stride, n_heads_q, d, 2) || !rows_ok(q_out, q_out_stride, n_heads_q, d, 2)))
    return TPA_ERR_INVALID_ARG;
  FwdParams p = {};
  p.rope = make_rope(rope);
  p.n_rows = cache->n_rows;
  p.hq = n_heads_q;
  p.hkv = cache->n_heads_kv;
  p.sq = n_heads_q ? units_of(n_heads_q, d) : 0;
  p.sk = units_of(cache->n_heads_kv, d);
  p.sv = units_of(2 * cache->n_heads_kv, d) == 1 ? 0 : p.sk;  // keys and values in one unit where they fit
  p.q = {static_cast<const uint8_t*>(q), q_stride * 2};
  p.k = {static_cast<const uint8_t*>(k), k_stride * 2};
  p.v = {static_cast<const uint8_t*>(v), v_stride * 2};
  p.qo = {static_cast<uint8_t*>(q_out), q_out_stride * 2};
  p.cache = *cache;
  p.wide = (!n_heads_q || aligned32(q_out, p.qo.stride)) && aligned32(cache->k_cache, 0) && aligned32(cache->v_cache, 0);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d == 128 ? launch_fwd<128, true>(p, rope->q_weight, st) : launch_fwd<64, true>(p, rope->q_weight, st);
}
