// The next token of each row of logits: temperature, top-k, top-p, min-p and a
// draw from a given uniform number.
//
// Tokens stand in the order of their logits, highest first, equal ones by
// index: the order of a 64-bit number (the logit as an ordered 32-bit key, below it the index
// complemented), all of which differ.  Top-k and top-p each keep the tokens from a cut on.
//
// Weights.  A draw has to be the same whatever the order of summation, so weights exp((x - max) / T) are
// whole numbers: 2^y, y = x c - M with c = log2(e) / T as a pair of fp32 and M a multiple of 1/32,
// y = k / 32 + g, 2^(k / 32) from a table to 30 bits, 2^g - 1 by its series (|g| <= 1/64, four terms, off by
// 2^-39).  The product of the two is off by 2^-29 of itself (the rounding of g and of the series' value),
// shifted to 31 + s bits at most, s = 32 - log2 vocabulary, and the part below 1 is cut off there.  A row's sum fits in 64
// bits, is exact, and nothing depends on the grouping: borders are off by what the weights are, 2^-29 of the whole, and by
// the units cut off, vocabulary 2^-(30 + s) of the largest weight at most (2^-26 for a vocabulary of 2^18).  Two kinds of sums are not: those of
// the histograms leave out the bits of a weight below 2^-30 of its bin's largest, 2^-28 of itself at most; and a row
// without any cut is summed in units that grow with the largest logit met (sum_online), which keeps parts of the last units and cuts off
// up to three of those a token, by the order of its logits and by its split.
//
// A row's way (sample_kernel; a cluster of 1 to 8 CTAs of 8 warps, each warp a contiguous part of the row):
//   1. the maximum, and for top-k a bound below which nothing is kept (the warp's threads' own maxima);
//   2. the tokens from a bound on are collected, each warp's in its list of 512 in shared memory, and the whole row's weights are
//      summed where top-p is of them.  Top-p's bound is a guess, max - 9 T (of a model's logits that is
//      nearly all the weight), which the listed weights confirm; else a wider one, max - 11 T, and then
//      one that no token below can pass (each weighs less than (1 - p) / vocabulary of the whole);
//   3. up to 256 candidates, one a thread of the first CTA, are ranked against each other; more, or a list that was too
//      short, have their cuts found by histograms (in shared memory, joined over the cluster): 1024 bins of 1/32 of a factor of 2
//      of the weights, then of the numbers within the bin, until 256 tokens are left; then each part's sum, and the
//      part in which the running sum passes u of the whole.
// Rows without any cut go through once (plain_kernel): each warp moves its sum when it meets a larger maximum.
//
// What it has to do is to read the row: 64 rows of 151936 in bf16, 19 MB, 2.9 us at the copy's rate.  Without a cut it is bound by
// the weights' instructions, 28 a token of which 7.5 us of issue slots are made here, and by a start and an end as long: 17.4 us.
// With cuts it is bound by passes over a row that follow one another, with a cluster barrier after each, in which a warp has
// little to overlap: 64 rows of 151936 in fp32, each with its own parameters, 42 us; with rows among them whose
// top-p keeps thousands of tokens, which then have the device to themselves, 72 to 79; 64 such rows (T = 1.3, p = 0.97) 112;
// 499 rows of 32000 45 us; one row of 32000 9.3 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "device_common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace {

__device__ unsigned int g_status_sample = 0;

constexpr int kMostCtas = 8;  // of a row: a cluster
constexpr int kMostVocab = 1 << 24;  // beyond, a weight's unit times the vocabulary is no longer small
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMostParts = kMostCtas * kWarps;  // contiguous parts of a row, one a warp
constexpr int kBins = 1024;
constexpr int kBinsEach = kBins / kThreads;  // bins that a thread adds up, at most
constexpr int kFew = kThreads;     // tokens that are ranked against each other, one a thread
constexpr int kList = 512;         // candidates that a warp has room for
constexpr int kBinsPerBit = 32;    // bins of the first level in a factor of 2 of the weights
constexpr int kTops = 8;           // maxima that a thread keeps, for top-k's bound
constexpr int kMostLevels = 8;
constexpr float kHead = 9.f, kWider = 11.f;  // distances from the maximum, in T, within which top_p's cut is looked for first

// round(2^(i / 32) * 2^30)
__constant__ uint32_t kRoots[32] = {
    1073741824u, 1097253708u, 1121280436u, 1145833280u, 1170923762u, 1196563654u, 1222764986u, 1249540052u,
    1276901417u, 1304861917u, 1333434672u, 1362633090u, 1392470869u, 1422962010u, 1454120821u, 1485961921u,
    1518500250u, 1551751076u, 1585730000u, 1620452965u, 1655936265u, 1692196547u, 1729250827u, 1767116489u,
    1805811301u, 1845353420u, 1885761398u, 1927054196u, 1969251188u, 2012372174u, 2056437387u, 2101467502u};

struct Params {
  const void* logits;
  int64_t row_stride;
  const float* temperature;
  const float* top_p;
  const float* min_p;
  const int32_t* top_k;
  const float* u;
  int32_t* tokens;
  float* logp;
  float temperature_all, top_p_all, min_p_all;
  int32_t top_k_all;
  int32_t vocab, shift;  // shift: 32 - log2 of the vocabulary, rounded up
  int32_t ctas;          // of a row
};

constexpr float kLargest = 3.402823466e38f;  // finite number

// A logit as it is compared: NaN as -inf, +inf as the largest finite number, one zero.
__device__ __forceinline__ float clean(float x) { return fminf(fmaxf(x, -INFINITY), kLargest) + 0.f; }

__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
// A token's number: the key of its logit, and below it `bits` bits of its index, complemented (bits: as many as indexes have, so that a
// histogram's bins over a range of numbers hold equal logits apart).
__device__ __forceinline__ uint64_t number_of(float x, int i, int bits) {
  return uint64_t(key_of(x)) << bits | (((1u << bits) - 1) - uint32_t(i));
}
__device__ __forceinline__ float logit_of(uint64_t n, int bits) { return of_key(uint32_t(n >> bits)); }
__device__ __forceinline__ int index_of(uint64_t n, int bits) {
  const uint32_t most = (1u << bits) - 1;
  return int(most - (uint32_t(n) & most));
}

constexpr float kMagic = 1.5f * 262144.f;  // its last place is 1/32
constexpr int kMagicBits = 0x48c00000;

// What a row's weights are made with.  y = x c - M, c = log2(e) / T = ch + cl, and M the multiple of 1/32 next to (max x) c, so that
// the maximum's weight is 2^(30 + shift) but for a factor of 2^(1/64) (all have it).  For a maximum so far
// from 0 that M does not fit beside kMagic's last place, x is first taken from the maximum (FAR): d + e = x - max, M = 0.
struct Scale {
  float m, ch, cl, base;  // base = kMagic - M
  float least;            // logits from here down weigh less than 2^-(30 + shift) of the largest: nothing
  int shift, s0;          // s0: 32 times the shift of a weight with y = 0, and kMagic's bits, and 31 to round up
};

// A weight, a whole number of at most 31 + shift bits: root (1 + q) shifted.
struct Weight {
  uint32_t w;
  int by;
  __device__ __forceinline__ uint64_t value() const {
    uint64_t r;
    asm("shr.b64 %0, %1, %2;" : "=l"(r) : "l"(uint64_t(w) << 32), "r"(by));
    return r;
  }
};

template <bool FAR>
struct Weigher {
  Scale k;
  const uint32_t* roots;
  uint32_t root;  // this lane's

  __device__ __forceinline__ Weigher(const Scale& k_, const uint32_t* roots_) : k(k_), roots(roots_), root(roots_[threadIdx.x & 31]) {}

  // Of two logits; by all lanes of the warp together (the roots come from the lanes), or by some (kApart).  Logits are not below
  // k.least, but in FAR and apart, where it is seen to here (NaN, too).
  template <bool kApart>
  __device__ __forceinline__ void pair(float x0, float x1, Weight (&w)[2]) const {
    using tc::f2;
    using tc::fma2;
    const uint64_t ch = f2(k.ch, k.ch), cl = f2(k.cl, k.cl), base = f2(k.base, k.base);
    const bool some[2] = {!FAR || x0 >= k.least, !FAR || x1 >= k.least};
    if (FAR || kApart) {
      x0 = fmaxf(x0, k.least);
      x1 = fmaxf(x1, k.least);
    }
    uint64_t x = f2(x0, x1), low;
    if (FAR) {
      const float v[2] = {fminf(x0, kLargest), fminf(x1, kLargest)};
      float d[2], e[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        d[i] = __fsub_rn(v[i], k.m);
        const float t = __fsub_rn(d[i], v[i]);
        e[i] = __fadd_rn(__fsub_rn(v[i], __fsub_rn(d[i], t)), -__fadd_rn(k.m, t));
      }
      x = f2(d[0], d[1]);
      low = fma2(f2(e[0], e[1]), ch, tc::mul2(x, cl));
    }
    const uint64_t y = fma2(x, ch, base);  // kMagic + k / 32
    uint64_t g = fma2(x, ch, tc::sub2(base, y));
    g = FAR ? tc::add2(g, low) : fma2(x, cl, g);
    // 2^g - 1, times 2^32: ln(2)^n / n!
    constexpr float k32 = 4294967296.f, c1 = 0.693147181f * k32, c2 = 0.240226507f * k32, c3 = 0.0555041087f * k32,
                    c4 = 0.00961812911f * k32;
    uint64_t q = fma2(g, f2(c4, c4), f2(c3, c3));
    q = fma2(g, q, f2(c2, c2));
    q = fma2(g, q, f2(c1, c1));
    q = tc::mul2(g, q);
    float ys[2], qs[2];
    tc::unf2(y, ys[0], ys[1]);
    tc::unf2(q, qs[0], qs[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int bits = __float_as_int(ys[i]);
      const int r = kApart ? int(roots[bits & 31]) : int(__shfl_sync(0xffffffffu, root, bits));  // the lane is a number mod 32
      w[i].w = uint32_t(r + __mulhi(r, __float2int_rn(qs[i])));
      w[i].by = (k.s0 - bits) >> 5;
      if (FAR && !some[i]) w[i].by = 64;  // where `least` may be the maximum itself
    }
  }
  // what logits are raised to before they are weighed together (FAR: nothing, pair sees to it)
  template <class P>
  __device__ __forceinline__ uint32_t floor_of() const {
    return FAR ? P::kNone : P::floor_of(k.least);
  }
  __device__ __forceinline__ uint64_t operator()(float x) const {
    Weight w[2];
    pair<true>(x, x, w);
    return w[0].value();
  }
};

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }
__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += shfl_xor64(v, o);
  return v;
}

__device__ __forceinline__ void st_cluster_u64(uint32_t at, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t at) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t add_cluster_u32(uint32_t at, uint32_t v) {
  uint32_t r;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(r) : "r"(at), "r"(v) : "memory");
  return r;
}

struct Shared {
  uint64_t sums[kBins];    // weights of each bin: the sums of their lower 16 bits and of the others, 32 bits each, or one sum
  uint32_t counts[kBins];  // tokens of each bin
  uint64_t few[kFew];      // the last tokens of a search, in the cluster's first CTA
  uint64_t few_w[kFew];
  uint64_t totals[kMostCtas];
  uint64_t part[kMostParts], whole[kMostParts], listed_w[kMostParts];
  uint64_t warp_v[kWarps];
  uint64_t found_above, cut;
  uint32_t found_bin, found_count, few_n, here_n, here_at;
  uint32_t roots[32];
  uint32_t listed[kMostParts];       // candidates of each part; more than kList: they did not fit
  float tops[kMostCtas], kth[kMostCtas];
  float warp_top[kWarps];
  uint32_t warp_n[2][kWarps];
  Scale scale;
  float list_x[kWarps][kList];       // a part's candidates in order
  uint16_t list_i[kWarps][kList];    // and their places in it
};
static_assert(sizeof(Shared) <= 48 * 1024, "static shared memory");

// The place of a CTA in its row's cluster.
struct Place {
  int ctas, rank;
  __device__ __forceinline__ int parts() const { return ctas * kWarps; }
  __device__ __forceinline__ int part() const { return rank * kWarps + (threadIdx.x >> 5); }
};

template <class T>
struct Piece;  // 16 bytes of logits
template <>
struct Piece<float> {
  static constexpr int N = 4;
  static constexpr uint32_t kNone = 0xff800000u;  // -inf
  static __device__ __forceinline__ float at(const uint4& v, int i) { return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w); }
  static __device__ __forceinline__ float top(const uint4& v) {
    return fmaxf(fmaxf(at(v, 0), at(v, 1)), fmaxf(at(v, 2), at(v, 3)));
  }
  // no element below `least`, and no NaN (bf16: the next value down)
  static __device__ __forceinline__ uint32_t floor_of(float least) { return __float_as_uint(least); }
  static __device__ __forceinline__ uint4 raised(const uint4& v, uint32_t least) {
    auto up = [least](uint32_t x) { return __float_as_uint(fmaxf(__uint_as_float(x), __uint_as_float(least))); };
    return make_uint4(up(v.x), up(v.y), up(v.z), up(v.w));
  }
};
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr uint32_t kNone = 0xff80ff80u;
  static __device__ __forceinline__ float at(const uint4& v, int i) {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float top(const uint4& v) {
    const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t floor_of(float least) {
    return uint32_t(__bfloat16_as_ushort(__float2bfloat16_rd(least))) * 0x10001u;
  }
  static __device__ __forceinline__ uint4 raised(const uint4& v, uint32_t least) {
    return make_uint4(max2(v.x, least), max2(v.y, least), max2(v.z, least), max2(v.w, least));
  }
};

// A row's tokens, as this warp reads them: a contiguous part of the row in whole
// 16-byte pieces of memory, wherever the row begins.  Pieces that pass an end of the row are read element by element.
template <class T>
struct Row {
  using P = Piece<T>;
  static constexpr int N = P::N;
  const T* x;
  int vocab, skew;  // skew: elements by which the row begins behind a 16-byte border
  int pieces, per;  // 16-byte pieces that the row touches, and of a part

  __device__ __forceinline__ Row(const T* x_, int vocab_, int parts) : x(x_), vocab(vocab_) {
    skew = int((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    pieces = int((int64_t(vocab) + skew + N - 1) / N);
    per = (pieces + parts - 1) / parts;
  }
  // first element of a part
  __device__ __forceinline__ int begin(int part) const {
    const int64_t i = int64_t(part) * per * N - skew;
    return int(i < 0 ? 0 : i < vocab ? i : vocab);
  }
  // a piece; -inf outside of the row
  __device__ __forceinline__ uint4 piece(int j) const {
    const int i = j * N - skew;
    if (i >= 0 && i <= vocab - N) return __ldg(reinterpret_cast<const uint4*>(x + i));
    uint4 v = make_uint4(P::kNone, P::kNone, P::kNone, P::kNone);
    T* e = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int t = 0; t < N; ++t)
      if (i + t >= 0 && i + t < vocab) e[t] = x[i + t];
    return v;
  }
  // f(piece, index of its first element, which may be below 0) by all lanes together, in the order of the row; -inf outside of it
  template <int kU, class F>
  __device__ __forceinline__ void pieces_of(int part, int lane, F f) const {
    const uint4 none = make_uint4(P::kNone, P::kNone, P::kNone, P::kNone);
    const int a = int(min(int64_t(part) * per, int64_t(pieces))), b = min(a + per, pieces);
    const bool first = a < b && a == 0 && skew, last = a < b && b == pieces && (vocab + skew) % N && !(first && b == 1);
    auto end = [&](int j) { f(lane == 0 ? piece(j) : none, lane == 0 ? j * N - skew : 0); };
    if (first) end(a);
    const int whole = b - last;
    const uint4* from = reinterpret_cast<const uint4*>(x - skew);
    for (int base = a + first + lane; base - lane < whole; base += 32 * kU) {
      uint4 v[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) v[u] = base + 32 * u < whole ? __ldg(from + base + 32 * u) : none;
#pragma unroll
      for (int u = 0; u < kU; ++u) f(v[u], (base + 32 * u) * N - skew);
    }
    if (last) end(b - 1);
  }
  // elements of a CTA's parts, at most
  __device__ __forceinline__ int64_t most(const Place&) const { return int64_t(per) * N * kWarps; }
  // f(logit, index), by lanes apart, of the logits in [lo, hi] (finite ones), as they are compared: few of a row.
  template <class F>
  __device__ __forceinline__ void some(int part, int lane, float lo, float hi, F f) const {
    pieces_of<4>(part, lane, [&](const uint4& v, int i) {
      if (!__any_sync(0xffffffffu, P::top(v) >= lo)) return;
      uint32_t which = 0;
#pragma unroll
      for (int t = 0; t < N; ++t) which |= uint32_t(P::at(v, t) >= lo && fminf(P::at(v, t), kLargest) <= hi) << t;
      while (which) {
        const int t = __ffs(which) - 1;
        which &= which - 1;
        f(clean(P::at(v, t)), i + t);
      }
    });
  }
  // f(logit, index, weight, whether it is in) of all logits from lo on, without branches: a warp by itself takes five cycles for an
  // instruction that waits for the one before.
  template <bool kWeigh, class W, class F>
  __device__ __forceinline__ void all(int part, int lane, const W& weigh, float lo, F f) const {
    const uint32_t least = weigh.template floor_of<P>();
    pieces_of<2>(part, lane, [&](const uint4& v, int i) {
      if (!__any_sync(0xffffffffu, P::top(v) >= lo)) return;
      const uint4 r = kWeigh ? P::raised(v, least) : v;
#pragma unroll
      for (int t = 0; t < N; t += 2) {
        Weight w[2];
        if (kWeigh) weigh.template pair<false>(P::at(r, t), P::at(r, t + 1), w);
#pragma unroll
        for (int u = 0; u < 2; ++u) f(fminf(P::at(v, t + u), kLargest) + 0.f, i + t + u, w[u], P::at(v, t + u) >= lo);
      }
    });
  }
};

// The same of the candidates: a warp's list stands for its part of the row.
struct List {
  const Shared& sh;
  int begin, n;  // first element of the part, candidates
  template <class F>
  __device__ __forceinline__ void some(int, int lane, float lo, float hi, F f) const {
    const int warp = threadIdx.x >> 5;
    for (int i = lane; i < n; i += 32) {
      const float x = sh.list_x[warp][i];
      if (x >= lo && x <= hi) f(x, begin + sh.list_i[warp][i]);
    }
  }
  template <bool kWeigh, class W, class F>
  __device__ __forceinline__ void all(int, int lane, const W& weigh, float lo, F f) const {
    const int warp = threadIdx.x >> 5;
#pragma unroll 2
    for (int i = lane; i < n; i += 32) {
      const float x = sh.list_x[warp][i];
      Weight w[2];
      if (kWeigh) weigh.template pair<true>(x, x, w);
      f(x, begin + sh.list_i[warp][i], w[0], x >= lo);
    }
  }
  __device__ __forceinline__ int64_t most(const Place&) const { return kWarps * kList; }
};

// The sum of a part's weights (a lane's share): of the tokens from `from` on that weigh `least` or more.  Loops over a row stand in
// functions of their own, which have the registers to themselves.
template <class T, class W>
__device__ __forceinline__ uint64_t sum_piece(const W& weigh, const uint4& v, uint64_t sum) {
#pragma unroll
  for (int t = 0; t < Piece<T>::N; t += 2) {
    Weight w[2];
    weigh.template pair<false>(Piece<T>::at(v, t), Piece<T>::at(v, t + 1), w);
    sum += w[0].value();
    sum += w[1].value();
  }
  return sum;
}
template <bool FAR, class T>
__device__ __noinline__ uint64_t sum_of(const Row<T> row, int part, const Shared& sh) {
  const Weigher<FAR> weigh(sh.scale, sh.roots);
  const uint32_t least = weigh.template floor_of<Piece<T>>();
  uint64_t sum = 0;
  row.template pieces_of<2>(part, threadIdx.x & 31, [&](const uint4& v, int) { sum = sum_piece<T>(weigh, Piece<T>::raised(v, least), sum); });
  return sum;
}
template <bool FAR, class T>
__device__ __noinline__ uint64_t sum_of(const Row<T> row, int part, uint64_t from, uint64_t least, const Shared& sh) {
  using P = Piece<T>;
  const Weigher<FAR> weigh(sh.scale, sh.roots);
  const uint32_t floor = weigh.template floor_of<P>();
  uint64_t sum = 0;
  const int bits = 32 - weigh.k.shift;
  const float last = from ? logit_of(from, bits) : -INFINITY;  // of its equals, those up to an index
  const int last_i = from ? index_of(from, bits) : 0x7fffffff;
  row.template pieces_of<2>(part, threadIdx.x & 31, [&](const uint4& v, int i) {
    if (!__any_sync(0xffffffffu, P::top(v) >= last)) return;
    const uint4 r = P::raised(v, floor);
#pragma unroll
    for (int t = 0; t < Row<T>::N; t += 2) {
      Weight w[2];
      weigh.template pair<false>(P::at(r, t), P::at(r, t + 1), w);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float e = P::at(v, t + u), x = e > kLargest ? kLargest : e;  // (a NaN stays one, and fails)
        const bool kept = x > last || (x == last && i + t + u <= last_i);
        const uint64_t a = w[u].value();
        sum += kept && a >= least ? a : 0;
      }
    }
  });
  return sum;
}
template <bool FAR, class T>
__device__ __forceinline__ uint64_t sum_of(const Row<T>& row, const Row<T>&, int part, uint64_t from, uint64_t least, const Shared& sh) {
  return from == 0 && least == 0 ? sum_of<FAR>(row, part, sh) : sum_of<FAR>(row, part, from, least, sh);
}
template <bool FAR, class T>
__device__ __forceinline__ uint64_t sum_of(const Row<T>&, const List& list, int part, uint64_t from, uint64_t least, const Shared& sh) {
  const Weigher<FAR> weigh(sh.scale, sh.roots);
  uint64_t sum = 0;
  list.all<true>(part, threadIdx.x & 31, weigh, -kLargest, [&](float x, int i, const Weight& w, bool) {
    const uint64_t v = w.value();
    sum += number_of(x, i, 32 - weigh.k.shift) >= from && v >= least ? v : 0;
  });
  return sum;
}

// What a search looks for at a level.
struct Search {
  uint64_t lo, hi;    // numbers that take part
  float lo_x, hi_x;   // their logits
  int level, chosen;  // the first level's bin
  int shift;          // of a number's distance from hi, to its bin, from the second level on
  float steps;        // bins of the first level in a distance of 1
  bool by_weight, halves;
  int bits;           // of an index, in a number
  __device__ __forceinline__ int bin0(float m, float x) const { return min(int(__fmul_rn(__fsub_rn(m, x), steps)), kBins - 1); }
  // bits of a weight that are left out in a bin
  static __device__ __forceinline__ int bits_off(int shift, int bin) { return max(shift - bin / kBinsPerBit, 0); }
  __device__ __forceinline__ float value(uint64_t n) const {  // the logit of a number, within those that there are
    return of_key(min(max(uint32_t(n >> bits), key_of(-kLargest)), key_of(kLargest)));
  }
  // whether a token whose logit is in [lo_x, hi_x] takes part
  __device__ __forceinline__ bool has(float x, int i) const {
    return !((x == lo_x && number_of(x, i, bits) < lo) || (x == hi_x && number_of(x, i, bits) > hi));
  }
};

// Into a bin: a token, and of a weight the bits that are not left out.
template <bool kHalves>
__device__ __forceinline__ void add_to(Shared& sh, int bin, bool ok, const Weight& w, int b0, const Search& q, int shift) {
  if (ok) atomicAdd(&sh.counts[bin], 1u);
  if (!q.by_weight) return;
  if (kHalves) {  // (by - (32 - shift) bits are off the weight: as many as the bin leaves out, or one more)
    const uint32_t v = w.w >> min(max(w.by - 32 + shift - min(b0 / kBinsPerBit, shift), 0), 31);
    uint32_t* sums = reinterpret_cast<uint32_t*>(&sh.sums[bin]);
    if (ok) atomicAdd(sums, v & 0xffffu);
    if (ok) atomicAdd(sums + 1, v >> 16);
  } else if (ok) {
    atomicAdd(reinterpret_cast<unsigned long long*>(&sh.sums[bin]), static_cast<unsigned long long>(w.value() >> q.bits_off(shift, b0)));
  }
}

// This warp's tokens into the CTA's histogram: all from q.lo on at the first level (kWeigh: with their weights), then those of the bin.
template <bool FAR, bool kWeigh, bool kHalves, class Source>
__device__ __noinline__ void count_first(const Source src, int part, const Search q, Shared& sh) {
  const Weigher<FAR> weigh(sh.scale, sh.roots);
  const int last_i = index_of(q.lo, q.bits), shift = weigh.k.shift;
  const float m = weigh.k.m;
  src.template all<kWeigh>(part, threadIdx.x & 31, weigh, q.lo_x, [&](float x, int i, const Weight& w, bool ok) {
    // (q.lo as a number has no token below it among those of its logit where it is a bound's: its lower half is 0)
    const bool in = ok && (x > q.lo_x || uint32_t(i) <= uint32_t(last_i));
    const int b = q.bin0(m, x);
    add_to<kHalves>(sh, in ? b : 0, in, w, b, q, shift);
  });
}
template <bool FAR, bool kHalves, class Source>
__device__ __noinline__ void count_more(const Source src, int part, const Search q, Shared& sh) {
  const Weigher<FAR> weigh(sh.scale, sh.roots);
  src.some(part, threadIdx.x & 31, q.lo_x, q.hi_x, [&](float x, int i) {
    if (!q.has(x, i) || q.bin0(weigh.k.m, x) != q.chosen) return;
    Weight w[2];
    if (q.by_weight) weigh.template pair<true>(x, x, w);
    add_to<kHalves>(sh, int((q.hi - number_of(x, i, q.bits)) >> q.shift), true, w[0], q.chosen, q, weigh.k.shift);
  });
}

// The last tokens of a search, to the first CTA: first brought together here, since an addition in another CTA takes 2000 cycles.
template <bool FAR, class Source>
__device__ __noinline__ void gather(const Source src, int part, const Search q, Shared& sh) {
  const float m = sh.scale.m;
  src.some(part, threadIdx.x & 31, q.lo_x, q.hi_x, [&](float x, int i) {
    if (!q.has(x, i) || q.bin0(m, x) != q.chosen) return;
    const uint32_t at = atomicAdd(&sh.here_n, 1u);
    if (at < kFew) sh.few_w[at] = number_of(x, i, q.bits);
  });
  __syncthreads();
  const uint32_t n = min(sh.here_n, uint32_t(kFew));
  if (threadIdx.x == 0 && n) sh.here_at = add_cluster_u32(tc::peer_addr(&sh.few_n, 0), n);
  __syncthreads();
  if (threadIdx.x < n && sh.here_at + threadIdx.x < kFew)
    st_cluster_u64(tc::peer_addr(&sh.few[sh.here_at + threadIdx.x], 0), sh.few_w[threadIdx.x]);
}

// Sum over the CTA.
__device__ __forceinline__ uint64_t cta_sum64(uint64_t v, Shared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_sum64(v);
  __syncthreads();
  if (lane == 0) sh.warp_v[warp] = v;
  __syncthreads();
  uint64_t t = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) t += sh.warp_v[w];
  return t;
}
// Running sum over the CTA, without the thread's own.
__device__ __forceinline__ uint64_t cta_scan64(uint64_t v, Shared& sh, uint64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  __syncthreads();
  if (lane == 31) sh.warp_v[warp] = incl;
  __syncthreads();
  uint64_t before = incl - v;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sh.warp_v[w];
    total += sh.warp_v[w];
  }
  return before;
}

// v f, f in [0, 1], rounded down or up: exactly, in whole numbers.  (fp64 has so few units here that an operation of a warp takes
// 16 cycles; with this and the like in fp64, 64 rows took a third longer.)
template <bool kUp>
__device__ __forceinline__ uint64_t times(uint64_t v, float f) {
  const uint32_t bits = __float_as_uint(f), exponent = bits >> 23;
  const uint64_t m = exponent ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
  const int e = 150 - int(exponent ? exponent : 1);  // f = m 2^-e, e >= 23
  const uint64_t lo = v * m, hi = __umul64hi(v, m);
  uint64_t r = 0, rest = lo | hi;
  if (e < 64) {
    r = lo >> e | hi << (64 - e);
    rest = lo << (64 - e);
  } else if (e < 128) {
    r = e == 64 ? hi : hi >> (e - 64);
    rest = lo | (e == 64 ? 0 : hi << (128 - e));
  }
  return r + (kUp && rest != 0);
}

// What is asked of top_p: the sum that the run from the first on has to reach.
__device__ __forceinline__ uint64_t target_of(float p, uint64_t whole) {
  const uint64_t t = times<true>(whole, p);
  return t ? t : 1;
}
// The draw is of the token at which the running sum passes this (the last one for u >= 1).
__device__ __forceinline__ uint64_t limit_of(float u, uint64_t all) {
  return u > 0.f ? min(times<false>(all, fminf(u, 1.f)), all - 1) : 0;
}

// The cut of top-k or top-p: the number of the last token kept.  With by_weight, the last
// is the first at which the sum of the weights from the highest on reaches p of `whole` (0: of all that take part); otherwise the
// count-th.  Only tokens from `from` on take part.
template <bool FAR, class Source>
__device__ __noinline__ uint64_t find_cut(const Source src, bool by_weight, uint64_t count, float p, uint64_t whole, uint64_t from,
                                          const Place place, Shared& sh) {
  const Weigher<FAR> weigh(sh.scale, sh.roots);
  const int part = place.part();
  const float m = weigh.k.m, steps = float(kBinsPerBit) * weigh.k.ch;
  // A search leaves out the bits of a weight below 2^-30 of the largest that its bin can hold, 31 are left, and a sum of 65536
  // of them fits in two halves of 32 bits (the hardware adds to no 64-bit number in shared memory but in a loop of
  // compare and swap, far slower where many meet in a bin).
  const int ib = 32 - weigh.k.shift;
  Search q{from, ((uint64_t(key_of(kLargest)) + 1) << ib) - 1, 0.f, 0.f, 0, -1, 0, steps, by_weight, src.most(place) <= 65536, ib};
  uint64_t &lo = q.lo, &hi = q.hi, above = 0, target = count;
  int &chosen = q.chosen, &shift = q.shift;
  for (int level = 0;; ++level) {
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
      sh.counts[i] = 0;
      sh.sums[i] = 0;
    }
    __syncthreads();  // (and the level before is read)
    if (threadIdx.x == 0) {
      sh.few_n = sh.here_n = 0;
      sh.found_bin = kBins;
      sh.cut = from;
    }
    q.level = level;
    q.lo_x = q.value(lo);
    q.hi_x = q.value(hi);
    if (level > 0) {
      if (q.halves) count_more<FAR, true>(src, part, q, sh);
      else count_more<FAR, false>(src, part, q, sh);
    } else if (by_weight) {
      if (q.halves) count_first<FAR, true, true>(src, part, q, sh);
      else count_first<FAR, true, false>(src, part, q, sh);
    } else {
      count_first<FAR, false, true>(src, part, q, sh);
    }
    tc::cluster_sync();  // the histograms are there
    // each CTA adds up a share of the bins, a run of them a thread
    const int each = kBins / place.ctas, run = (each + kThreads - 1) / kThreads;
    const int first = place.rank * each + int(threadIdx.x) * run;
    const bool mine = int(threadIdx.x) * run < each;
    uint64_t v[kBinsEach], sum = 0;
    uint32_t tokens[kBinsEach];
#pragma unroll
    for (int j = 0; j < kBinsEach; ++j) {
      v[j] = 0;
      tokens[j] = 0;
      if (mine && j < run && place.ctas == 1) {
        tokens[j] = sh.counts[first + j];
        const uint64_t t = sh.sums[first + j];
        if (by_weight) v[j] = q.halves ? ((t >> 32) << 16) + uint32_t(t) : t;
      } else if (mine && j < run) {
        uint32_t n[kMostCtas];  // under way together (of CTAs that are not there, this one's, which do not count)
        uint64_t t[kMostCtas];
#pragma unroll
        for (int c = 0; c < kMostCtas; ++c) {
          const int from_cta = c < place.ctas ? c : place.rank;
          n[c] = ld_cluster_u32(tc::peer_addr(&sh.counts[first + j], from_cta));
          t[c] = ld_cluster_u64(tc::peer_addr(&sh.sums[first + j], from_cta));
        }
#pragma unroll
        for (int c = 0; c < kMostCtas; ++c) {
          tokens[j] += c < place.ctas ? n[c] : 0;
          v[j] += c < place.ctas ? (q.halves ? ((t[c] >> 32) << 16) + uint32_t(t[c]) : t[c]) : 0;
        }
      }
      if (by_weight) v[j] <<= q.bits_off(weigh.k.shift, level > 0 ? chosen : first + j);
      else v[j] = tokens[j];
      sum += v[j];
    }
    uint64_t total;
    const uint64_t here = cta_scan64(sum, sh, total);
    if (int(threadIdx.x) < place.ctas) st_cluster_u64(tc::peer_addr(&sh.totals[place.rank], threadIdx.x), total);
    tc::cluster_sync();
    uint64_t before = above, all = 0;
    for (int c = 0; c < place.ctas; ++c) {
      if (c < place.rank) before += sh.totals[c];
      all += sh.totals[c];
    }
    if (level == 0) {
      if (by_weight) target = target_of(p, whole ? whole : all);
      if (target > all) target = all;  // (fewer tokens than k have a finite logit; min_p has left less than top_p would)
    }
    // the thread that has it finds the first bin at which the running sum reaches the target
    uint64_t at = before + here;
#pragma unroll
    for (int j = 0; j < kBinsEach; ++j) {
      if (target > at && target <= at + v[j]) {
        for (int c = 0; c < place.ctas; ++c) {
          tc::st_cluster_u32(tc::peer_addr(&sh.found_bin, c), first + j);
          tc::st_cluster_u32(tc::peer_addr(&sh.found_count, c), tokens[j]);
          st_cluster_u64(tc::peer_addr(&sh.found_above, c), at);
        }
      }
      at += v[j];
    }
    tc::cluster_sync();
    const int b = int(sh.found_bin);
    if (b == kBins || level > kMostLevels) {  // not reached: a bin holds the target, and a level takes 10 of 64 bits
      if (threadIdx.x == 0) atomicOr(&g_status_sample, TPA_DEV_BAD_INPUT);
      return from;
    }
    const uint32_t left = sh.found_count;
    above = sh.found_above;
    if (level == 0) {
      chosen = b;
      // the numbers that the bin can hold: its logits, and the roundings of their distances
      const float far = float(b + 1) / steps, near = float(b) / steps;
      const float slack = 1e-6f * (fabsf(m) + far) + 1e-37f;
      const uint64_t low = uint64_t(key_of(clean(m - far - slack))) << q.bits;
      const uint64_t high = ((uint64_t(key_of(clean(m - near + slack))) + 1) << q.bits) - 1;
      if (b < kBins - 1 && low > lo) lo = low;
      if (high < hi) hi = high;
    } else {
      const uint64_t top = hi - (uint64_t(b) << shift);
      const uint64_t size = uint64_t(1) << shift;
      hi = top;
      if (top - lo >= size) lo = top - size + 1;
    }
    if (left <= kFew) break;
    const int bits = 64 - __clzll(static_cast<long long>(hi - lo));
    shift = bits > 10 ? bits - 10 : 0;
  }
  q.lo_x = q.value(lo);
  q.hi_x = q.value(hi);
  gather<FAR>(src, part, q, sh);
  tc::cluster_sync();
  if (place.rank == 0) {
    const int n = min(int(sh.few_n), kFew), me = threadIdx.x;
    uint64_t mine = 0, w = 0, before = above;
    if (me < n) {
      mine = sh.few[me];
      const int off = q.bits_off(weigh.k.shift, chosen);
      w = by_weight ? weigh(logit_of(mine, q.bits)) >> off << off : 1;
      sh.few_w[me] = w;
    }
    __syncthreads();
    if (me < n) {
#pragma unroll 8
      for (int j = 0; j < n; ++j) {
        const uint64_t v = sh.few_w[j];
        before += sh.few[j] > mine ? v : 0;
      }
      if (before < target && before + w >= target)
        for (int c = 0; c < place.ctas; ++c) st_cluster_u64(tc::peer_addr(&sh.cut, c), mine);
    }
  }
  tc::cluster_sync();
  return sh.cut;
}

// Where a row's results go.
struct Result {
  int32_t* token;
  float* logp;
};

struct Request {
  float t, top_p, min_p;
  int top_k;
  float u;
};

// The token, whose logit is x, and the logarithm of its weight w 2^-down over `all`.
template <bool FAR>
__device__ __forceinline__ void write_token(const Result& out, const Scale& k, float x_, int token, uint64_t w, int down, uint64_t all) {
  *out.token = token;
  // A weight of few bits is off by the part of a unit that was cut off: of those, 2^(30 + shift + y), the logarithm is taken by y
  // itself (u next to 0 draws such a token).
  if (w < (1 << 25)) {
    const float y = FAR ? __fsub_rn(x_, k.m) * k.ch : fmaf(x_, k.ch, k.base - kMagic) + x_ * k.cl;
    *out.logp = (float(30 + k.shift - down) + y) * 0.693147181f - logf(float(all));
    return;
  }
  // The quotient's logarithm, with what its roundings lost added; next to 1 from what is missing, so that little is lost where one
  // token has nearly all the weight.
  const uint64_t part = down < 64 ? w >> down : 0;
  const bool most = part > all - part;
  const uint64_t num = most ? all - part : w;
  const float a = float(num), b = float(all), x = a / b;
  const float off = (fmaf(-x, b, a) + float(int64_t(num - uint64_t(a))) - x * float(int64_t(all - uint64_t(b)))) / b;
  *out.logp = most ? log1pf(-(x + off)) : logf(x) + (off / x - float(down) * 0.693147181f);
}

// kFew candidates or fewer, in order in the first CTA's few (their numbers): a thread each.  `whole`: top_p is of it (0: of
// those that top_k leaves).
template <bool FAR>
__device__ __noinline__ void finish_few(const Result out, const Request q, int n, uint64_t whole, uint64_t least,
                                        Shared& sh) {
  const Weigher<FAR> weigh(sh.scale, sh.roots);
  const int me = threadIdx.x;
  uint64_t mine = 0, w = 0, before = 0;
  int rank = 0;
  if (me < n) {
    mine = sh.few[me];
    w = weigh(logit_of(mine, 32 - weigh.k.shift));
    sh.few_w[me] = w;
  }
  __syncthreads();
  const bool top_k = q.top_k > 0;
  if (me < n && (top_k || q.top_p < 1.f)) {
#pragma unroll 8
    for (int j = 0; j < n; ++j) {
      const uint64_t v = sh.few_w[j];
      const bool higher = sh.few[j] > mine;
      rank += higher;
      before += higher ? v : 0;
    }
  }
  bool kept = me < n && (!top_k || rank < q.top_k);
  if (q.top_p < 1.f) {
    if (whole == 0) whole = cta_sum64(kept ? w : 0, sh);
    kept = kept && before < target_of(q.top_p, whole);
  }
  kept = kept && w >= least;
  uint64_t all;
  const uint64_t at = cta_scan64(kept ? w : 0, sh, all);
  const uint64_t limit = limit_of(q.u, all);
  if (kept && at <= limit && at + w > limit) write_token<FAR>(out, weigh.k, logit_of(mine, 32 - weigh.k.shift), index_of(mine, 32 - weigh.k.shift), w, 0, all);
}

// The token of a part at which its running sum passes `limit`, among those from `from` on that weigh `least` or more; their weights are
// 2^down of those that `all` is made of.  By the CTA, a run of the part's entries a thread.
// Where the part was summed beside a moving maximum (sum_online), that sum holds parts of units that are cut off here: `limit` may pass what
// is there, by a unit a token, and then it is the last token with a weight (the part's largest has one: there always is one).
template <bool FAR, class T>
__device__ __noinline__ void find_in_part(const Result out, const Row<T> row, int part, uint64_t limit, uint64_t from,
                                          uint64_t least, int down, uint64_t all, Shared& sh) {
  const Weigher<FAR> weigh(sh.scale, sh.roots);
  const int i0 = row.begin(part), i1 = row.begin(part + 1), run = (i1 - i0 + kThreads - 1) / kThreads;
  const int a = min(i0 + int(threadIdx.x) * run, i1), b = min(a + run, i1);
  auto weight_of = [&](int i) -> uint64_t {
    const float x = clean(float(row.x[i]));
    const uint64_t w = weigh(x);
    return number_of(x, i, 32 - weigh.k.shift) >= from && w >= least ? w : 0;
  };
  uint64_t mine = 0;
#pragma unroll 4
  for (int i = a; i < b; ++i) mine += weight_of(i);
  uint64_t total;
  uint64_t at = cta_scan64(mine, sh, total);
  limit = min(limit, total - 1);
  if (at > limit || at + mine <= limit) return;
#pragma unroll 1
  for (int i = a; i < b; ++i) {
    const uint64_t w = weight_of(i);
    at += w;
    if (at > limit) {
      write_token<FAR>(out, weigh.k, clean(float(row.x[i])), i, w, down, all);
      return;
    }
  }
}

// Any number of tokens, of which those below `above` are not kept: the cuts, the sums of the parts, and the one in which the running sum passes u of the whole.
template <bool FAR, class T, class Source>
__device__ __noinline__ void finish_many(const Result out, const Request q, const Row<T> row, const Source src,
                                         uint64_t whole, float above, uint64_t least, const Place place, Shared& sh) {
  const Weigher<FAR> weigh(sh.scale, sh.roots);
  const int lane = threadIdx.x & 31, part = place.part();
  uint64_t from = above > -INFINITY ? uint64_t(key_of(above)) << (32 - weigh.k.shift) : 0;
  if (q.top_k > 0) from = find_cut<FAR>(src, false, uint64_t(q.top_k), 0.f, 0, from, place, sh);
  if (q.top_p < 1.f) from = find_cut<FAR>(src, true, 0, q.top_p, whole, from, place, sh);
  const uint64_t sum = warp_sum64(sum_of<FAR>(row, src, part, from, least, sh));
  if (lane < place.ctas) st_cluster_u64(tc::peer_addr(&sh.part[part], lane), sum);
  tc::cluster_sync();
  // two parts a lane, in every warp
  uint64_t v[2], incl = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[i] = 2 * lane + i < place.parts() ? sh.part[2 * lane + i] : 0;
    incl += v[i];
  }
  const uint64_t own = incl;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  const uint64_t all = __shfl_sync(0xffffffffu, incl, 31), limit = limit_of(q.u, all);
  if (all == 0) return;
  // the first lane whose sum passes the limit
  const int at_lane = __ffs(__ballot_sync(0xffffffffu, incl > limit)) - 1;
  const uint64_t first = incl - own;
  const bool second = first + v[0] <= limit;
  const int owner = __shfl_sync(0xffffffffu, 2 * lane + second, at_lane);
  const uint64_t before = __shfl_sync(0xffffffffu, first + (second ? v[0] : 0), at_lane);
  if (owner / kWarps == place.rank) find_in_part<FAR>(out, row, owner, limit - before, from, least, 0, all, sh);
}

// Rows without a cut, gone through once: each warp's weights are made for the largest logit that it has met, M a whole number of powers of 2
// above it, and its sum is moved down when a larger one comes: up to a unit of each token is cut off as it is added, and two of a lane's sum
// by all its moves (each leaves less than one, which the next ones halve at least).  (With the maximum found first, 64 rows
// of 151936 in bf16 took 22 us, now 18.)  A row of which a warp's first step is all masked by a large finite number (-1e9) counts as too far
// from 0 and goes the way of the rows with cuts: 64 rows with their first third at -1e9 take 31 us, at -inf 17.5.
struct Online {
  uint64_t sum;  // a lane's share
  int top;       // M; kNothing: no logit that can be drawn; kFar: too far from 0 for this
};
constexpr int kNothing = -(1 << 30), kFar = 1 << 30;
template <class T>
__device__ __noinline__ Online sum_online(const Row<T> row, int part, float ch, float cl, int shift, const Shared& sh) {
  using P = Piece<T>;
  Scale k = {};
  k.ch = ch;
  k.cl = cl;
  k.s0 = 32 * (32 - shift) + kMagicBits + 31;
  Weigher<false> weigh(k, sh.roots);
  float limit = -INFINITY;  // of the logits that M covers
  uint32_t least = 0;
  Online o{0, kNothing};
  row.template pieces_of<2>(part, threadIdx.x & 31, [&](const uint4& v, int) {
    const float top = P::top(v);
    if (__any_sync(0xffffffffu, top > limit)) {
      const float most = warp_max_f(top) * ch;
      if (!(fabsf(most) < 65000.f)) o.top = kFar;
      if (o.top == kFar) return;
      const int m = int(ceilf(most));  // 1/64 and more above the largest, or that much below at most: the 31 bits have room
      const int by = o.top == kNothing ? 0 : m - o.top;
      o.sum = by < 64 ? o.sum >> by : 0;
      o.top = m;
      limit = float(m) / ch;
      weigh.k.base = kMagic - float(m);
      least = P::floor_of((float(m) - float(31 + shift)) / ch);
    }
    if (o.top == kNothing || o.top == kFar) return;
    o.sum = sum_piece<T>(weigh, P::raised(v, least), o.sum);
  });
  return o;
}

// False where a part is too far from 0.
template <class T>
__device__ __forceinline__ bool draw_plain(const Result& out, const Request& q, const Row<T>& row, float ch, float cl, int shift,
                                           const Place& place, Shared& sh) {
  const int lane = threadIdx.x & 31, part = place.part();
  const Online o = sum_online(row, part, ch, cl, shift, sh);
  const uint64_t sum = warp_sum64(o.sum);
  cluster_wait();  // the other CTAs run: their shared memory may be written
  if (lane < place.ctas) {
    st_cluster_u64(tc::peer_addr(&sh.part[part], lane), sum);
    tc::st_cluster_u32(tc::peer_addr(&sh.listed[part], lane), uint32_t(o.top));
  }
  tc::cluster_sync();
  // two parts a lane, in every warp
  int top[2], m = kNothing;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    top[i] = 2 * lane + i < place.parts() ? int(sh.listed[2 * lane + i]) : kNothing;
    m = max(m, top[i]);
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, s));
  if (m == kFar) return false;
  if (m == kNothing) {
    if (place.rank == 0 && threadIdx.x == 0) {
      *out.token = -1;
      *out.logp = __int_as_float(0x7fc00000);
    }
    return true;
  }
  uint64_t v[2], own = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[i] = m - top[i] < 64 ? sh.part[min(2 * lane + i, kMostParts - 1)] >> (m - top[i]) : 0;
    own += v[i];
  }
  uint64_t incl = own;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const uint64_t t = __shfl_up_sync(0xffffffffu, incl, s);
    if (lane >= s) incl += t;
  }
  const uint64_t all = __shfl_sync(0xffffffffu, incl, 31), limit = limit_of(q.u, all);
  const int at_lane = __ffs(__ballot_sync(0xffffffffu, incl > limit)) - 1;
  const uint64_t first = incl - own;
  const bool second = first + v[0] <= limit;
  const int owner = __shfl_sync(0xffffffffu, 2 * lane + second, at_lane);
  const uint64_t rest = limit - __shfl_sync(0xffffffffu, first + (second ? v[0] : 0), at_lane);
  const int down = m - __shfl_sync(0xffffffffu, second ? top[1] : top[0], at_lane);
  if (owner / kWarps != place.rank) return true;
  // In the part's own numbers: floor(sum / 2^down) passes `rest` where the sum is (rest + 1) 2^down.
  if (threadIdx.x == 0) {
    const int own_top = m - down;
    Scale& k = sh.scale;
    k.m = 0.f;
    k.ch = ch;
    k.cl = cl;
    k.base = kMagic - float(own_top);
    k.least = (float(own_top) - float(31 + shift)) / ch;
    k.shift = shift;
    k.s0 = 32 * (32 - shift) + kMagicBits + 31;
  }
  __syncthreads();
  find_in_part<false>(out, row, owner, ((rest + 1) << down) - 1, 0, 0, down, all, sh);
  return true;
}

// A part's tokens from `bound` on, in order, into the warp's list; their number, and the sum of all weights of the part (a lane's share).
struct Collected {
  uint64_t sum;
  int n;  // more than kList: there was no room
};
template <bool FAR, bool kSums, class T>
__device__ __noinline__ Collected collect(const Row<T> row, int part, float bound, Shared& sh) {
  using P = Piece<T>;
  constexpr int N = P::N;
  const Weigher<FAR> weigh(sh.scale, sh.roots);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, begin = row.begin(part);
  const uint32_t least = weigh.template floor_of<P>();
  uint64_t sum = 0;
  int n = 0;
  row.template pieces_of<kSums ? 2 : 4>(part, lane, [&](const uint4& v, int i) {
    if (kSums) sum = sum_piece<T>(weigh, P::raised(v, least), sum);
    if (n > kList || !__any_sync(0xffffffffu, P::top(v) >= bound)) return;  // (more than there is room for)
    uint32_t which = 0;
#pragma unroll
    for (int t = 0; t < N; ++t) which |= uint32_t(P::at(v, t) >= bound) << t;
    // candidates of the lanes before, and of all
    const unsigned before = (1u << lane) - 1, lanes = __ballot_sync(0xffffffffu, which != 0);
    int at = n + __popc(lanes & before);
    n += __popc(lanes);
    if (__any_sync(0xffffffffu, which & (which - 1))) {  // more than one of a lane: the counts' higher parts, less one
      const int more = which ? __popc(which) - 1 : 0;
#pragma unroll
      for (int bit = 0; bit < 3; ++bit) {
        const unsigned m = __ballot_sync(0xffffffffu, more >> bit & 1);
        at += __popc(m & before) << bit;
        n += __popc(m) << bit;
      }
    }
    while (which) {
      const int t = __ffs(which) - 1;
      which &= which - 1;
      if (at < kList) {
        sh.list_x[warp][at] = clean(P::at(v, t));
        sh.list_i[warp][at] = uint16_t(i + t - begin);
      }
      ++at;
    }
  });
  return Collected{sum, n};
}

// From the maximum on.  With a cut, the tokens that may be kept are first collected: those from `bound` on, which may be a guess.
template <class T, bool FAR>
__device__ void draw(const Result& out, const Request& q, const Row<T>& row, float bound, bool guess, const Place& place,
                     Shared& sh) {
  constexpr int N = Piece<T>::N;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = place.part();
  const Weigher<FAR> weigh(sh.scale, sh.roots);
  const uint64_t least = q.min_p > 0.f ? times<true>(weigh(weigh.k.m), q.min_p) : 0;
  const bool of_all = q.top_p < 1.f && q.top_k <= 0;  // top_p of the whole row's weights
  if (bound == -INFINITY || row.per * N > 65536) {
    finish_many<FAR>(out, q, row, row, 0, -INFINITY, least, place, sh);
    return;
  }
  const int begin = row.begin(part);
  uint64_t whole = 0;
  for (int attempt = 0;; ++attempt) {
    const bool sums = of_all && whole == 0;
    const Collected got = sums ? collect<FAR, true>(row, part, bound, sh) : collect<FAR, false>(row, part, bound, sh);
    const int n = got.n;
    uint64_t sum = got.sum;
    __syncwarp();
    const List list{sh, begin, min(n, kList)};
    uint64_t in_list = 0;
    if (sums) {
      sum = warp_sum64(sum);
    }
    if (guess && attempt < 2) in_list = warp_sum64(sum_of<FAR>(row, list, part, 0, 0, sh));
    if (lane < place.ctas) {
      tc::st_cluster_u32(tc::peer_addr(&sh.listed[part], lane), uint32_t(n));
      st_cluster_u64(tc::peer_addr(&sh.whole[part], lane), sum);
      st_cluster_u64(tc::peer_addr(&sh.listed_w[part], lane), in_list);
    }
    tc::cluster_sync();
    // two parts a lane, in every warp
    int before = 0, all = 0;
    bool fits = true;
    uint64_t known = 0, listed = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int o = lane + 32 * i;
      if (o < place.parts()) {
        const int c = int(sh.listed[o]);
        fits &= c <= kList;
        all += min(c, kList);
        if (o < part) before += min(c, kList);
        known += sh.whole[o];
        listed += sh.listed_w[o];
      }
    }
    before = warp_sum(before);
    all = warp_sum(all);
    fits = __all_sync(0xffffffffu, fits);
    if (sums) whole = warp_sum64(known);
    // A guess holds when the candidates' weights reach top_p's target.  Tokens that each weigh less than (1 - top_p) / vocab of
    // the whole are less than 1 - top_p of it together: none has the cut, so the last attempt needs no luck.
    if (guess && attempt < 2 && warp_sum64(listed) < target_of(q.top_p, whole)) {
      const float share = 0.98f * float(whole) / float(uint64_t(1) << 30 << weigh.k.shift) * (1.f - q.top_p) / float(row.vocab);
      const float safe = weigh.k.m + q.t * logf(share) - 1e-5f * (fabsf(weigh.k.m) + 100.f * q.t);
      // (where the first guess misses more than 0.15 of the whole, the wider one hardly ever holds: without it 64 rows of 151936
      // at T = 1.3 with p = 0.97 take 112 us, not 127)
      const bool near = target_of(q.top_p, whole) - warp_sum64(listed) < times<false>(whole, 0.15f);
      const float next = attempt == 0 && fits && near ? fmaxf(weigh.k.m - kWider * q.t, safe) : safe;
      bound = next < bound ? next : safe;
      if (bound == safe) attempt = 1;
      // (with a quarter of the room used, a wider guess will hardly fit; nor will the last bound's, but in a short row)
      if (bound > -kLargest && fits && all <= place.parts() * (kList / 4) && (bound != safe || row.per * N <= 2 * kList)) {
        tc::cluster_sync();  // all have read what is written again
        continue;
      }
      bound = safe > -kLargest ? safe : -INFINITY;
      fits = false;
    }
    if (!fits) {
      finish_many<FAR>(out, q, row, row, whole, bound, least, place, sh);
    } else if (all > kFew) {
      finish_many<FAR>(out, q, row, list, whole, -INFINITY, least, place, sh);
    } else {
      for (int i = lane; i < list.n; i += 32)
        st_cluster_u64(tc::peer_addr(&sh.few[before + i], 0), number_of(sh.list_x[warp][i], begin + sh.list_i[warp][i], 32 - weigh.k.shift));
      tc::cluster_sync();
      if (place.rank == 0) finish_few<FAR>(out, q, all, whole, least, sh);
    }
    return;
  }
}

// log2(e) / T as a pair.
__device__ __forceinline__ float2 per_log(float t) {
  const float ch = __fdiv_rn(1.44269502f, t);
  return make_float2(ch, __fdiv_rn(__fmaf_rn(-ch, t, 1.44269502f) + 1.92596299e-8f, t));
}

// A row, from its parameters on; the cluster's CTAs have met (kMet), or arrived at their barrier.
template <class T, bool kMet>
__device__ __forceinline__ void draw_row(const Result& out, const Request& q, bool fine, const Row<T>& row, int shift,
                                         const Place& place, Shared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float2 c = per_log(q.t);
  const float ch = c.x, cl = c.y;
  // the maximum
  float own[kTops];  // of every kTops-th piece
#pragma unroll
  for (int i = 0; i < kTops; ++i) own[i] = -INFINITY;
  row.template pieces_of<4>(place.part(), lane, [&](const uint4& v, int) {
    const float t = fmaxf(own[0], Piece<T>::top(v));
#pragma unroll
    for (int i = 0; i < kTops - 1; ++i) own[i] = own[i + 1];
    own[kTops - 1] = t;
  });
  float most = own[0];
#pragma unroll
  for (int i = 1; i < kTops; ++i) most = fmaxf(most, own[i]);
  float top = warp_max_f(most);
  if (lane == 0) sh.warp_top[warp] = top;
  __syncthreads();
  top = sh.warp_top[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sh.warp_top[w]);
  // A logit that top_k does not leave out is at least the ceil(k / CTAs)-th largest of the threads' own maxima in the CTA where that
  // is lowest: k of the maxima are.  Bisection finds it to 2^-9 of itself, which is near enough for a bound.  Where k is not small beside
  // the threads, each one's eight maxima are taken apart, so that few tokens more than k pass the bound: 500 rows of 16000 with
  // k = 1000 76 -> 40 us, k = 300 91 -> 44, k = 200 33 -> 29.5; below that it costs 2 us and more a call (k = 100 20.8 -> 21.8, 20 14 -> 18).
  const int share = (q.top_k + place.ctas - 1) / place.ctas;
  float kth = -INFINITY;
  if (q.top_k > 0 && share <= kTops * kThreads) {
    const bool few = share <= kThreads / 2;
    const uint32_t mine = key_of(most);
    int turn = 0;
    auto at_least = [&](uint32_t key) -> int {  // maxima from a key on
      if (few) return __syncthreads_count(mine >= key);
      uint32_t n = 0;
#pragma unroll
      for (int i = 0; i < kTops; ++i) n += key_of(own[i]) >= key;
      n = __reduce_add_sync(0xffffffffu, n);
      turn ^= 1;
      if (lane == 0) sh.warp_n[turn][warp] = n;
      __syncthreads();
      n = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) n += sh.warp_n[turn][w];
      return int(n);
    };
    uint32_t lo = key_of(-kLargest), hi = key_of(top);  // lo: so many are at least that
    if (at_least(lo) >= share) {
      for (int i = 0; i < 18 && lo < hi; ++i) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        if (at_least(mid) >= share) lo = mid;
        else hi = mid - 1;
      }
      kth = of_key(lo);
    }
  }
  if (!kMet) cluster_wait();  // the other CTAs run: their shared memory may be written
  if (int(threadIdx.x) < place.ctas) {
    tc::st_cluster_u32(tc::peer_addr(&sh.tops[place.rank], threadIdx.x), __float_as_uint(top));
    tc::st_cluster_u32(tc::peer_addr(&sh.kth[place.rank], threadIdx.x), __float_as_uint(kth));
  }
  tc::cluster_sync();
  float low = INFINITY, bound = -INFINITY;
  for (int c = 0; c < place.ctas; ++c) {
    top = fmaxf(top, sh.tops[c]);
    low = fminf(low, sh.kth[c]);
  }
  if (q.top_k > 0) bound = fminf(low, kLargest);
  if (!fine || top == -INFINITY) {  // nothing to draw from, or no way to
    if (place.rank == 0 && threadIdx.x == 0) {
      if (!fine) atomicOr(&g_status_sample, TPA_DEV_BAD_INPUT);
      *out.token = -1;
      *out.logp = __int_as_float(0x7fc00000);
    }
    return;
  }
  top = fminf(top, kLargest);
  // (of the tokens that top_k leaves, top_p needs the weights of all)
  if (q.min_p > 0.f && !(q.top_k > 0 && q.top_p < 1.f)) bound = fmaxf(bound, top + q.t * logf(q.min_p) - 1e-5f * (fabsf(top) + 100.f * q.t));
  // top_p's cut is first looked for next to the maximum
  const bool guess = q.top_p < 1.f && q.top_k <= 0 && top - kHead * q.t > bound;
  if (guess) bound = top - kHead * q.t;
  const bool far = !(fabsf(top) * ch < 65536.f);
  if (threadIdx.x == 0) {
    const float near = far ? 0.f : __fsub_rn(__fmaf_rn(top, ch, kMagic), kMagic);
    Scale& k = sh.scale;
    k.m = top;
    k.ch = ch;
    k.cl = cl;
    k.base = kMagic - near;
    k.least = fmaxf(top - float(31 + shift) / ch, -kLargest);
    k.shift = shift;
    k.s0 = 32 * (32 - shift) + kMagicBits + 31;
  }
  __syncthreads();
  if (far) draw<T, true>(out, q, row, bound, guess, place, sh);
  else draw<T, false>(out, q, row, bound, guess, place, sh);
}

template <class T>
__global__ void __launch_bounds__(kThreads, 4) sample_kernel(const Params p) {
  __shared__ Shared sh;
  cluster_arrive();  // this CTA runs
  const Place place{p.ctas, int(tc::cta_rank())};
  const int64_t r = blockIdx.x / p.ctas;
  const Row<T> row(static_cast<const T*>(p.logits) + r * p.row_stride, p.vocab, place.parts());
  Request q;
  q.t = p.temperature ? __ldg(p.temperature + r) : p.temperature_all;
  q.top_p = p.top_p ? __ldg(p.top_p + r) : p.top_p_all;
  q.min_p = p.min_p ? __ldg(p.min_p + r) : p.min_p_all;
  q.top_k = p.top_k ? __ldg(p.top_k + r) : p.top_k_all;
  q.u = __ldg(p.u + r);
  const bool fine = (q.t == 0.f || (q.t >= 1e-6f && q.t <= 1e6f)) && q.top_p >= 0.f && q.top_p <= 1.f && q.min_p >= 0.f &&
                    q.min_p <= 1.f;
  if (q.t == 0.f) {  // the first of the largest
    q.t = 1.f;
    q.top_k = 1;
    q.top_p = 1.f;
  }
  if (q.top_k >= p.vocab) q.top_k = 0;
  if (threadIdx.x < 32) sh.roots[threadIdx.x] = kRoots[threadIdx.x];
  draw_row<T, false>(Result{p.tokens + r, p.logp + r}, q, fine, row, p.shift, place, sh);
}

// All rows without a cut, of one temperature.  (In the kernel above these rows' code costs the others 2 us.)
template <class T>
__device__ __noinline__ void draw_far(const Result out, const Request q, const Row<T> row, int shift, const Place place, Shared& sh) {
  draw_row<T, true>(out, q, true, row, shift, place, sh);
}
template <class T>
__global__ void __launch_bounds__(kThreads, 4) plain_kernel(const Params p) {
  __shared__ Shared sh;
  cluster_arrive();  // this CTA runs
  const Place place{p.ctas, int(tc::cta_rank())};
  const int64_t r = blockIdx.x / p.ctas;
  const Row<T> row(static_cast<const T*>(p.logits) + r * p.row_stride, p.vocab, place.parts());
  const Request q{p.temperature_all, 1.f, 0.f, 0, __ldg(p.u + r)};
  if (threadIdx.x < 32) sh.roots[threadIdx.x] = kRoots[threadIdx.x];
  __syncthreads();
  const float2 c = per_log(q.t);
  const Result out{p.tokens + r, p.logp + r};
  if (!draw_plain<T>(out, q, row, c.x, c.y, p.shift, place, sh)) draw_far(out, q, row, p.shift, place, sh);
}

template <class T>
int launch(Params& p, int n_rows, cudaStream_t st) {
  // CTAs of a row: as many as are at work together on the device (4 an SM), and not less than kLeast bytes for each.  64 rows of
  // 151936 with their own parameters take 42 us with 8, 59 with 4; 200 rows of 32000 13.2 with 2, 20.5 with 4; 499 rows
  // 45.1 with 1, 47.5 with 2; one row of 32000 9.0 with 8, 10.4 with 4.
  constexpr int kLeast = 8192;
  p.ctas = kMostCtas;
  while (p.ctas > 1 && (int64_t(n_rows) * p.ctas > 600 || int64_t(p.vocab) * int(sizeof(T)) < int64_t(kLeast) * p.ctas)) p.ctas /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(n_rows) * p.ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool plain = !p.temperature && !p.top_p && !p.min_p && !p.top_k && p.temperature_all > 0.f && p.top_p_all >= 1.f &&
                     p.min_p_all <= 0.f && (p.top_k_all <= 0 || p.top_k_all >= p.vocab);
  TPA_CUDA_TRY(cudaLaunchKernelEx(&cfg, plain ? plain_kernel<T> : sample_kernel<T>, static_cast<const Params>(p)));
  return TPA_OK;
}

}  // namespace

TPA_DEFINE_STATUS_READER(tpa_internal_status_sample, g_status_sample)

extern "C" int tpa_sample_tokens(const void* logits, int32_t logits_type, int64_t row_stride, int32_t n_rows, int32_t vocab,
                                 const tpa_sample_params* params, const float* u, int32_t* tokens, float* logp,
                                 void* stream) {
  TPA_NVTX_RANGE("tpa_sample_tokens");
  if (n_rows < 0 || n_rows > 0x7fffffff / kMostCtas || vocab < 1 || vocab > kMostVocab || !params ||
      (logits_type != TPA_LOGITS_F32 && logits_type != TPA_LOGITS_BF16))
    return TPA_ERR_INVALID_ARG;
  auto in = [](float v, float lo, float hi) { return v >= lo && v <= hi; };
  if ((!params->temperature && params->temperature_all != 0.f && !in(params->temperature_all, 1e-6f, 1e6f)) ||
      (!params->top_p && !in(params->top_p_all, 0.f, 1.f)) || (!params->min_p && !in(params->min_p_all, 0.f, 1.f)))
    return TPA_ERR_INVALID_ARG;
  if (n_rows == 0) return TPA_OK;
  if (!logits || !u || !tokens || !logp || row_stride < vocab || row_stride >= (int64_t(1) << 40)) return TPA_ERR_INVALID_ARG;
  const uintptr_t al = reinterpret_cast<uintptr_t>(u) | reinterpret_cast<uintptr_t>(tokens) | reinterpret_cast<uintptr_t>(logp) |
                       reinterpret_cast<uintptr_t>(params->temperature) | reinterpret_cast<uintptr_t>(params->top_p) |
                       reinterpret_cast<uintptr_t>(params->min_p) | reinterpret_cast<uintptr_t>(params->top_k);
  const bool f32 = logits_type == TPA_LOGITS_F32;
  if ((al & 3) || (reinterpret_cast<uintptr_t>(logits) & (f32 ? 3 : 1))) return TPA_ERR_INVALID_ARG;
  int bits = 0;
  while ((int64_t(1) << bits) < vocab) ++bits;
  Params p{logits, row_stride, params->temperature, params->top_p, params->min_p, params->top_k, u, tokens, logp,
                 params->temperature_all, params->top_p_all, params->min_p_all, params->top_k_all, vocab, 32 - bits, 1};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return f32 ? launch<float>(p, n_rows, st) : launch<__nv_bfloat16>(p, n_rows, st);
}
