// Verification of drafted tokens against the target's probabilities, with the
// next token drawn from what is left: one cluster of 8 CTAs a sequence.
//
// The acceptance run needs one entry of each row: every CTA forms it for
// itself (a warp, 32 drafts at a time).  It names the one row (or pair of
// rows) whose weights r(v) = max(p(v) - q(v), 0) are summed and searched:
// 4 bytes of p and 4 of q for each entry, read from HBM once, which bounds
// the kernel.  Each warp sums a contiguous 1/64 of the row; the 64 sums are
// exchanged through distributed shared memory; the part in which the
// running sum passes u * total is read again, by its whole CTA, to find the token.
//
// A draw has to be the same whatever the order of summation, so sums are held
// to far more than fp32: every weight and every sum is an unevaluated pair
// hi + lo of fp32, formed by error-free additions (Knuth's and Dekker's).  With
// u = 2^-24, an addition of two pairs is off by at most 3 u^2 of its result and
// one of a run of 8 weights to a lane's pair (Sum) by 12 u^2, so that a draw's
// sums are within 2^-41 + vocab 2^-56 of the row's (64 parts of 32 lanes with two pairs each;
// some 30 additions between them).  fp64 would do, but this GPU has so few of its units
// that the reductions alone took longer than the reads (part sums, prefix sums and the search in
// fp64: 42 us for 64 sequences at vocabulary 151936).
#include <cuda_runtime.h>

#include "device_common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace {

__device__ unsigned int g_status_verify = 0;

constexpr int kCluster = 8;
// Four CTAs of 256 threads an SM: with 512 the registers leave room for two, and 64 sequences take two rounds (25 us
// instead of 20 at vocabulary 151936).
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kParts = kCluster * kWarps;  // contiguous parts of a row, one a warp

struct Params {
  const float* target;
  const float* draft;
  const int32_t* draft_tokens;
  const int32_t* n_drafts;
  const float* u_accept;
  const float* u_next;
  int32_t* tokens;
  int32_t* n_accepted;
  int64_t target_stride, draft_stride;
  int32_t max_drafts, vocab;
};

// max(p - q, 0) as hi + lo, exactly; 0 where either is NaN
__device__ __forceinline__ void weight(float p, float q, float& hi, float& lo) {
  const float d = __fsub_rn(p, q), b = __fsub_rn(d, p);
  const float e = __fsub_rn(__fsub_rn(p, __fsub_rn(d, b)), __fadd_rn(q, b));
  const bool some = p > q;
  hi = some ? d : 0.f;
  lo = some ? e : 0.f;
}

// hi + lo, |lo| at most half a unit in the last place of hi
struct Pair {
  float hi = 0.f, lo = 0.f;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return Pair{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair normal(float a, float b) {  // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return Pair{s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Pair operator+(const Pair& a, const Pair& b) {
  const Pair s = two_sum(a.hi, b.hi);
  return normal(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ Pair operator*(const Pair& a, float u) {
  const float p = __fmul_rn(a.hi, u);
  return normal(p, __fmaf_rn(a.lo, u, __fmaf_rn(a.hi, u, -p)));
}
__device__ __forceinline__ bool operator>(const Pair& a, const Pair& b) {
  return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo);
}

// A running sum of weights.  The low halves are added up in plain fp32 and stay below 2 k + 1 units of u times the
// sum for k weights behind the last tidy(), whose roundings then are off by k^2 + 4 k units of u^2 of it: 96 for a run
// of 8.  Left to grow, they cost a row of 2^27 entries all but 2^-24.
struct Sum {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float p, float q) {
    float h, l;
    weight(p, q, h, l);
    const Pair s = two_sum(hi, h);
    hi = s.hi;
    lo = __fadd_rn(lo, __fadd_rn(s.lo, l));
  }
  __device__ __forceinline__ void tidy() {
    const Pair s = normal(hi, lo);
    hi = s.hi;
    lo = s.lo;
  }
  __device__ __forceinline__ Pair value() const { return Pair{hi, lo}; }
};

__device__ __forceinline__ Pair shfl_pair(const Pair& v, int from) {
  return Pair{__shfl_sync(0xffffffffu, v.hi, from), __shfl_sync(0xffffffffu, v.lo, from)};
}
__device__ __forceinline__ Pair warp_sum(Pair v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = v + Pair{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)};
  return v;
}
// The sum of the lanes before, and this one's added.
__device__ __forceinline__ void warp_scan(const Pair& v, int lane, Pair& before, Pair& incl) {
  incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair t{__shfl_up_sync(0xffffffffu, incl.hi, o), __shfl_up_sync(0xffffffffu, incl.lo, o)};
    if (lane >= o) incl = t + incl;
  }
  before = Pair{__shfl_up_sync(0xffffffffu, incl.hi, 1), __shfl_up_sync(0xffffffffu, incl.lo, 1)};
  if (lane == 0) before = Pair{};
}

// Where a row's weights come from: p, and what is taken off it.
struct Row {
  const float* p;
  const float* q;  // NULL: nothing, or all on `only`
  int32_t only;    // -1: none
};

// This warp's sum of the weights in [i0, i1), i0 a multiple of 4.  `only` is
// left out of the sum, not taken off it, so that nothing is lost where it has nearly all the weight.
__device__ __forceinline__ Pair part_sum(const Row& r, int i0, int i1, int lane) {
  Sum a, b;  // two chains
  const bool vec = ((reinterpret_cast<uintptr_t>(r.p) | reinterpret_cast<uintptr_t>(r.q)) & 15) == 0;
  if (vec) {
    constexpr int kU = 4;  // loads of 16 bytes a row on their way together
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int base = i0; base < i1; base += 128 * kU) {
      float4 p[kU], q[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int i = base + 128 * u + 4 * lane;
        p[u] = q[u] = none;
        if (i + 4 <= i1) {
          p[u] = __ldcs(reinterpret_cast<const float4*>(r.p + i));
          if (r.q) q[u] = __ldcs(reinterpret_cast<const float4*>(r.q + i));
        } else if (i < i1) {
          float* pf = reinterpret_cast<float*>(&p[u]);
          float* qf = reinterpret_cast<float*>(&q[u]);
#pragma unroll
          for (int t = 0; t < 3; ++t)
            if (i + t < i1) {
              pf[t] = __ldg(r.p + i + t);
              if (r.q) qf[t] = __ldg(r.q + i + t);
            }
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int i = base + 128 * u + 4 * lane;
        const int at = r.only - i;  // 0..3: one of this lane's four
        a.add(at == 0 ? 0.f : p[u].x, q[u].x);
        b.add(at == 1 ? 0.f : p[u].y, q[u].y);
        a.add(at == 2 ? 0.f : p[u].z, q[u].z);
        b.add(at == 3 ? 0.f : p[u].w, q[u].w);
      }
      a.tidy();
      b.tidy();
    }
  } else {
    constexpr int kU = 8;
    for (int base = i0 + lane; base < i1; base += 32 * kU) {
      float p[kU], q[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int i = base + 32 * u;
        p[u] = i < i1 && i != r.only ? __ldcs(r.p + i) : 0.f;
        q[u] = i < i1 && r.q ? __ldcs(r.q + i) : 0.f;
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) (u & 1 ? b : a).add(p[u], q[u]);
      a.tidy();
      b.tidy();
    }
  }
  return warp_sum(a.value() + b.value());
}

// The lowest v in [i0, i1) at which `before` plus the weights up to v pass
// `limit`; the last v with a weight where none does, -1 without any.  By the
// whole CTA, a run of entries a thread.
__device__ int part_find(const Row& r, int i0, int i1, const Pair& before, const Pair& limit, Pair* warp_s, int* found_s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int run = (i1 - i0 + kThreads - 1) / kThreads;
  const int64_t a0 = i0 + int64_t(threadIdx.x) * run;
  const int a = int(a0 < i1 ? a0 : i1), b = i1 - a < run ? i1 : a + run;
  auto weight_at = [&](int i) {
    Pair w;
    if (i != r.only) weight(__ldg(r.p + i), r.q ? __ldg(r.q + i) : 0.f, w.hi, w.lo);
    return w;
  };
  Pair mine;
  int last = -1;
#pragma unroll 4
  for (int i = a; i < b; ++i) {
    const Pair w = weight_at(i);
    mine = mine + w;
    if (w.hi > 0.f) last = i;
  }
  Pair lanes, incl;
  warp_scan(mine, lane, lanes, incl);
  if (lane == 31) warp_s[warp] = incl;
  if (threadIdx.x == 0) {
    found_s[0] = 0x7fffffff;
    found_s[1] = -1;
  }
  __syncthreads();
  Pair at = before;
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    if (w < warp) at = at + warp_s[w];
  at = at + lanes;
  if (last >= 0) atomicMax(found_s + 1, last);
  if (last >= 0 && at + mine > limit) {
    for (int i = a; i <= last; ++i) {
      const Pair w = weight_at(i);
      at = at + w;
      // (the last entry counts as passed: `at + mine`, rounded differently, passes the limit)
      if (w.hi > 0.f && (at > limit || i == last)) {
        atomicMin(found_s, i);
        break;
      }
    }
  }
  __syncthreads();
  return found_s[0] != 0x7fffffff ? found_s[0] : found_s[1];
}

__device__ __forceinline__ void st_cluster_pair(uint32_t addr, const Pair& v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(v.hi), "f"(v.lo) : "memory");
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 4) verify_kernel(const Params p) {
  __shared__ __align__(8) Pair sum_s[2][kParts];  // every part's sum, written by its CTA into all eight; one for each pass
  __shared__ Pair before_s[kParts], find_s[kWarps], limit_s;
  __shared__ int count_s, n_s, owner_s, found_s[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = int(tc::cta_rank());
  const int64_t seq = blockIdx.x / kCluster;
  const int K = p.max_drafts, V = p.vocab;
  const float* target = p.target + seq * p.target_stride;
  const float* draft = p.draft ? p.draft + seq * p.draft_stride : nullptr;
  const int32_t* toks = p.draft_tokens + seq * K;

  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // this CTA runs
  int n = p.n_drafts ? __ldg(p.n_drafts + seq) : K;  // looked at behind the first loads of the drafts
  if (warp == 0) {
    int a = 0;
    for (int base = 0; base < K; base += 32) {
      const int i = base + lane;
      bool stands = false, bad = false;
      if (i < K) {
        const int x = __ldg(toks + i);
        const float u = __ldg(p.u_accept + seq * K + i);
        if (x >= 0 && x < V) {
          const float pi = __ldg(target + int64_t(i) * V + x);
          const float qi = draft ? __ldg(draft + int64_t(i) * V + x) : 1.f;
          stands = double(u) * double(qi) < double(pi);  // an exact product
        } else {
          bad = true;
        }
      }
      if (base == 0 && (n < 0 || n > K)) {
        if (rank == 0 && lane == 0) atomicOr(&g_status_verify, TPA_DEV_BAD_INPUT);
        n = n < 0 ? 0 : K;
      }
      const unsigned stood = __ballot_sync(0xffffffffu, stands && i < n);
      const int here = stood == 0xffffffffu ? 32 : __ffs(~stood) - 1;
      if (bad && lane == here && i < n && rank == 0) atomicOr(&g_status_verify, TPA_DEV_BAD_INPUT);
      a += here;
      if (here < 32) break;
    }
    if (K == 0 && n != 0 && rank == 0 && lane == 0) atomicOr(&g_status_verify, TPA_DEV_BAD_INPUT);
    if (lane == 0) {
      count_s = a;
      n_s = K == 0 ? 0 : n;
    }
  }
  __syncthreads();
  const int a = count_s;
  n = n_s;
  Row r{target + int64_t(a) * V, nullptr, -1};
  if (a < n) {
    if (draft) r.q = draft + int64_t(a) * V;
    else r.only = __ldg(toks + a);
  }
  const int per = ((V + kParts - 1) / kParts + 3) & ~3;
  const int me = rank * kWarps + warp;
  const int64_t b0 = int64_t(me) * per, b1 = b0 + per;
  const int i0 = int(b0 < V ? b0 : V), i1 = int(b1 < V ? b1 : V);

  // the other CTAs run: their shared memory may be written
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  for (int pass = 0; pass < 2; ++pass) {
    const Pair t = part_sum(r, i0, i1, lane);
    if (lane < kCluster) st_cluster_pair(tc::peer_addr(&sum_s[pass][me], lane), t);
    tc::cluster_sync();  // every part of the row is summed, and known here
    if (warp == 0) {  // prefix sums of the parts, and the part that holds the token
      constexpr int kOwn = kParts / 32;
      Pair v[kOwn], run;
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        v[i] = sum_s[pass][lane * kOwn + i];
        run = run + v[i];
      }
      Pair at, incl;
      warp_scan(run, lane, at, incl);
      const Pair limit = shfl_pair(incl, 31) * __ldg(p.u_next + seq);
      int mine = kParts, some = -1;
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int part = lane * kOwn + i;
        before_s[part] = at;
        at = at + v[i];
        if (v[i].hi > 0.f) {
          some = part;
          if (mine == kParts && at > limit) mine = part;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        mine = min(mine, __shfl_xor_sync(0xffffffffu, mine, o));
        some = max(some, __shfl_xor_sync(0xffffffffu, some, o));
      }
      if (lane == 0) {
        owner_s = mine < kParts ? mine : some;
        limit_s = limit;
      }
    }
    __syncthreads();
    const bool nothing = owner_s < 0;
    if (nothing && pass == 0 && a < n) {  // the draft covers the target: draw from the target's own row
      r.q = nullptr;
      r.only = -1;
      continue;
    }
    int32_t* out = p.tokens + seq * (K + 1);
    if (nothing) {
      if (me == 0 && lane == 0) out[a] = -1;
    } else if (owner_s / kWarps == rank) {
      const int64_t c0 = int64_t(owner_s) * per, c1 = c0 + per;
      const int found = part_find(r, int(c0), int(c1 < V ? c1 : V), before_s[owner_s], limit_s, find_s, found_s);
      if (threadIdx.x == 0) out[a] = found;
    }
    break;
  }
  // what surrounds the drawn token
  if (rank == 0) {
    int32_t* out = p.tokens + seq * (K + 1);
    for (int i = threadIdx.x; i <= K; i += kThreads)
      if (i != a) out[i] = i < a ? __ldg(toks + i) : -1;
    if (threadIdx.x == 0) p.n_accepted[seq] = a;
  }
}

}  // namespace

TPA_DEFINE_STATUS_READER(tpa_internal_status_verify, g_status_verify)

extern "C" int tpa_verify_drafts(const float* target, int64_t target_stride, const float* draft, int64_t draft_stride,
                                 const int32_t* draft_tokens, const int32_t* n_drafts, const float* u_accept,
                                 const float* u_next, int32_t* tokens, int32_t* n_accepted, int32_t n_seqs,
                                 int32_t max_drafts, int32_t vocab, void* stream) {
  TPA_NVTX_RANGE("tpa_verify_drafts");
  if (n_seqs < 0 || n_seqs > 0x7fffffff / kCluster || max_drafts < 0 || max_drafts > 1024 || vocab < 1 ||
      vocab > (1 << 30))
    return TPA_ERR_INVALID_ARG;
  if (n_seqs == 0) return TPA_OK;
  if (!target || !u_next || !tokens || !n_accepted) return TPA_ERR_INVALID_ARG;
  if (max_drafts > 0 && (!draft_tokens || !u_accept)) return TPA_ERR_INVALID_ARG;
  if (target_stride < int64_t(max_drafts + 1) * vocab || (draft && draft_stride < int64_t(max_drafts) * vocab))
    return TPA_ERR_INVALID_ARG;
  const uintptr_t al = reinterpret_cast<uintptr_t>(target) | reinterpret_cast<uintptr_t>(draft) |
                       reinterpret_cast<uintptr_t>(draft_tokens) | reinterpret_cast<uintptr_t>(n_drafts) |
                       reinterpret_cast<uintptr_t>(u_accept) | reinterpret_cast<uintptr_t>(u_next) |
                       reinterpret_cast<uintptr_t>(tokens) | reinterpret_cast<uintptr_t>(n_accepted);
  if (al & 3) return TPA_ERR_INVALID_ARG;
  Params p{target, draft, draft_tokens, n_drafts, u_accept, u_next, tokens, n_accepted, target_stride,
           draft_stride, max_drafts, vocab};
  verify_kernel<<<unsigned(n_seqs) * kCluster, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  TPA_CUDA_TRY(cudaGetLastError());
  return TPA_OK;
}
