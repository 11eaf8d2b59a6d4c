// Verification of drafted tokens against the target's probabilities, with the
// next token drawn from what is left: one cluster of 8 CTAs a sequence.
//
// The acceptance run needs one entry of each row: every CTA forms it for
// itself (a warp, 32 drafts at a time).  It names the one row (or pair of
// rows) whose weights r(v) = max(p(v) - q(v), 0) are summed and searched:
// 4 bytes of p and 4 of q for each entry, read from HBM once, which bounds
// the kernel.  Each warp sums a contiguous 1/128 of the row; the 128 sums are
// exchanged through distributed shared memory; the warp in whose part the
// running sum passes u * total reads that part again (from L2) and finds the
// token.
//
// A draw has to be the same whatever the order of summation, so sums are held
// to far more than fp32: r and the running sum are unevaluated pairs hi + lo
// of fp32 (error-free additions), about 2^-46 of the sum, and fp64 from the
// lanes' totals on.  fp64 throughout would cost more than the reads: this GPU
// has a few fp64 operations a cycle and SM, and a row needs five an entry.
#include <cuda_runtime.h>

#include "device_common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace {

__device__ unsigned int g_status_verify = 0;

constexpr int kCluster = 8;
constexpr int kThreads = 512;
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

struct Sum {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float p, float q) {
    float h, l;
    weight(p, q, h, l);
    const float s = __fadd_rn(hi, h), b = __fsub_rn(s, hi);
    const float e = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(h, b));
    hi = s;
    lo = __fadd_rn(lo, __fadd_rn(e, l));
  }
  __device__ __forceinline__ double value() const { return double(hi) + double(lo); }
};

__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// inclusive prefix sums over the lanes
__device__ __forceinline__ double warp_scan_d(double v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

// Where a row's weights come from: p, and what is taken off it.
struct Row {
  const float* p;
  const float* q;  // NULL: nothing, or all on `only`
  int32_t only;    // -1: none
};

// This warp's sum of the weights in [i0, i1), i0 a multiple of 4.
__device__ double part_sum(const Row& r, int i0, int i1, int lane) {
  Sum a, b;  // two chains
  const bool vec = ((reinterpret_cast<uintptr_t>(r.p) | reinterpret_cast<uintptr_t>(r.q)) & 15) == 0;
  if (vec) {
    constexpr int kU = 4;
    int i = i0 + 4 * lane;
    for (; i + 128 * (kU - 1) + 4 <= i1; i += 128 * kU) {
      float4 p[kU], q[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        p[u] = __ldg(reinterpret_cast<const float4*>(r.p + i + 128 * u));
        q[u] = r.q ? __ldg(reinterpret_cast<const float4*>(r.q + i + 128 * u)) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        a.add(p[u].x, q[u].x);
        b.add(p[u].y, q[u].y);
        a.add(p[u].z, q[u].z);
        b.add(p[u].w, q[u].w);
      }
    }
    for (; i < i1; i += 128)
      for (int t = i; t < min(i + 4, i1); ++t) a.add(__ldg(r.p + t), r.q ? __ldg(r.q + t) : 0.f);
  } else {
    constexpr int kU = 8;
    int i = i0 + lane;
    for (; i + 32 * (kU - 1) < i1; i += 32 * kU) {
      float p[kU], q[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        p[u] = __ldg(r.p + i + 32 * u);
        q[u] = r.q ? __ldg(r.q + i + 32 * u) : 0.f;
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) (u & 1 ? b : a).add(p[u], q[u]);
    }
    for (; i < i1; i += 32) a.add(__ldg(r.p + i), r.q ? __ldg(r.q + i) : 0.f);
  }
  double t = a.value() + b.value();
  // the drafted token of a draft without probabilities: its weight is taken out again
  t = warp_sum_d(t);
  if (r.only >= i0 && r.only < i1) {
    // summed anew without it, so that nothing is lost where it holds nearly all the weight
    Sum c;
    for (int i = i0 + lane; i < i1; i += 32)
      if (i != r.only) c.add(__ldg(r.p + i), 0.f);
    t = warp_sum_d(c.value());
  }
  return t;
}

// The lowest v in [i0, i1) at which `before` plus the weights up to v pass
// `limit`; the last v with a weight where none does, -1 without any.
__device__ int part_find(const Row& r, int i0, int i1, double before, double limit, int lane) {
  int last = -1;
  double run = before;
  for (int base = i0; base < i1; base += 32) {
    const int i = base + lane;
    float h = 0.f, l = 0.f;
    if (i < i1 && i != r.only) weight(__ldg(r.p + i), r.q ? __ldg(r.q + i) : 0.f, h, l);
    const double w = double(h) + double(l);
    const double s = run + warp_scan_d(w, lane);
    const unsigned hit = __ballot_sync(0xffffffffu, w > 0.0 && s > limit);
    if (hit) return base + __ffs(hit) - 1;
    const unsigned any = __ballot_sync(0xffffffffu, w > 0.0);
    if (any) last = base + 31 - __clz(any);
    run = __shfl_sync(0xffffffffu, s, 31);
  }
  return last;
}

__device__ __forceinline__ double ld_cluster_f64(uint32_t addr) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
  return v;
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) verify_kernel(const Params p) {
  __shared__ double sum_s[2][kWarps];    // this CTA's parts; the two passes use one each
  __shared__ double prefix_s[kParts];
  __shared__ double limit_s;
  __shared__ int count_s, owner_s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = int(tc::cta_rank());
  const int64_t seq = blockIdx.x / kCluster;
  const int K = p.max_drafts, V = p.vocab;
  const float* target = p.target + seq * p.target_stride;
  const float* draft = p.draft ? p.draft + seq * p.draft_stride : nullptr;
  const int32_t* toks = p.draft_tokens + seq * K;

  int n = K;
  if (p.n_drafts) {
    n = __ldg(p.n_drafts + seq);
    if (n < 0 || n > K) {
      if (rank == 0 && threadIdx.x == 0) atomicOr(&g_status_verify, TPA_DEV_BAD_INPUT);
      n = n < 0 ? 0 : K;
    }
  }
  if (warp == 0) {
    int a = 0;
    for (int base = 0; base < n; base += 32) {
      const int i = base + lane;
      bool stands = false, bad = false;
      if (i < n) {
        const int x = __ldg(toks + i);
        if (x >= 0 && x < V) {
          const float pi = __ldg(target + int64_t(i) * V + x);
          const float qi = draft ? __ldg(draft + int64_t(i) * V + x) : 1.f;
          stands = double(__ldg(p.u_accept + seq * K + i)) * double(qi) < double(pi);  // an exact product
        } else {
          bad = true;
        }
      }
      const unsigned stood = __ballot_sync(0xffffffffu, stands);
      const int run = __ffs(~stood) - 1;  // 32 (-1 of ffs 0) when all stand
      const int here = stood == 0xffffffffu ? 32 : run;
      if (bad && lane == here && rank == 0) atomicOr(&g_status_verify, TPA_DEV_BAD_INPUT);
      a += here;
      if (here < 32) break;
    }
    if (lane == 0) count_s = a < n ? a : n;
  }
  __syncthreads();
  const int a = count_s;
  Row r{target + int64_t(a) * V, nullptr, -1};
  if (a < n) {
    if (draft) r.q = draft + int64_t(a) * V;
    else r.only = __ldg(toks + a);
  }
  const int per = ((V + kParts - 1) / kParts + 3) & ~3;
  const int me = rank * kWarps + warp;
  const int64_t b0 = int64_t(me) * per, b1 = b0 + per;
  const int i0 = int(b0 < V ? b0 : V), i1 = int(b1 < V ? b1 : V);

  for (int pass = 0; pass < 2; ++pass) {
    const double t = part_sum(r, i0, i1, lane);
    if (lane == 0) sum_s[pass][warp] = t;
    tc::cluster_sync();  // every part of the row is summed
    if (threadIdx.x < kParts)
      prefix_s[threadIdx.x] =
          ld_cluster_f64(tc::peer_addr(&sum_s[pass][threadIdx.x % kWarps], threadIdx.x / kWarps));
    __syncthreads();
    if (warp == 0) {  // prefix sums of the parts, and the part that holds the token
      double v[kParts / 32], run = 0.0;
#pragma unroll
      for (int i = 0; i < kParts / 32; ++i) {
        v[i] = prefix_s[lane * (kParts / 32) + i];
        run += v[i];
      }
      const double incl = warp_scan_d(run, lane), total = __shfl_sync(0xffffffffu, incl, 31);
      const double limit = double(__ldg(p.u_next + seq)) * total;
      double at = incl - run;  // may differ from the sum of the parts before by a rounding: only compared upwards
      int mine = kParts, some = -1;
#pragma unroll
      for (int i = 0; i < kParts / 32; ++i) {
        const int part = lane * (kParts / 32) + i;
        prefix_s[part] = at;
        at += v[i];
        if (v[i] > 0.0) {
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
    } else if (owner_s == me) {
      const int found = part_find(r, i0, i1, prefix_s[me], limit_s, lane);
      if (lane == 0) out[a] = found;
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
  tc::cluster_sync();  // no CTA leaves while another may read its sums
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
