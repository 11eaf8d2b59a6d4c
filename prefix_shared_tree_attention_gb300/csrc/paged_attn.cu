// Attention of each sequence's new tokens over a paged key/value cache.
//
//   O_i = sum_j softmax_j(scale q_i . k_j) v_j  over the keys j <= pos_i (and
//   j > pos_i - window with a window),  LSE_i = log sum_j exp(scale q_i . k_j)
//
// The queries of a key/value head's group are the rows of one tile: row
// r = token * group + head, so every key and value is read once for all of
// them.  Here: the checks, the choice of the kernel, and the joining of tiles
// whose keys were split over several CTAs.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "device_common.cuh"
#include "internal.h"
#include "paged_common.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace {

using namespace paged;

// Joins the parts of a tile whose steps went to several CTAs.  The parts'
// values, maxima and sums are loaded together; parts are added in a fixed order.
// With 16 parts or fewer (the usual case: a tile on two or three CTAs) a warp
// takes a row; with more (a long sequence by itself) the CTA's eight warps take
// a share of one row's parts each.
constexpr int kFewParts = 16;

template <int D>
__device__ __forceinline__ void join_row_by_warp(const Params& p, const Split& s, int r, int lane) {
  constexpr int V = D / 32;  // columns of a lane
  using Vec = typename std::conditional<V == 4, float4, float2>::type;
  const int parts = s.c1 - s.c0 + 1;
  auto slot = [&](int i) { return int64_t(2) * (s.c0 + i) + (i == 0 ? 1 : 0); };
  float2 ml = make_float2(-INFINITY, 0.f);  // lane i: part i
  if (lane < parts) ml = p.part_ml[slot(lane) * p.rows + r];
  float acc[V], top = -INFINITY, mu = 0.f, a = 0.f, sum = 0.f;
#pragma unroll
  for (int c = 0; c < V; ++c) acc[c] = 0.f;
#pragma unroll
  for (int k0 = 0; k0 < kFewParts; k0 += 8) {
    if (k0 >= parts) break;
    Vec v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[k] = Vec{};
      if (k0 + k < parts) v[k] = reinterpret_cast<const Vec*>(p.part_o + (slot(k0 + k) * p.rows + r) * D)[lane];
    }
    if (k0 == 0) {
      top = warp_max_f(ml.x);
      mu = top == -INFINITY ? 0.f : top;
      a = tc::ex2(ml.x - mu);
      sum = ml.y * a;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float w = __shfl_sync(0xffffffffu, a, k0 + k);
      const float* f = reinterpret_cast<const float*>(&v[k]);
      if (k0 + k < parts) {
#pragma unroll
        for (int c = 0; c < V; ++c) acc[c] = fmaf(f[c], w, acc[c]);
      }
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const int tok = r / p.b.group, head = s.head * p.b.group + r - tok * p.b.group;
  const int64_t row = int64_t(s.first + tok) * p.hq + head;
  uint32_t w[V / 2];
#pragma unroll
  for (int c = 0; c < V / 2; ++c) w[c] = tc::pack_bf16(acc[2 * c] * inv, acc[2 * c + 1] * inv);
  uint32_t* out = reinterpret_cast<uint32_t*>(p.o + row * D) + lane * (V / 2);
  if constexpr (V == 4) *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
  else out[0] = w[0];
  if (lane == 0) p.lse[row] = sum > 0.f ? (mu + __log2f(sum)) * kLn2 : -INFINITY;
}

template <int D>
__global__ void __launch_bounds__(256, 4) paged_join_kernel(const Params p) {
  constexpr int V = D / 32;  // columns of a lane
  constexpr int kMost = (kMaxGrid + 7) / 8;
  constexpr int kAhead = 5;  // parts of a warp whose values are under way together
  using Vec = typename std::conditional<V == 4, float4, float2>::type;
  __shared__ float acc_s[8][D];
  __shared__ float scale_s[kMaxGrid];
  __shared__ float top_s[8], sum_s[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  tc::grid_launch_dependents();
  tc::grid_wait_prior();
  const Split s = p.split[blockIdx.x];
  if (!s.valid) return;
  const int parts = s.c1 - s.c0 + 1;
  if (parts <= kFewParts) {
    for (int r = blockIdx.y * 8 + warp; r < s.n * p.b.group; r += gridDim.y * 8) join_row_by_warp<D>(p, s, r, lane);
    return;
  }
  auto slot = [&](int i) { return int64_t(2) * (s.c0 + i) + (i == 0 ? 1 : 0); };
  for (int r = blockIdx.y; r < s.n * p.b.group; r += gridDim.y) {
    float2 ml = make_float2(-INFINITY, 0.f);  // thread i: part i
    if (int(threadIdx.x) < parts) ml = p.part_ml[slot(threadIdx.x) * p.rows + r];
    auto value = [&](int k) {
      const int i = warp + 8 * k;
      Vec v = {};
      if (i < parts) v = reinterpret_cast<const Vec*>(p.part_o + (slot(i) * p.rows + r) * D)[lane];
      return v;
    };
    Vec v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) v[k] = value(k);
    float top = warp_max_f(ml.x);
    if (lane == 0) top_s[warp] = top;
    __syncthreads();
    top = top_s[0];
#pragma unroll
    for (int w = 1; w < 8; ++w) top = fmaxf(top, top_s[w]);
    const float mu = top == -INFINITY ? 0.f : top;
    const float a = tc::ex2(ml.x - mu);
    float sum = ml.y * a;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) sum_s[warp] = sum;
    if (int(threadIdx.x) < kMaxGrid) scale_s[threadIdx.x] = int(threadIdx.x) < parts ? a : 0.f;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] = 0.f;
#pragma unroll
    for (int k0 = 0; k0 < kMost; k0 += kAhead) {
      if (warp + 8 * k0 >= parts) break;
      if (k0 > 0) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) v[k] = value(k0 + k);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = warp + 8 * (k0 + k);
        if (i < parts) {
          const float w = scale_s[i];
          const float* f = reinterpret_cast<const float*>(&v[k]);
#pragma unroll
          for (int c = 0; c < V; ++c) acc[c] = fmaf(f[c], w, acc[c]);
        }
      }
    }
#pragma unroll
    for (int c = 0; c < V; ++c) acc_s[warp][lane * V + c] = acc[c];
    __syncthreads();
    if (threadIdx.x < D / 2) {
      float t = 0.f, x = 0.f, y = 0.f;
      const int c = threadIdx.x * 2;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        t += sum_s[w];
        x += acc_s[w][c];
        y += acc_s[w][c + 1];
      }
      const float inv = t > 0.f ? 1.f / t : 0.f;
      const int tok = r / p.b.group, head = s.head * p.b.group + r - tok * p.b.group;
      const int64_t row = int64_t(s.first + tok) * p.hq + head;
      *reinterpret_cast<uint32_t*>(p.o + row * D + c) = tc::pack_bf16(x * inv, y * inv);
      if (threadIdx.x == 0) p.lse[row] = t > 0.f ? (mu + __log2f(t)) * kLn2 : -INFINITY;
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ host side

// Multiprocessors of the current device, after a check that the kernels run on it.
int device_sms(int* sms) {
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return TPA_ERR_CUDA;
  }
  return major == 10 && minor == 3 ? TPA_OK : TPA_ERR_UNSUPPORTED_DEVICE;
}

// Rows of a tile: 16 or 32 while every sequence's queries fit in them, else 256.
int tile_rows(int64_t max_q, int group) {
  const int64_t rows = max_q * group;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 256;
}

uint64_t part_bytes(int rows, int d) {
  return uint64_t(2) * kMaxGrid * rows * (uint64_t(d) * 4 + 8) + uint64_t(kMaxGrid) * sizeof(Split);
}

template <int D>
int launch_join(const Params& p, int grid, int64_t rows, cudaStream_t st) {
  return launch_overlapped(paged_join_kernel<D>, dim3(grid, unsigned(rows < 8 ? rows : 8)), 256, 0, st,
                           static_cast<const Params>(p));
}

}  // namespace

extern "C" uint64_t tpa_paged_attn_workspace_bytes(int32_t max_q_len, int32_t n_heads_q, int32_t n_heads_kv,
                                                   int32_t head_dim) {
  if (max_q_len < 1 || n_heads_kv < 1 || n_heads_q < 1 || n_heads_q % n_heads_kv || n_heads_q / n_heads_kv > 64 ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  return part_bytes(tile_rows(max_q_len, n_heads_q / n_heads_kv), head_dim);
}

extern "C" int tpa_paged_attn_fwd(const tpa_paged_view* cache, const void* q, int64_t q_stride, void* o, float* lse,
                                  int32_t n_heads_q, int32_t max_q_len, float softmax_scale, int32_t window,
                                  void* workspace, uint64_t workspace_bytes, void* stream) {
  TPA_NVTX_RANGE("tpa_paged_attn_fwd");
  const int rc = tpa_internal_check_paged(cache);
  if (rc != TPA_OK) return rc;
  const int d = cache->head_dim, hkv = cache->n_heads_kv;
  if (n_heads_q < 1 || n_heads_q > 65535 || n_heads_q % hkv || n_heads_q / hkv > 64 || window < 0 ||
      max_q_len < (cache->n_rows ? 1 : 0) || std::isnan(softmax_scale) || std::isinf(softmax_scale))
    return TPA_ERR_INVALID_ARG;
  if (cache->n_rows == 0) return TPA_OK;
  auto al = [](const void* x, uintptr_t a) { return (reinterpret_cast<uintptr_t>(x) & (a - 1)) == 0; };
  if (!q || !o || !lse || !workspace || !al(q, 16) || !al(o, 16) || !al(lse, 4) || !al(workspace, 256) ||
      q_stride < int64_t(n_heads_q) * d || q_stride % 8 || q_stride >= (int64_t(1) << 40))
    return TPA_ERR_INVALID_ARG;
  const int group = n_heads_q / hkv, R = tile_rows(max_q_len, group);
  const int64_t rows = int64_t(max_q_len) * group;  // of the largest sequence
  if (workspace_bytes < part_bytes(R, d)) return TPA_ERR_BUFFER_TOO_SMALL;
  Params p = {};
  p.b.pages = cache->pages;
  p.b.offsets = cache->offsets;
  p.b.kv_lens = cache->kv_lens;
  p.b.n_pages = cache->n_pages;
  p.b.page_shift = cache->page_size == 16 ? 4 : cache->page_size == 32 ? 5 : cache->page_size == 64 ? 6 : 7;
  p.b.n_seqs = cache->n_seqs;
  p.b.max_pages = cache->max_pages;
  p.b.page_stride = cache->page_stride;
  p.b.hkv = hkv;
  p.b.n_rows = cache->n_rows;
  p.b.group = group;
  // positions are below 2^30: a longer window reaches no further, and differences with this one stay in 32 bits
  p.b.window = window < (1 << 30) ? window : 1 << 30;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = q_stride;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.hq = n_heads_q;
  p.rows = R;
  p.scale_log2 = (softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf(float(d))) * kLog2e;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + uint64_t(2) * kMaxGrid * R * d * 4);
  p.split = reinterpret_cast<Split*>(ws + uint64_t(2) * kMaxGrid * R * (uint64_t(d) * 4 + 8));
  int sms = 0;
  const int dv = device_sms(&sms);
  if (dv != TPA_OK) return dv;
  const int grid = sms < kMaxGrid ? sms : kMaxGrid;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int rt = R == 256 ? tpa_internal_paged_tile(cache, p, grid, st) : tpa_internal_paged_few(cache, p, R, grid, st);
  if (rt != TPA_OK) return rt;
  return d == 128 ? launch_join<128>(p, grid, rows, st) : launch_join<64>(p, grid, rows, st);
}
