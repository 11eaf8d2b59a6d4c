// Head norms and rotary positions: forward, gradient, and the form that
// appends the new tokens of a batch to a paged cache.
//
//   y = R(p) (x r w),  r = rsqrt(mean(x^2) + eps)          (x: one head's d values)
//   z = R(p)^T dy,  h = x r:   dw = sum z h,  dx = r (z w - h mean(z w h))
//
// Bound by HBM: 2 bytes in and 2 out for each value, the cos | sin row of a
// token read once for all its heads.  A row of d values is held by d / 16
// lanes, each with two 16-byte pieces whose pairs of the rotation are both in
// the lane: pieces l and l + rot/16 where halves are paired, pieces 2l and
// 2l + 1 where neighbours are, so the rotation needs no exchange and the norm
// only 3 shuffles (2 for d 64).  All pieces of a lane use cos and sin values
// [8l, 8l + 8) of the token.  The rows of a warp are heads of one token: the
// weights and the angles are in registers for all of them.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "device_common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace {

__device__ unsigned int g_status_rope = 0;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

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

__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(tc::pack_bf16(x[0], x[1]), tc::pack_bf16(x[2], x[3]), tc::pack_bf16(x[4], x[5]),
                    tc::pack_bf16(x[6], x[7]));
}

__device__ __forceinline__ void load_f8(const float* p, float* x) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

__device__ __forceinline__ void load_weight(const void* w, bool bf16, int pa, int pb, float* x) {
  if (bf16) {
    unpack8(__ldg(reinterpret_cast<const uint4*>(w) + pa), x);
    unpack8(__ldg(reinterpret_cast<const uint4*>(w) + pb), x + 8);
  } else {
    load_f8(static_cast<const float*>(w) + 8 * pa, x);
    load_f8(static_cast<const float*>(w) + 8 * pb, x + 8);
  }
}

// cos and sin of this lane's 8 pairs, where it holds any (l < rot / 16)
__device__ __forceinline__ void load_angles(const Rope& r, int pos, int l, float* c, float* s) {
  if (l < (r.rot >> 4)) {
    const float* row = r.table + int64_t(pos) * r.rot + 8 * l;
    load_f8(row, c);
    load_f8(row + (r.rot >> 1), s);
  }
}

// (a, b) <- (a c - b s, b c + a s) for each pair of the lane's 16 values
__device__ __forceinline__ void rotate(float* x, const float* c, const float* s, bool interleaved, float sign) {
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = x[2 * j], b = x[2 * j + 1], sj = sign * s[j];
      x[2 * j] = a * c[j] - b * sj;
      x[2 * j + 1] = b * c[j] + a * sj;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = x[j], b = x[j + 8], sj = sign * s[j];
      x[j] = a * c[j] - b * sj;
      x[j + 8] = b * c[j] + a * sj;
    }
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int D>
__device__ __forceinline__ float rstd16(const float* x, float eps) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
  return rsqrtf(row_sum<Geo<D>::LPR>(ss) * (1.f / D) + eps);
}

// ------------------------------------------------------------------ forward

struct FwdParams {
  Rope rope;
  const int32_t* positions;
  const int32_t* n_tokens;
  int64_t n_rows;
  int32_t t_pad, hq, hkv;
  int32_t sq, skv;  // units of a token for its query rows, and for its key rows
  Rows q, k, v;
  RowsOut qo, ko;
  tpa_paged_view cache;  // append
};

// Rows of a unit: kU groups of RPW rows of one token, all loads issued before
// the first is used (4 KB a warp in flight).
constexpr int kU = 4;

// Number of entries of the sorted array a[0..n) that are <= v, found by the
// whole warp (32 probes a round).  Ends for any contents.
__device__ __forceinline__ int warp_count_le(const int32_t* a, int n, int v, int lane) {
  int lo = 0, len = n;
  while (len > 0) {
    const int step = (len + 31) >> 5;
    const int at = (lane + 1) * step - 1;
    const bool below = at < len && __ldg(a + lo + at) <= v;
    const int cnt = __popc(__ballot_sync(0xffffffffu, below));
    const int done = cnt * step;
    lo += done;
    len = min(step - 1, len - done);
  }
  return lo;
}

template <int D, bool NORM, bool APPEND>
__global__ void __launch_bounds__(kThreads) fwd_kernel(const FwdParams p) {
  using G = Geo<D>;
  const int lane = threadIdx.x & 31, l = lane % G::LPR, sub = lane / G::LPR;
  const int per_token = p.sq + p.skv * (APPEND ? 2 : 1);
  const int64_t unit = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t tok = unit / per_token;
  if (tok >= p.n_rows) return;
  int part = int(unit - tok * per_token);
  int kind = 0;  // query, key, value rows
  if (part >= p.sq) {
    part -= p.sq;
    kind = 1;
    if (APPEND && part >= p.skv) {
      part -= p.skv;
      kind = 2;
    }
  }
  const int heads = kind == 0 ? p.hq : p.hkv;
  const Rows src = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
  const bool inter = p.rope.interleaved != 0;
  int pa, pb;
  pieces<D>(l, p.rope.rot, inter, pa, pb);

  uint4 va[kU], vb[kU];
  const int h0 = part * kU * G::RPW + sub;
  const uint8_t* row = src.p + tok * src.stride + int64_t(h0) * (D * 2);
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    va[u] = vb[u] = make_uint4(0, 0, 0, 0);
    if (h0 + u * G::RPW < heads) {
      const uint4* r = reinterpret_cast<const uint4*>(row + u * (G::RPW * D * 2));
      va[u] = __ldcs(r + pa);
      vb[u] = __ldcs(r + pb);
    }
  }

  int pos;
  int64_t slot_row = 0;  // append: row of (page, head 0, slot) in the cache
  bool pad = false;
  if constexpr (APPEND) {
    const tpa_paged_view& c = p.cache;
    const int s = warp_count_le(c.offsets + 1, c.n_seqs, int(tok), lane);
    if (s >= c.n_seqs) return;  // rows behind the last sequence
    const int first = __ldg(c.offsets + s), last = __ldg(c.offsets + s + 1), kv = __ldg(c.kv_lens + s);
    // in 64 bits: nothing here is known to be in range yet
    const int64_t at = int64_t(kv) - last + tok;
    bool ok = first >= 0 && tok >= first && at >= 0 && at < int64_t(c.max_pages) * c.page_size &&
              (!p.rope.table || at < p.rope.table_rows);
    int page = 0;
    if (ok) {
      page = __ldg(c.pages + int64_t(s) * c.page_stride + int(at) / c.page_size);
      ok = page >= 0 && page < c.n_pages;
    }
    if (!ok) {
      if (lane == 0) atomicOr(&g_status_rope, TPA_DEV_BAD_INPUT);
      return;
    }
    pos = int(at);
    slot_row = int64_t(page) * c.n_heads_kv * c.page_size + pos % c.page_size;
  } else {
    pos = __ldg(p.positions + tok);
    if (p.n_tokens) {
      const int64_t b = tok / p.t_pad;
      pad = int(tok - b * p.t_pad) >= __ldg(p.n_tokens + b);
    }
    if (!pad && pos >= p.rope.table_rows) {
      if (lane == 0) atomicOr(&g_status_rope, TPA_DEV_BAD_INPUT);
      pad = true;
    }
    pad |= pos < 0;
  }

  float w[16], c[8], s[8];
  if (kind < 2 && !pad) {
    if constexpr (NORM) load_weight(kind == 0 ? p.rope.wq : p.rope.wk, p.rope.w_bf16, pa, pb, w);
    load_angles(p.rope, pos, l, c, s);
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int h = h0 + u * G::RPW;
    if (part * kU * G::RPW + u * G::RPW >= heads) break;  // the warp's rows end here
    uint4 oa = va[u], ob = vb[u];
    if (pad) {
      oa = ob = make_uint4(0, 0, 0, 0);
    } else if (kind < 2) {
      float x[16];
      unpack8(oa, x);
      unpack8(ob, x + 8);
      if constexpr (NORM) {
        const float r = rstd16<D>(x, p.rope.eps);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = x[i] * r * w[i];
      }
      if (l < (p.rope.rot >> 4)) rotate(x, c, s, inter, 1.f);
      oa = pack8(x);
      ob = pack8(x + 8);
    }
    if (h < heads) {
      uint8_t* out;
      if (APPEND && kind > 0)
        out = static_cast<uint8_t*>(kind == 1 ? p.cache.k_cache : p.cache.v_cache) +
              (slot_row + int64_t(h) * p.cache.page_size) * (D * 2);
      else
        out = (kind == 0 ? p.qo.p + tok * p.qo.stride : p.ko.p + tok * p.ko.stride) + int64_t(h) * (D * 2);
      reinterpret_cast<uint4*>(out)[pa] = oa;
      reinterpret_cast<uint4*>(out)[pb] = ob;
    }
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
};

constexpr int kBwdU = 2;         // groups of rows whose loads a warp issues together
constexpr int kBwdMaxGrid = 608;  // CTAs: bounds the partial sums

template <bool F32>
struct Grad16 {
  uint4 v[F32 ? 4 : 2];
  __device__ __forceinline__ void load(const uint8_t* row, int pa, int pb) {
    const uint4* r = reinterpret_cast<const uint4*>(row);
    if constexpr (F32) {
      v[0] = __ldcs(r + 2 * pa);
      v[1] = __ldcs(r + 2 * pa + 1);
      v[2] = __ldcs(r + 2 * pb);
      v[3] = __ldcs(r + 2 * pb + 1);
    } else {
      v[0] = __ldcs(r + pa);
      v[1] = __ldcs(r + pb);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (F32 ? 4 : 2); ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float* x) const {
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[4 * i] = __uint_as_float(v[i].x);
        x[4 * i + 1] = __uint_as_float(v[i].y);
        x[4 * i + 2] = __uint_as_float(v[i].z);
        x[4 * i + 3] = __uint_as_float(v[i].w);
      }
    } else {
      unpack8(v[0], x);
      unpack8(v[1], x + 8);
    }
  }
};

template <bool F32>
__device__ __forceinline__ void store16(uint8_t* row, int pa, int pb, const float* x) {
  if constexpr (F32) {
    float4* r = reinterpret_cast<float4*>(row);
    r[2 * pa] = make_float4(x[0], x[1], x[2], x[3]);
    r[2 * pa + 1] = make_float4(x[4], x[5], x[6], x[7]);
    r[2 * pb] = make_float4(x[8], x[9], x[10], x[11]);
    r[2 * pb + 1] = make_float4(x[12], x[13], x[14], x[15]);
  } else {
    reinterpret_cast<uint4*>(row)[pa] = pack8(x);
    reinterpret_cast<uint4*>(row)[pb] = pack8(x + 8);
  }
}

template <int D, bool NORM, bool GIN32, bool GOUT32>
__global__ void __launch_bounds__(kThreads) bwd_kernel(const BwdParams p) {
  using G = Geo<D>;
  constexpr int GB = GIN32 ? 4 : 2, OB = GOUT32 ? 4 : 2;
  __shared__ float part_s[kWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % G::LPR, sub = lane / G::LPR;
  const int64_t n_warps = int64_t(gridDim.x) * kWarps, me = int64_t(blockIdx.x) * kWarps + warp;
  const bool inter = p.rope.interleaved != 0;
  int pa, pb;
  pieces<D>(l, p.rope.rot, inter, pa, pb);

  for (int kind = 0; kind < 2; ++kind) {
    const int heads = kind == 0 ? p.hq : p.hkv;
    const int slices = (heads + G::RPW * kBwdU - 1) / (G::RPW * kBwdU);
    const Rows g = kind == 0 ? p.gq : p.gk, x_in = kind == 0 ? p.q : p.k;
    const RowsOut out = kind == 0 ? p.dq : p.dk;
    float w[16], acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    if constexpr (NORM) load_weight(kind == 0 ? p.rope.wq : p.rope.wk, p.rope.w_bf16, pa, pb, w);
    const int64_t units = p.n_rows * slices;
    for (int64_t unit = me; unit < units; unit += n_warps) {
      const int64_t tok = unit / slices;
      const int hbase = int(unit - tok * slices) * kBwdU * G::RPW, h0 = hbase + sub;
      const int pos = __ldg(p.positions + tok);
      bool pad = pos < 0;
      if (p.n_tokens) {
        const int64_t b = tok / p.t_pad;
        pad |= int(tok - b * p.t_pad) >= __ldg(p.n_tokens + b);
      }
      if (!pad && pos >= p.rope.table_rows) {
        if (lane == 0) atomicOr(&g_status_rope, TPA_DEV_BAD_INPUT);
        pad = true;
      }
      Grad16<GIN32> gv[kBwdU];
      Grad16<false> xv[kBwdU];
#pragma unroll
      for (int u = 0; u < kBwdU; ++u) {
        gv[u].zero();
        xv[u].zero();
        const int h = h0 + u * G::RPW;
        if (!pad && h < heads) {
          gv[u].load(g.p + tok * g.stride + int64_t(h) * (D * GB), pa, pb);
          if constexpr (NORM) xv[u].load(x_in.p + tok * x_in.stride + int64_t(h) * (D * 2), pa, pb);
        }
      }
      float c[8], s[8];
      if (!pad) load_angles(p.rope, pos, l, c, s);
#pragma unroll
      for (int u = 0; u < kBwdU; ++u) {
        if (hbase + u * G::RPW >= heads) break;
        const int h = h0 + u * G::RPW;
        float z[16];
        gv[u].get(z);
        if (!pad) {
          if (l < (p.rope.rot >> 4)) rotate(z, c, s, inter, -1.f);
          if constexpr (NORM) {
            float x[16];
            xv[u].get(x);
            const float r = rstd16<D>(x, p.rope.eps);
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              x[i] *= r;
              acc[i] = fmaf(z[i], x[i], acc[i]);
              z[i] *= w[i];
              dot = fmaf(z[i], x[i], dot);
            }
            dot = row_sum<G::LPR>(dot) * (1.f / D);
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = r * (z[i] - x[i] * dot);
          }
        }
        if (h < heads) store16<GOUT32>(out.p + tok * out.stride + int64_t(h) * (D * OB), pa, pb, z);
      }
    }
    if constexpr (NORM) {
      // rows of the warp, then warps of the CTA, in a fixed order
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int o = G::LPR; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
      if (sub == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          part_s[warp][8 * pa + i] = acc[i];
          part_s[warp][8 * pb + i] = acc[8 + i];
        }
      }
      __syncthreads();
      if (threadIdx.x < D) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) t += part_s[i][threadIdx.x];
        p.partial[(int64_t(blockIdx.x) * 2 + kind) * D + threadIdx.x] = t;
      }
      __syncthreads();
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
  const int rows = (32 / (d / 16)) * kU;
  return (heads + rows - 1) / rows;
}

template <int D, bool APPEND>
int launch_fwd(const FwdParams& p, bool norm, cudaStream_t st) {
  const int per_token = p.sq + p.skv * (APPEND ? 2 : 1);
  const int64_t ctas = (p.n_rows * per_token + kWarps - 1) / kWarps;
  if (ctas > 0x7fffffff) return TPA_ERR_INVALID_ARG;
  if (norm)
    fwd_kernel<D, true, APPEND><<<unsigned(ctas), kThreads, 0, st>>>(p);
  else
    fwd_kernel<D, false, APPEND><<<unsigned(ctas), kThreads, 0, st>>>(p);
  TPA_CUDA_TRY(cudaGetLastError());
  return TPA_OK;
}

template <int D, bool GIN32, bool GOUT32>
int launch_bwd(const BwdParams& p, bool norm, float* dwq, float* dwk, cudaStream_t st) {
  const int rows = Geo<D>::RPW * kBwdU;
  const int64_t units = p.n_rows * ((p.hq + rows - 1) / rows);
  const int64_t want = (units + kWarps - 1) / kWarps;
  const int grid = int(want < 1 ? 1 : want < kBwdMaxGrid ? want : kBwdMaxGrid);
  if (!norm) {
    bwd_kernel<D, false, GIN32, GOUT32><<<grid, kThreads, 0, st>>>(p);
    TPA_CUDA_TRY(cudaGetLastError());
    return TPA_OK;
  }
  bwd_kernel<D, true, GIN32, GOUT32><<<grid, kThreads, 0, st>>>(p);
  TPA_CUDA_TRY(cudaGetLastError());
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
  p.skv = units_of(n_heads_kv, d);
  p.q = {static_cast<const uint8_t*>(q), q_stride * 2};
  p.k = {static_cast<const uint8_t*>(k), k_stride * 2};
  p.qo = {static_cast<uint8_t*>(q_out), q_out_stride * 2};
  p.ko = {static_cast<uint8_t*>(k_out), k_out_stride * 2};
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
  if (!c || !c->k_cache || !c->v_cache || !c->pages || !c->offsets || !c->kv_lens) return TPA_ERR_INVALID_ARG;
  if (!aligned16(c->k_cache) || !aligned16(c->v_cache)) return TPA_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return TPA_ERR_INVALID_ARG;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return TPA_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->n_seqs < 1 || c->max_pages < 1 || c->page_stride < c->max_pages || c->n_rows < 0 ||
      c->n_heads_kv < 1 || c->n_heads_kv > 65535)
    return TPA_ERR_INVALID_ARG;
  if (int64_t(c->n_pages) * c->n_heads_kv >= (int64_t(1) << 31) / c->page_size) return TPA_ERR_INVALID_ARG;
  // positions are held in 32 bits
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
  p.skv = units_of(cache->n_heads_kv, d);
  p.q = {static_cast<const uint8_t*>(q), q_stride * 2};
  p.k = {static_cast<const uint8_t*>(k), k_stride * 2};
  p.v = {static_cast<const uint8_t*>(v), v_stride * 2};
  p.qo = {static_cast<uint8_t*>(q_out), q_out_stride * 2};
  p.cache = *cache;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d == 128 ? launch_fwd<128, true>(p, rope->q_weight, st) : launch_fwd<64, true>(p, rope->q_weight, st);
}
