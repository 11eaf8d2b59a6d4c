// Attention of each sequence's new tokens over a paged key/value cache.
//
//   O_i = sum_j softmax_j(scale q_i . k_j) v_j  over the keys j <= pos_i (and
//   j > pos_i - window with a window),  LSE_i = log sum_j exp(scale q_i . k_j)
//
// The queries of a key/value head's group are the rows of one tile: row
// r = token * group + head, so every key and value is read once for all of
// them.  Few rows (a decode step, a few drafted tokens) leave the reads of the
// cache as the bound; paged_rows_kernel below is for those.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "device_common.cuh"
#include "internal.h"
#include "paged_common.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace {

__device__ unsigned int g_status_paged = 0;

using namespace paged;

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ------------------------------------------------------------------ few rows
//
// Rows of 16 MT (tokens x heads), keys dealt to the CTA's eight warps 16 at a
// time.  A warp is on its own from the load of its keys and values (its own
// ring of NST stages, filled by TMA with 128-byte swizzle, running ahead across
// tiles) to its own maximum, sum and output; the eight are joined once a tile.
// m16n8k16 MMAs: with at most 32 rows the tensor work is a small part of the
// time that the reads take, and 128-row tcgen05 tiles would be empty but for
// those rows.
template <int D, int MT>
struct RowsCfg {
  static constexpr int WARPS = 8, THREADS = 256;
  static constexpr int R = 16 * MT;
  static constexpr int KEYS = 16;                        // keys of a warp's unit
  static constexpr uint32_t CH = KEYS * 128;             // one 64-column piece of a unit
  static constexpr uint32_t UNIT = 2 * (D / 64) * CH;    // K and V of a unit
  static constexpr uint32_t MERGE = 4 * R * D * 4;       // four warps' sums
  static constexpr uint32_t ML = 2 * WARPS * R * 8;      // two buffers of (maximum, sum)
  static constexpr uint32_t FIXED = MERGE + ML + 2112 + 512;
  static constexpr int NST_FIT = int((kSmemMax - 1024 - FIXED) / (WARPS * UNIT));
  static constexpr int NST = NST_FIT > 4 ? 4 : NST_FIT;
  static constexpr uint32_t OFF_MERGE = WARPS * NST * UNIT;
  static constexpr uint32_t OFF_ML = OFF_MERGE + MERGE;
  static constexpr uint32_t OFF_SCAN = OFF_ML + ML;
  static constexpr uint32_t OFF_BAR = OFF_SCAN + 2112;
  static constexpr uint32_t BYTES = OFF_BAR + 512 + 1024;
  static_assert(sizeof(Scan) <= 2112 && WARPS * NST * 8 + 16 <= 512 && NST >= 2, "layout");
  static_assert(BYTES <= kSmemMax, "shared memory budget");
};

template <int D, int MT>
__global__ void __launch_bounds__(256, 1)
    paged_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const Params p) {
  using C = RowsCfg<D, MT>;
  constexpr int NST = C::NST, NT = D / 8, KS = D / 16, R = C::R;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float2* merge = reinterpret_cast<float2*>(smem + C::OFF_MERGE);
  float2* ml_s = reinterpret_cast<float2*>(smem + C::OFF_ML);
  Scan* sc = reinterpret_cast<Scan*>(smem + C::OFF_SCAN);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + warp * NST;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_BAR + C::WARPS * NST * 8);
  uint8_t* ring = smem + warp * NST * C::UNIT;

  tc::grid_launch_dependents();  // the joining kernel waits for this one's end by itself
  if (threadIdx.x == 0) *abort_flag = 0;
  if (lane == 0) {
    for (int s = 0; s < NST; ++s) tc::mbar_init(full + s, 1);
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&tm_k);
    tc::tma_prefetch_desc(&tm_v);
  }
  const long long per_head = scan_batch(p.b, sc, &g_status_paged);
  const long long total = per_head * p.b.hkv;
  const int n_ctas = used_ctas(total, gridDim.x, p.min_steps);
  if (int(blockIdx.x) >= n_ctas) {
    if (threadIdx.x == 0) p.split[blockIdx.x].valid = 0;
    return;
  }
  const long long f0 = cta_begin(total, n_ctas, blockIdx.x), f1 = cta_begin(total, n_ctas, blockIdx.x + 1);
  Walk cur;
  cur.start(p.b, sc, per_head, f0, f1 - f0);
  if (threadIdx.x == 0) write_split(p, cur, total, n_ctas);

  // -------- this warp's loads: the units of its steps in order, ahead of their use
  Walk ld = cur;
  int ld_step = ld.begin, ld_count = 0, pg_base = ld.begin, pg = 0;
  bool ld_more = true, dead = false;
  auto unit_key = [&](const Tile& t, int step) { return ((t.step0 + step) * C::WARPS + warp) * C::KEYS; };
  auto load_pages = [&]() {  // the pages of this warp's units of the next 32 steps, one a lane
    pg_base = ld_step;
    const int k0 = unit_key(ld.t, ld_step + lane);
    pg = 0;
    if (ld_step + lane < ld.end && k0 < ld.t.hi && k0 + C::KEYS > ld.t.lo) {
      pg = __ldg(p.b.pages + int64_t(ld.seq) * p.b.page_stride + (k0 >> p.b.page_shift));
      if (pg < 0 || pg >= p.b.n_pages) {  // never followed: page 0 is read in its place
        atomicOr(&g_status_paged, TPA_DEV_BAD_INPUT);
        pg = 0;
      }
    }
  };
  load_pages();
  auto produce = [&]() {  // loads the next unit, if there is one
    while (ld_more) {
      if (ld_step >= ld.end) {
        ld_more = ld.next(p.b);
        if (!ld_more) return;
        ld_step = ld.begin;
        load_pages();
      }
      if (ld_step - pg_base >= 32) load_pages();
      const int k0 = unit_key(ld.t, ld_step);
      const int page = __shfl_sync(0xffffffffu, pg, ld_step - pg_base);
      ++ld_step;
      if (k0 >= ld.t.hi || k0 + C::KEYS <= ld.t.lo) continue;
      const int s = ld_count % NST;
      if (lane == 0) {
        uint8_t* dst = ring + s * C::UNIT;
        const int row = ((page * p.b.hkv + ld.head) << p.b.page_shift) + (k0 & (p.b.page_size - 1));
        tc::mbar_arrive_expect_tx(full + s, C::UNIT);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          tma_load_2d(dst + c * C::CH, &tm_k, full + s, c * 64, row);
          tma_load_2d(dst + (D / 64 + c) * C::CH, &tm_v, full + s, c * 64, row);
        }
      }
      ++ld_count;
      return;
    }
  };
  __syncwarp();
#pragma unroll
  for (int s = 0; s < NST; ++s) produce();

  int used = 0, parity = 0;
  const int r_lo = lane >> 2;
  bool more = true;
  for (; more; parity ^= 1) {
    const Tile t = cur.t;
    const int rows = t.n * p.b.group;
    const bool whole = cur.begin == 0 && cur.end == t.steps;
    const int slot = blockIdx.x * 2 + (cur.begin == 0 ? 1 : 0);
    // query fragments; rows past the tile are zero and see nothing
    uint32_t qf[MT][KS][4];
    int pos[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = m * 16 + h * 8 + r_lo;
        const bool live = r < rows;
        const int tok = live ? r / p.b.group : 0;
        pos[m][h] = live ? t.pos0 + tok : -1;
        const __nv_bfloat16* src =
            p.q + int64_t(t.first + tok) * p.q_stride + int64_t(cur.head * p.b.group + (live ? r - tok * p.b.group : 0)) * D +
            (lane & 3) * 2;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          qf[m][k][h] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + k * 16)) : 0u;
          qf[m][k][h + 2] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + k * 16 + 8)) : 0u;
        }
      }
    float o[MT][NT][4];
    float mx[MT][2], l[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[m][n][i] = 0.f;
      mx[m][0] = mx[m][1] = -INFINITY;
      l[m][0] = l[m][1] = 0.f;
    }
    // every token of the tile sees the keys in [all_lo, all_hi); what rows past the tile compute is not used
    const int all_hi = t.pos0 + 1;
    const int all_lo = p.b.window > 0 ? t.pos0 + t.n - p.b.window : 0;

    for (int step = cur.begin; step < cur.end; ++step) {
      const int k0 = unit_key(t, step);
      if (k0 >= t.hi || k0 + C::KEYS <= t.lo) continue;
      const int s = used % NST;
      if (!dead && !__all_sync(0xffffffffu, tc::mbar_wait(full + s, (used / NST) & 1, abort_flag, &g_status_paged))) {
        dead = true;
        ld_more = false;
      }
      ++used;
      if (dead) continue;
      const uint32_t kb = tc::smem_u32(ring + s * C::UNIT), vb = kb + (D / 64) * C::CH;
      float sv[MT][2][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) sv[m][n][i] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t b[4];
        ldsm4(kb + (k >> 2) * C::CH + tc::sw128_offset(((lane >> 4) << 3) + (lane & 7), (k & 3) * 2 + ((lane >> 3) & 1)), b);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          mma16816(sv[m][0], qf[m][k], b[0], b[1]);
          mma16816(sv[m][1], qf[m][k], b[2], b[3]);
        }
      }
      const bool open = k0 + C::KEYS <= all_hi && k0 >= all_lo;  // nothing to mask
      uint32_t pf[MT][4];
      bool grow = false;
      float top[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (!open) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = k0 + n * 8 + (lane & 3) * 2 + (i & 1), at = pos[m][i >> 1];
              if (key > at || (p.b.window > 0 && key <= at - p.b.window)) sv[m][n][i] = -INFINITY;
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          top[m][h] = fmaxf(fmaxf(sv[m][0][2 * h], sv[m][0][2 * h + 1]), fmaxf(sv[m][1][2 * h], sv[m][1][2 * h + 1])) *
                      p.scale_log2;
          grow |= top[m][h] > mx[m][h] + kRescale;
        }
      }
      // the maximum is moved only when some row's has grown by 2^8: exact, since
      // numerator and denominator keep the same one
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v = top[m][h];
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
            v = fmaxf(v, mx[m][h]);
            const float a = v > mx[m][h] ? tc::ex2(mx[m][h] - v) : 1.f;
            mx[m][h] = v;
            l[m][h] *= a;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              o[m][n][2 * h] *= a;
              o[m][n][2 * h + 1] *= a;
            }
          }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mu = mx[m][h] == -INFINITY ? 0.f : mx[m][h];
          float e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) e[i] = tc::ex2(fmaf(sv[m][i >> 1][2 * h + (i & 1)], p.scale_log2, -mu));
          l[m][h] += (e[0] + e[1]) + (e[2] + e[3]);
          // probabilities enter the second product as bf16, its operand type
          pf[m][h] = tc::pack_bf16(e[0], e[1]);
          pf[m][2 + h] = tc::pack_bf16(e[2], e[3]);
        }
      // values of keys that no row sees may be anything: zero, so that 0 x NaN does not come in
      uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
      if (k0 < t.lo || k0 + C::KEYS > t.hi) {
        const int key = k0 + (lane & 3) * 2;
        auto in = [&](int x) { return x >= t.lo && x < t.hi; };
        keep0 = (in(key) ? 0xffffu : 0u) | (in(key + 1) ? 0xffff0000u : 0u);
        keep1 = (in(key + 8) ? 0xffffu : 0u) | (in(key + 9) ? 0xffff0000u : 0u);
      }
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
        uint32_t b[4];
        ldsm4_t(vb + (n >> 3) * C::CH + tc::sw128_offset((((lane >> 3) & 1) << 3) + (lane & 7), (n & 7) + (lane >> 4)), b);
        b[0] &= keep0;
        b[1] &= keep1;
        b[2] &= keep0;
        b[3] &= keep1;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          mma16816(o[m][n], pf[m], b[0], b[1]);
          mma16816(o[m][n + 1], pf[m], b[2], b[3]);
        }
      }
      __syncwarp();  // every lane has read the stage
      produce();
    }

    // -------- join the eight warps
    float2* ml = ml_s + parity * (C::WARPS * R);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[m][h] += __shfl_xor_sync(0xffffffffu, l[m][h], 1);
        l[m][h] += __shfl_xor_sync(0xffffffffu, l[m][h], 2);
        if ((lane & 3) == 0) ml[warp * R + m * 16 + h * 8 + r_lo] = make_float2(mx[m][h], l[m][h]);
      }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) top = fmaxf(top, ml[w * R + m * 16 + h * 8 + r_lo].x);
        const float a = mx[m][h] == -INFINITY ? 0.f : tc::ex2(mx[m][h] - top);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          o[m][n][2 * h] *= a;
          o[m][n][2 * h + 1] *= a;
        }
      }
    auto at = [&](int w, int m, int n, int h) { return merge + (((w * MT + m) * NT + n) * 2 + h) * 32; };
    if (warp >= 4) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) at(warp - 4, m, n, h)[lane] = make_float2(o[m][n][2 * h], o[m][n][2 * h + 1]);
    }
    __syncthreads();
    if (warp < 4) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float2 v = at(warp, m, n, h)[lane];
            v.x += o[m][n][2 * h];
            v.y += o[m][n][2 * h + 1];
            at(warp, m, n, h)[lane] = v;
          }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < R * NT; e += C::THREADS) {  // 8 columns of a row
      const int r8 = e & 7, h = (e >> 3) & 1, n = (e >> 4) % NT, m = (e >> 4) / NT;
      const int r = m * 16 + h * 8 + r8;
      if (r >= rows) continue;
      float v[8] = {};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float4* src = reinterpret_cast<const float4*>(at(w, m, n, h) + r8 * 4);
        const float4 x = src[0], y = src[1];
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
      }
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < C::WARPS; ++w) top = fmaxf(top, ml[w * R + r].x);
      const float mu = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int w = 0; w < C::WARPS; ++w) sum += ml[w * R + r].y * tc::ex2(ml[w * R + r].x - mu);
      if (whole) {
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        const int tok = r / p.b.group, head = cur.head * p.b.group + r - tok * p.b.group;
        const int64_t row = int64_t(t.first + tok) * p.hq + head;
        *reinterpret_cast<uint4*>(p.o + row * D + n * 8) =
            make_uint4(tc::pack_bf16(v[0] * inv, v[1] * inv), tc::pack_bf16(v[2] * inv, v[3] * inv),
                       tc::pack_bf16(v[4] * inv, v[5] * inv), tc::pack_bf16(v[6] * inv, v[7] * inv));
        if (n == 0) p.lse[row] = sum > 0.f ? (mu + __log2f(sum)) * kLn2 : -INFINITY;
      } else {
        float4* dst = reinterpret_cast<float4*>(p.part_o + (int64_t(slot) * R + r) * D + n * 8);
        dst[0] = make_float4(v[0], v[1], v[2], v[3]);
        dst[1] = make_float4(v[4], v[5], v[6], v[7]);
        if (n == 0) p.part_ml[int64_t(slot) * R + r] = make_float2(top, sum);
      }
    }
    more = cur.next(p.b);
  }
  if (dead && lane == 0) {  // let the copies already issued land before the CTA exits
    volatile int never = 0;
    for (int j = ld_count > NST ? ld_count - NST : 0; j < ld_count; ++j)
      tc::mbar_wait(full + (j % NST), (j / NST) & 1, const_cast<volatile int*>(&never), &g_status_paged, 100000000ull);
  }
}

// Joins the parts of a tile whose steps went to several CTAs: a warp takes one
// row and a share of the parts, the CTA's four warps are joined through shared
// memory.  Parts are added in a fixed order.
template <int D>
__global__ void __launch_bounds__(128) paged_join_kernel(const Params p, int R) {
  constexpr int V = D / 32;  // columns of a lane
  __shared__ float acc_s[4][D];
  __shared__ float2 ml_s[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  tc::grid_wait_prior();
  const Split s = p.split[blockIdx.x];
  if (!s.valid) return;
  const int parts = s.c1 - s.c0 + 1;
  auto slot = [&](int i) { return int64_t(2) * (s.c0 + i) + (i == 0 ? 1 : 0); };
  for (int r = blockIdx.y; r < s.n * p.b.group; r += gridDim.y) {
    float top = -INFINITY;
    for (int i = lane; i < parts; i += 32) top = fmaxf(top, p.part_ml[slot(i) * R + r].x);
    top = warp_max_f(top);
    const float mu = top == -INFINITY ? 0.f : top;
    float acc[V], sum = 0.f;
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] = 0.f;
#pragma unroll 4
    for (int i = warp; i < parts; i += 4) {
      const float2 ml = p.part_ml[slot(i) * R + r];
      const float a = tc::ex2(ml.x - mu);
      sum = fmaf(ml.y, a, sum);
      const float* src = p.part_o + (slot(i) * R + r) * D + lane * V;
#pragma unroll
      for (int c = 0; c < V; ++c) acc[c] = fmaf(src[c], a, acc[c]);
    }
#pragma unroll
    for (int c = 0; c < V; ++c) acc_s[warp][lane * V + c] = acc[c];
    if (lane == 0) ml_s[warp].x = sum;
    __syncthreads();
    if (threadIdx.x < D / 2) {
      const float t = (ml_s[0].x + ml_s[1].x) + (ml_s[2].x + ml_s[3].x);
      const float inv = t > 0.f ? 1.f / t : 0.f;
      const int tok = r / p.b.group, head = s.head * p.b.group + r - tok * p.b.group;
      const int64_t row = int64_t(s.first + tok) * p.hq + head;
      const int c = threadIdx.x * 2;
      const float x = (acc_s[0][c] + acc_s[1][c]) + (acc_s[2][c] + acc_s[3][c]);
      const float y = (acc_s[0][c + 1] + acc_s[1][c + 1]) + (acc_s[2][c + 1] + acc_s[3][c + 1]);
      *reinterpret_cast<uint32_t*>(p.o + row * D + c) = tc::pack_bf16(x * inv, y * inv);
      if (threadIdx.x == 0) p.lse[row] = t > 0.f ? (mu + __log2f(t)) * kLn2 : -INFINITY;
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ host side

int num_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return 148;
  }
  return sms;
}

// Rows of a tile: 16 or 32 (m16n8k16) while every sequence's queries fit in
// them, else tcgen05 tiles of 128, or pairs of them when that leaves them full.
int tile_rows(int64_t max_q, int group) {
  const int64_t rows = max_q * group;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 128 ? 128 : 256;
}

uint64_t part_bytes(int rows, int d) {
  return uint64_t(2) * kMaxGrid * rows * (uint64_t(d) * 4 + 8) + uint64_t(kMaxGrid) * sizeof(Split);
}

template <int D>
int launch_join(const Params& p, int grid, int R, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, R < 32 ? R : 32);
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  TPA_CUDA_TRY(cudaLaunchKernelEx(&cfg, paged_join_kernel<D>, p, R));
  return TPA_OK;
}

template <int D, int MT>
int launch_rows(const tpa_paged_view* c, Params& p, int grid, cudaStream_t st) {
  using C = RowsCfg<D, MT>;
  CUtensorMap tk, tv;
  const uint64_t rows = uint64_t(c->n_pages) * c->n_heads_kv * c->page_size;
  if (!cache_map(&tk, c->k_cache, rows, D, C::KEYS) || !cache_map(&tv, c->v_cache, rows, D, C::KEYS)) return TPA_ERR_CUDA;
  p.b.tile_tok = C::R / p.b.group;
  p.min_steps = 1;
  TPA_CUDA_TRY(cudaFuncSetAttribute(paged_rows_kernel<D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES));
  paged_rows_kernel<D, MT><<<grid, C::THREADS, C::BYTES, st>>>(tk, tv, p);
  TPA_CUDA_TRY(cudaGetLastError());
  return launch_join<D>(p, grid, C::R, st);
}

}  // namespace

TPA_DEFINE_STATUS_READER(tpa_internal_status_paged, g_status_paged)

extern "C" uint64_t tpa_paged_attn_workspace_bytes(int32_t max_q_len, int32_t n_heads_q, int32_t n_heads_kv,
                                                   int32_t head_dim) {
  if (max_q_len < 1 || n_heads_kv < 1 || n_heads_q < 1 || n_heads_q % n_heads_kv || n_heads_q / n_heads_kv > 32 ||
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
  if (n_heads_q < 1 || n_heads_q > 65535 || n_heads_q % hkv || n_heads_q / hkv > 32 || max_q_len < 1 || window < 0 ||
      std::isnan(softmax_scale) || std::isinf(softmax_scale))
    return TPA_ERR_INVALID_ARG;
  if (cache->n_rows == 0) return TPA_OK;
  auto al = [](const void* x, uintptr_t a) { return (reinterpret_cast<uintptr_t>(x) & (a - 1)) == 0; };
  if (!q || !o || !lse || !workspace || !al(q, 16) || !al(o, 16) || !al(lse, 4) || !al(workspace, 256) ||
      q_stride < int64_t(n_heads_q) * d || q_stride % 8 || q_stride >= (int64_t(1) << 40))
    return TPA_ERR_INVALID_ARG;
  const int group = n_heads_q / hkv, R = tile_rows(max_q_len, group);
  if (workspace_bytes < part_bytes(R, d)) return TPA_ERR_BUFFER_TOO_SMALL;
  Params p = {};
  p.b.pages = cache->pages;
  p.b.offsets = cache->offsets;
  p.b.kv_lens = cache->kv_lens;
  p.b.n_pages = cache->n_pages;
  p.b.page_size = cache->page_size;
  p.b.page_shift = cache->page_size == 16 ? 4 : cache->page_size == 32 ? 5 : cache->page_size == 64 ? 6 : 7;
  p.b.n_seqs = cache->n_seqs;
  p.b.max_pages = cache->max_pages;
  p.b.page_stride = cache->page_stride;
  p.b.hkv = hkv;
  p.b.n_rows = cache->n_rows;
  p.b.group = group;
  p.b.window = window;
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
  const int sms = num_sms(), grid = sms < kMaxGrid ? sms : kMaxGrid;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (R >= 128) {
    const int rt = tpa_internal_paged_tile(cache, p, R, grid, st);
    if (rt != TPA_OK) return rt;
    return d == 128 ? launch_join<128>(p, grid, R, st) : launch_join<64>(p, grid, R, st);
  }
  if (d == 128) return R == 16 ? launch_rows<128, 1>(cache, p, grid, st) : launch_rows<128, 2>(cache, p, grid, st);
  return R == 16 ? launch_rows<64, 1>(cache, p, grid, st) : launch_rows<64, 2>(cache, p, grid, st);
}
