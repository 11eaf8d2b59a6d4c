// Paged attention for many rows (chunks of a prompt): tcgen05 tiles.
//
// A tile is two sub-tiles of 128 rows, row r = token * group + head, so a K/V
// tile of 128 keys is read once for 256 / group tokens of all the group's
// heads.  The roles and the softmax are those of the tree attention's forward:
//   warpgroup 0, 1    softmax of sub-tile h: thread r owns row r (TMEM lane r),
//                     online in the log2 domain; P goes to TMEM over S as the
//                     bf16 operand of the second MMA; O is rescaled in TMEM
//                     only when a row's maximum has grown by 2^8
//   warps 8, 10, 11   one thread each: walk this CTA's steps and load the pages of
//                     K (and hand each segment to the other roles), of V, and Q (a
//                     page of 16 to 128 slots is a box; one of 128-byte rows
//                     swizzled as the MMA descriptors want)
//   warp 9            one thread issues the MMAs
// A tile whose tokens all fit in the first sub-tile (a sequence's last tile; one
// new token next to others' chunks) leaves the second one's work out.
// Work: 4 d operations and one exponential for each (row, key).  Bound by the way
// from a step's scores to the next's, which each sub-tile goes alone: at d 128
// 1024 cycles of MMAs, 1350 of softmax and 600 of handing over by barriers, so that
// with two sub-tiles the MMAs run 69 % of the time (72 by the counters).  4001 tokens
// after 28002 cached ones, 32/8 heads: 1.30 to 1.43 ms with the clock that the power cap
// leaves, 1380 to 1510 TFLOP/s (measured GEMM rates: 1939 in a burst, 1739 sustained).
// Polling the barriers without suspending, and one arrival a warp instead of one a
// thread, gave nothing or lost 2 %.
// Few rows cost no more here than in the kernel made for them: one chunk of 512 tokens
// beside 63 single ones of other sequences takes 114 us, the two by themselves 32 and 79.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "device_common.cuh"
#include "internal.h"
#include "paged_common.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace {

__device__ unsigned int g_status_ptile = 0;

using namespace paged;
using tc::add2;
using tc::f2;
using tc::fma2;
using tc::unf2;

constexpr uint32_t kChunk = 128 * 128;  // bytes of a 128-row x 64-column bf16 tile

constexpr int NH = 2;  // sub-tiles

template <int D>
struct TileCfg {
  static constexpr int NCH = D / 64;
  static constexpr uint32_t TILE = NCH * kChunk;  // 128 x D bf16
  static constexpr uint32_t STAGE = NH * 4 * 4096;  // 32 rows x 128 bytes of results a warp
  static constexpr int NS_FIT = int((kSmemMax - 2048 - STAGE - NH * TILE) / (2 * TILE));
  static constexpr int NS = NS_FIT > 3 ? 3 : NS_FIT;  // K and V ring depth
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_K = OFF_Q + NH * TILE;
  static constexpr uint32_t OFF_V = OFF_K + NS * TILE;
  static constexpr uint32_t OFF_STAGE = OFF_V + NS * TILE;
  static constexpr uint32_t OFF_SCAN = OFF_STAGE + STAGE;
  static constexpr uint32_t OFF_SEG = OFF_SCAN + 160;
  static constexpr uint32_t OFF_BAR = OFF_SEG + 128;
  // q_full, q_empty, k_full[NS], k_empty[NS], v_full[NS], v_empty[NS], s_full[NH], p_full[2 NH], o_free[NH],
  // o_final[NH], drain, seg_full[2], seg_empty[2]
  static constexpr int NBAR = 2 + 4 * NS + 5 * NH + 1 + 4;
  static constexpr uint32_t OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr uint32_t BYTES = OFF_MISC + 16 + 1024;
  // Registers move from the producer/issuer warpgroup to the
  // softmax warpgroups, within what the CTA was launched with.
  static constexpr int THREADS = 384;
  static constexpr int REG_LAUNCH = 168, REG_LOW = 120, REG_HIGH = 184;
  static_assert(REG_HIGH * 256 + REG_LOW * 128 <= REG_LAUNCH * 384, "register split");
  static constexpr uint32_t TMEM_COLS = 512;
  // P is handed over in this many parts, so that its product can begin while the rest is formed.  Two shorten the way
  // from scores to scores where it is what the MMAs wait for: 4001 tokens at d 64 495 -> 450 us (now 462, since the
  // sub-tiles' ends are apart).  At d 128, with twice the MMA work in the same softmax, they cost 1 to 2 % (8 chunks
  // of 512: 160.5 -> 162.5 us).
  static constexpr int PARTS = D == 64 ? 2 : 1;
  static_assert(sizeof(Scan) <= 160 && sizeof(Segment) * 2 <= 128 && NS >= 2, "layout");
  static_assert(BYTES <= kSmemMax, "shared memory budget");
};

template <int D>
__global__ void __launch_bounds__(TileCfg<D>::THREADS, 1)
    paged_tile_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const Params p) {
  using C = TileCfg<D>;
  constexpr int NCH = C::NCH, NS = C::NS, PARTS = C::PARTS;
  constexpr uint32_t TILE = C::TILE;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  Scan* sc = reinterpret_cast<Scan*>(smem + C::OFF_SCAN);
  volatile Segment* seg_ring = reinterpret_cast<volatile Segment*>(smem + C::OFF_SEG);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_empty = q_full + 1;
  uint64_t* k_full = q_full + 2;
  uint64_t* k_empty = k_full + NS;
  uint64_t* v_full = k_empty + NS;
  uint64_t* v_empty = v_full + NS;
  uint64_t* s_full = v_empty + NS;
  uint64_t* p_full = s_full + NH;  // [part][sub-tile]
  uint64_t* o_free = p_full + 2 * NH;
  uint64_t* o_final = o_free + NH;
  uint64_t* drain = o_final + NH;
  uint64_t* seg_full = drain + 1;   // [2]
  uint64_t* seg_empty = drain + 3;  // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);

  const int warp = threadIdx.x >> 5;
  constexpr int W_K = 4 * NH, W_MMA = W_K + 1, W_V = W_K + 2, W_Q = W_K + 3;
  const int sub_tok = p.b.tile_tok / NH;  // tokens of a sub-tile

  if (threadIdx.x == 0) {
    tc::mbar_init(q_full, 1);
    tc::mbar_init(q_empty, 1);
    for (int s = 0; s < NS; ++s) {
      tc::mbar_init(k_full + s, 1);
      tc::mbar_init(k_empty + s, 1);
      tc::mbar_init(v_full + s, 1);
      tc::mbar_init(v_empty + s, 1);
    }
    for (int h = 0; h < NH; ++h) {
      tc::mbar_init(s_full + h, 1);
      tc::mbar_init(p_full + h, 128);
      tc::mbar_init(p_full + NH + h, 128);
      tc::mbar_init(o_free + h, 128);
      tc::mbar_init(o_final + h, 1);
    }
    tc::mbar_init(drain, 1);
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(seg_full + s, 1);
      tc::mbar_init(seg_empty + s, 1 + 128 * NH);
    }
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == W_MMA) tc::tmem_alloc(tmem_slot, C::TMEM_COLS);
  tc::tc_fence_before();
  // From here on memory is read and written that the kernel before may write and read.
  tc::grid_wait_prior();
  tc::grid_launch_dependents();  // the joining kernel waits for this one's end by itself
  const Shares shares = scan_batch(p.b, sc, &g_status_ptile);
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (int(blockIdx.x) >= shares.n) {  // nothing to do here
    if (threadIdx.x == 0) write_split(p, sc, shares, &g_status_ptile);
  } else if (warp >= W_K) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REG_LOW));
    if (warp == W_K || warp == W_V) {
      // ---------------------------------------------------------- producers: one thread for the keys (and the segments
      // that the other roles read), one for the values; each walks the steps.  One thread for both, with the queries
      // too, was what the MMAs waited for: 3000 cycles a step, whatever the head size.
      const bool keys = warp == W_K;
      if (tc::elect_one()) {
        const CUtensorMap* tm = keys ? &tm_k : &tm_v;
        tc::tma_prefetch_desc(tm);
        auto wait1 = [&](uint64_t* b_, uint32_t par) { return tc::mbar_wait(b_, par, abort_flag, &g_status_ptile); };
        LoadRing ring{keys ? k_full : v_full, keys ? k_empty : v_empty, keys ? sK : sV};
        Walk w;
        w.start(p.b, sc, shares);
        bool ok = true, more = w.end > w.begin;
        for (int k = 0; ok; ++k) {
          const int n_it = more ? w.end - w.begin : -1;
          const int key0 = (w.t.step0 + w.begin) * kStep;
          if (keys) {
            if (!(ok = wait1(seg_empty + (k & 1), ((k >> 1) & 1) ^ 1))) break;
            volatile Segment* sg = seg_ring + (k & 1);
            sg->n_it = n_it;
            sg->head = w.head;
            sg->first = w.t.first;
            sg->n = w.t.n;
            sg->pos0 = w.t.pos0;
            sg->lo = w.t.lo;
            sg->hi = w.t.end;
            sg->key0 = key0;
            sg->whole = w.begin == 0 && w.end == w.t.steps;
            sg->slot = blockIdx.x * 2 + (w.begin == 0 ? 1 : 0);
            tc::mbar_arrive(seg_full + (k & 1));
          }
          if (!more) break;
          ok = load_steps<NS, NCH>(p.b, ring, tm, p.b.pages + int64_t(w.seq) * p.b.page_stride, w.head, key0, n_it,
                                          w.t.lo, w.t.end, &g_status_ptile, wait1);
          if (ok) more = w.next(p.b);
        }
        if (*abort_flag) {  // let the copies already issued land before the CTA exits
          volatile int never = 0;
          for (int j = (ring.t > NS ? ring.t - NS : 0); j < ring.t; ++j)
            tc::mbar_wait(ring.full + (j % NS), (j / NS) & 1, &never, &g_status_ptile, 100000000ull);
        }
      }
      __syncwarp();
    } else if (warp == W_Q) {
      // ---------------------------------------------------------- one thread for the queries of each segment
      if (tc::elect_one()) {
        tc::tma_prefetch_desc(&tm_q);
        const uint32_t q_bytes = uint32_t(NCH) * sub_tok * p.b.group * 128;  // of a sub-tile
        Walk w;
        w.start(p.b, sc, shares);
        int nq = 0;
        bool more = w.end > w.begin;
        while (more && tc::mbar_wait(q_empty, (nq & 1) ^ 1, abort_flag, &g_status_ptile)) {
          const int nh = w.t.n > sub_tok ? NH : 1;
          tc::mbar_arrive_expect_tx(q_full, nh * q_bytes);
          for (int h = 0; h < nh; ++h)
            for (int c = 0; c < NCH; ++c)
              tc::tma_load_3d(sQ + h * TILE + c * kChunk, &tm_q, q_full, c * 64, w.head * p.b.group,
                              w.t.first + h * sub_tok);
          if (nq++ == 0) write_split(p, sc, shares, &g_status_ptile);
          more = w.next(p.b);
        }
        if (*abort_flag && nq > 0) {
          volatile int never = 0;
          tc::mbar_wait(q_full, (nq - 1) & 1, &never, &g_status_ptile, 100000000ull);
        }
      }
      __syncwarp();
    } else if (warp == W_MMA) {
      // ---------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc_qk = tc::idesc_bf16(128, 128, false, false);
      constexpr uint32_t idesc_pv = tc::idesc_bf16(128, D, false, true);
      const uint64_t dQ = tc::smem_desc(tc::smem_u32(sQ), 16, 1024);
      const uint64_t dK = tc::smem_desc(tc::smem_u32(sK), 16, 1024);
      const uint64_t dV = tc::smem_desc(tc::smem_u32(sV), kChunk, 1024);
      auto issue_s = [&](int h, int s) {  // S_h = Q_h K(s)^T
        const uint64_t qa = dQ + ((h * TILE) >> 4), kb_ = dK + ((s * TILE) >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * kChunk + (k & 3) * 32) >> 4;
          tc::mma_ss(tmem + h * 128, qa + off, kb_ + off, idesc_qk, k > 0);
        }
        tc::mma_commit(s_full + h);
      };
      auto issue_pv = [&](int h, int s, int part, bool first) {  // O_h (+)= P_h V(s), a part of the keys
        const uint64_t vb = dV + ((s * TILE) >> 4);
#pragma unroll
        for (int k = part * (8 / PARTS); k < (part + 1) * (8 / PARTS); ++k)
          mma_ts(tmem + 128 * NH + h * 128, tmem + h * 128 + k * 8, vb + ((k * 2048) >> 4), idesc_pv,
                 (!first || k > 0) ? 1u : 0u);
      };
      auto wait1 = [&](uint64_t* b_, uint32_t par) { return tc::mbar_wait(b_, par, abort_flag, &g_status_ptile); };
      if (tc::elect_one()) {
        int t = 0;                    // steps so far
        int uses[NH] = {}, segs[NH] = {};  // of them each sub-tile's, and its segments
        bool ok = true;
        for (int k = 0; ok; ++k) {
          if (!(ok = wait1(seg_full + (k & 1), (k >> 1) & 1))) break;
          const int n_it = seg_ring[k & 1].n_it, nh = seg_ring[k & 1].n > sub_tok ? NH : 1;
          tc::mbar_arrive(seg_empty + (k & 1));
          if (n_it < 0) break;
          if (!(ok = wait1(q_full, k & 1) && wait1(k_full + t % NS, (t / NS) & 1))) break;
          tc::tc_fence_after();
          for (int h = 0; h < nh; ++h) issue_s(h, t % NS);
          tc::mma_commit(k_empty + t % NS);
          if (n_it == 1) tc::mma_commit(q_empty);
          for (int j = 0; ok && j < n_it; ++j) {
            const int g = t + j, sv = g % NS, s1 = (g + 1) % NS;
            const bool more = j + 1 < n_it;
            if (!(ok = wait1(v_full + sv, (g / NS) & 1))) break;
#pragma unroll
            for (int h = 0; h < NH; ++h) {
              if (h >= nh) break;
#pragma unroll
              for (int part = 0; ok && part < PARTS; ++part) {
                if (!(ok = wait1(p_full + part * NH + h, uses[h] & 1))) break;
                if (part == 0 && j == 0 && segs[h]++ > 0 && !(ok = wait1(o_free + h, segs[h] & 1))) break;
                tc::tc_fence_after();
                issue_pv(h, sv, part, part == 0 && j == 0);
              }
              if (!ok) break;
              ++uses[h];
              if (!more) tc::mma_commit(o_final + h);
              if (more) {
                if (h == 0 && !(ok = wait1(k_full + s1, ((g + 1) / NS) & 1))) break;
                tc::tc_fence_after();
                issue_s(h, s1);
              }
            }
            if (!ok) break;
            tc::mma_commit(v_empty + sv);
            if (more) {
              tc::mma_commit(k_empty + s1);
              if (j + 2 == n_it) tc::mma_commit(q_empty);  // the segment's last S was just issued
            }
          }
          t += n_it;
        }
        if (*abort_flag) {  // let issued MMAs finish before TMEM is released
          volatile int never = 0;
          tc::mma_commit(drain);
          tc::mbar_wait(drain, 0, &never, &g_status_ptile, 100000000ull);
        }
      }
      __syncwarp();
    }
  } else if (warp < 4 * NH) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REG_HIGH));
    // ------------------------------------------------------------ softmax (sub-tile h)
    const int h = warp >> 2;
    const int r = threadIdx.x & 127, lane = threadIdx.x & 31;  // row of the sub-tile = TMEM lane
    uint8_t* const stage = smem + C::OFF_STAGE + warp * 4096;
    const int tok = h * sub_tok + r / p.b.group, gh = r % p.b.group;
    const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + h * 128;
    const uint32_t tO = tmem + lane_base + 128 * NH + h * 128;
    const uint64_t sl2 = f2(p.scale_log2, p.scale_log2);
    auto wait_all = [&](uint64_t* b_, uint32_t par) {
      return __all_sync(0xffffffffu, tc::mbar_wait(b_, par, abort_flag, &g_status_ptile));
    };
    int tb = 0, uses = 0, segs = 0;  // steps so far, of them this sub-tile's, and its segments
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!wait_all(seg_full + (k & 1), (k >> 1) & 1)) break;
      const volatile Segment* sg = seg_ring + (k & 1);
      const int n_it = sg->n_it, first = sg->first, n_tok = sg->n, lo = sg->lo, end = sg->hi, key_first = sg->key0;
      const int slot = sg->whole ? -1 : sg->slot, head = sg->head * p.b.group + gh, pos_first = sg->pos0;
      tc::mbar_arrive(seg_empty + (k & 1));
      if (n_it < 0) break;
      if (h * sub_tok >= n_tok) {  // nothing in this sub-tile
        tb += n_it;
        continue;
      }
      const bool live = r < sub_tok * p.b.group && tok < n_tok;
      const int pos = live ? pos_first + tok : -1;
      // every live row of the sub-tile sees the keys in [all_lo, all_hi)
      const int all_hi = pos_first + h * sub_tok + 1;
      const int all_lo = p.b.window > 0 ? pos_first + min((h + 1) * sub_tok, n_tok) - p.b.window : 0;
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = 0; j < n_it; ++j) {
        const int key0 = key_first + j * kStep;
        if (!wait_all(s_full + h, uses & 1)) { ok = false; break; }
        ++uses;
        if (key0 < lo || key0 + kStep > end) {
          // Slots that no row sees may hold anything: zero their values, so that 0 x NaN does not come in.  (Those from
          // the last key that this tile sees to the sequence's end are loaded, and finite: other rows see them.)  This S was
          // issued behind waits for the V of all steps before, so the stage's last V has landed and this wait can only
          // end with this step's.
          const int g = tb + j, sv_ = g % NS;
          if (!wait_all(v_full + sv_, (g / NS) & 1)) { ok = false; break; }
          const int head_rows = min(max(lo - key0, 0), kStep), live_rows = min(max(end - key0, 0), kStep);
#pragma unroll
          for (int c = 0; c < NCH; ++c) {
            uint4* v = reinterpret_cast<uint4*>(sV + sv_ * TILE + c * kChunk);
            for (int i = r; i < head_rows * 8; i += 128) v[i] = make_uint4(0, 0, 0, 0);
            for (int i = live_rows * 8 + r; i < kStep * 8; i += 128) v[i] = make_uint4(0, 0, 0, 0);
          }
          tc::fence_proxy_async_smem();
        }
        tc::tc_fence_after();
        uint32_t sv[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::tmem_ld32(tS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(sv + c * 32));
        tc::tmem_ld_wait();
        if (key0 + kStep > all_hi || key0 < all_lo) {
          const int last = pos - key0;
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c > last) sv[c] = 0xff800000u;  // -inf
          if (p.b.window > 0) {
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (c <= last - p.b.window) sv[c] = 0xff800000u;
          }
        }
        // row max: 8 independent chains, then a short tree
        float mxs[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) mxs[t] = fmaxf(__uint_as_float(sv[2 * t]), __uint_as_float(sv[2 * t + 1]));
#pragma unroll
        for (int c = 16; c < 128; c += 16)
#pragma unroll
          for (int t = 0; t < 8; ++t)
            mxs[t] = max3(mxs[t], __uint_as_float(sv[c + 2 * t]), __uint_as_float(sv[c + 2 * t + 1]));
        const float mx = fmaxf(max3(mxs[0], mxs[1], mxs[2]), max3(mxs[3], mxs[4], max3(mxs[5], mxs[6], mxs[7])));
        const float m_new = fmaxf(m_run, mx * p.scale_log2);
        const bool resc = m_new > m_run + kRescale;
        float alpha = 1.f;
        if (resc) {
          alpha = tc::ex2(m_run - m_new);
          m_run = m_new;
        }
        const float m_use = (m_run == -INFINITY) ? 0.f : m_run;
        const uint64_t negm = f2(-m_use, -m_use);
        auto rescale = [&] {  // O holds the result of the step before: s_full was committed after it
          if (j < 1 || !__any_sync(0xffffffffu, resc)) return;
          constexpr int W = PARTS > 1 ? 16 : 32;  // columns at a time: while the scores are held there is room for 16
#pragma unroll
          for (int c = 0; c < D; c += W) {
            uint32_t ov[W];
            if constexpr (W == 16) tc::tmem_ld16(tO + c, ov);
            else tc::tmem_ld32(tO + c, ov);
            tc::tmem_ld_wait();
#pragma unroll
            for (int u = 0; u < W; ++u) ov[u] = __float_as_uint(__uint_as_float(ov[u]) * alpha);
            if constexpr (W == 16) tc::tmem_st16(tO + c, ov);
            else tc::tmem_st32(tO + c, ov);
          }
        };
        if (PARTS > 1) rescale();
        // P goes over the first 64 columns of S
        uint64_t sum2[4] = {f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f)};  // 4 chains
#pragma unroll
        for (int part = 0; part < PARTS; ++part) {
          constexpr int N = 64 / PARTS;
          uint32_t pk[N];
#pragma unroll
          for (int c = 0; c < N; ++c) {
            const int at = part * 2 * N + 2 * c;
            float a, bb;
            unf2(fma2(f2(__uint_as_float(sv[at]), __uint_as_float(sv[at + 1])), sl2, negm), a, bb);
            const float p0 = tc::ex2(a), p1 = tc::ex2(bb);
            sum2[c & 3] = add2(sum2[c & 3], f2(p0, p1));
            pk[c] = tc::pack_bf16(p0, p1);
          }
          if (PARTS == 1) rescale();  // here the scores' registers are free
#pragma unroll
          for (int c = 0; c < N; c += 32)
            tc::tmem_st32(tS + part * N + c, *reinterpret_cast<const uint32_t(*)[32]>(pk + c));
          tc::tmem_st_wait();
          tc::tc_fence_before();
          tc::mbar_arrive(p_full + part * NH + h);
        }
        float s_lo, s_hi;
        unf2(add2(add2(sum2[0], sum2[1]), add2(sum2[2], sum2[3])), s_lo, s_hi);
        l_run = l_run * alpha + (s_lo + s_hi);
      }
      if (!ok || !wait_all(o_final + h, segs & 1)) { ok = false; break; }
      ++segs;
      tc::tc_fence_after();
      const float inv = slot < 0 ? (l_run > 0.f ? 1.f / l_run : 0.f) : 1.f;
      const int64_t row = int64_t(first + tok) * p.hq + head;
      const int64_t prow = int64_t(slot) * p.rows + tok * p.b.group + gh;
      // The rows leave through shared memory, 128 bytes of each at a time and a warp's rows by itself, so that a store
      // covers four whole lines.  Straight from the registers, where each of a store's 32 pieces is in a line of its
      // own, a tile's end took 5500 cycles (10000 for a part in fp32), two to three steps' time: 8 chunks of 512 tokens
      // 160.5 us, so 148.5 (now 135).
      uint8_t* const to = slot < 0 ? reinterpret_cast<uint8_t*>(p.o) : reinterpret_cast<uint8_t*>(p.part_o);
      const int64_t mine = live ? (slot < 0 ? row * (D * 2) : prow * (D * 4)) : -1;
      int64_t at[8];  // of rows 4 i + lane / 8
#pragma unroll
      for (int i = 0; i < 8; ++i) at[i] = __shfl_sync(0xffffffffu, mine, 4 * i + (lane >> 3));
      auto write_piece = [&](int piece, const uint32_t (&w)[32]) {
        __syncwarp();  // the piece before is read
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(stage + lane * 128 + ((c ^ (lane & 7)) << 4)) =
              make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        __syncwarp();
        const int c = lane & 7;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r_ = 4 * i + (lane >> 3);
          const uint4 v = *reinterpret_cast<const uint4*>(stage + r_ * 128 + ((c ^ (r_ & 7)) << 4));
          if (at[i] >= 0) *reinterpret_cast<uint4*>(to + at[i] + piece * 128 + c * 16) = v;
        }
      };
      auto loaded = [&](bool last) {
        tc::tmem_ld_wait();
        if (last) {
          tc::tc_fence_before();
          tc::mbar_arrive(o_free + h);  // O may be overwritten by the next segment
        }
      };
      if (slot < 0) {
        uint32_t ov[D];
#pragma unroll
        for (int c = 0; c < D; c += 32) tc::tmem_ld32(tO + c, *reinterpret_cast<uint32_t(*)[32]>(ov + c));
        loaded(true);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t w[32];
#pragma unroll
          for (int x = 0; x < 32; ++x)
            w[x] = tc::pack_bf16(__uint_as_float(ov[64 * c + 2 * x]) * inv, __uint_as_float(ov[64 * c + 2 * x + 1]) * inv);
          write_piece(c, w);
        }
      } else {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32];
          tc::tmem_ld32(tO + c * 32, ov);
          loaded(c == D / 32 - 1);
          write_piece(c, ov);
        }
      }
      if (live) {
        if (slot < 0)
          p.lse[row] = l_run > 0.f ? (m_run + __log2f(l_run)) * kLn2 : -INFINITY;
        else
          p.part_ml[prow] = make_float2(m_run, l_run);
      }
      tb += n_it;
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == W_MMA) tc::tmem_dealloc(tmem, C::TMEM_COLS);
}

template <int D>
int launch_tile(const tpa_paged_view* c, Params& p, int grid, cudaStream_t st) {
  using C = TileCfg<D>;
  const int sub_tok = 128 / p.b.group;
  CUtensorMap tq, tk, tv;
  const uint64_t rows = uint64_t(c->n_pages) * c->n_heads_kv * c->page_size;
  if (!query_map(&tq, c, p, sub_tok) || !cache_map(&tk, c->k_cache, rows, D, c->page_size) ||
      !cache_map(&tv, c->v_cache, rows, D, c->page_size))
    return TPA_ERR_CUDA;
  p.b.tile_tok = NH * sub_tok;
  TPA_CUDA_TRY(cudaFuncSetAttribute(paged_tile_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES));
  {
    cudaFuncAttributes fa;
    TPA_CUDA_TRY(cudaFuncGetAttributes(&fa, paged_tile_kernel<D>));
    if (fa.numRegs != C::REG_LAUNCH) return TPA_ERR_BAD_BUILD;  // the setmaxnreg split would not add up
  }
  return launch_overlapped(paged_tile_kernel<D>, dim3(grid), C::THREADS, C::BYTES, st, tq, tk, tv,
                           static_cast<const Params>(p));
}

}  // namespace

TPA_DEFINE_STATUS_READER(tpa_internal_status_ptile, g_status_ptile)

int tpa_internal_paged_tile(const tpa_paged_view* c, Params& p, int grid, cudaStream_t st) {
  return c->head_dim == 128 ? launch_tile<128>(c, p, grid, st) : launch_tile<64>(c, p, grid, st);
}
