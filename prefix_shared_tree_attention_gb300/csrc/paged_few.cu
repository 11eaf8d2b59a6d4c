// Paged attention for few rows (a decode step, drafted tokens): at most NR = 16
// or 32 rows (tokens x heads of a key/value head's group) a tile.
//
// Bound by the reads of the cache; the kernel is built around them.  Two threads
// keep the keys and values of NS steps of 128 keys (192 KB of them) on their
// way by TMA, pages of 16 to 128 slots as boxes, across tiles.  The products
// are turned over so that the 128-row side of the tcgen05 tiles holds keys and
// head dimensions, of which there are enough, and the rows are the short side:
//   S^T = K Q^T  (128 keys x NR),   O^T += V^T P^T  (D x NR, V read transposed)
// Thread t of a warpgroup owns key t of a step: NR exponentials a thread, all
// 128 threads at work however few rows there are.  A row's running maximum is
// then shared by the whole warpgroup; it is moved only when some score passes it
// by 2^8 (one vote a step finds out), which is exact, since numerator and
// denominator keep the same one.  Sums stay per thread until the tile's end.
// Two warpgroups take the steps in turn, each with its own maximum, sums, S^T and
// O^T (in TMEM), so that one's softmax runs beside the other's products.  At a
// tile's end they go on with the next, whose scores are there already; a third
// joins the two and writes the tile out, from the one of two sets of O^T that the
// next tile does not use.  In the middle of a batch a step's 64 KB (d 128) take
// 2950 cycles, what HBM gives an SM; the start (lengths, first pages, first
// keys: 7 us) and the joining of cut tiles (3 us) come on top: 64 sequences of 300
// to 3000 tokens, 440 MB, 78 us; 256 of 50 to 600, where a tile has three steps, 80.4 us for 342 MB.
//
// Drafted trees (TREE, an instance of its own: chains keep their code) differ in steps that hold new tokens, or a window's
// border: a thread builds, for its key, the word of rows that see it, from the tokens' masks and positions, which few
// steps of a sequence do.  64 sequences of 300 to 3000 tokens, 8 drafted each, 499 MB: 95 us, as chains of that length.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "device_common.cuh"
#include "internal.h"
#include "paged_common.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace {

__device__ unsigned int g_status_pfew = 0;

using namespace paged;

constexpr uint32_t kChunk = kStep * 128;    // bytes of a 64-column piece of a step's keys or values
constexpr float kNoMax = -1.0e30f;       // running maximum (log2 units) of a row that has seen nothing

template <int D, int NR>
struct FewCfg {
  static constexpr int NCH = D / 64;
  static constexpr uint32_t TILE = NCH * kChunk;       // keys or values of a step
  static constexpr uint32_t QCH = NR * 128;            // a 64-column piece of the queries
  static constexpr uint32_t PT = NR * kStep * 2;          // P^T of a warpgroup: NR rows of two 64-key pieces
  static constexpr uint32_t FIXED = NCH * QCH + 2 * PT + 160 + 192 + NR * 136 + 1024;
  static constexpr int NS_FIT = int((kSmemMax - 1024 - FIXED) / (2 * TILE));
  static constexpr int NS = NS_FIT > 6 ? 6 : NS_FIT;
  // Queries of the next segment beside the present one's, where they fit (not with 32 rows at d 128).
  static constexpr int NQ = FIXED + NCH * QCH + 2 * NS * TILE + 1024 <= kSmemMax ? 2 : 1;
  // The values come first: for d 64 the transposed product reads 128 "dimensions" from each step, the second
  // 64 being whatever follows (the next step's, or the first keys), and their results are not used.
  static constexpr uint32_t OFF_V = 0;
  static constexpr uint32_t OFF_K = OFF_V + NS * TILE;
  static constexpr uint32_t OFF_Q = OFF_K + NS * TILE;
  static constexpr uint32_t OFF_P = OFF_Q + NQ * NCH * QCH;
  static constexpr uint32_t OFF_SCAN = OFF_P + 2 * PT;
  static constexpr uint32_t OFF_SEG = OFF_SCAN + 160;
  static constexpr uint32_t OFF_F = OFF_SEG + 192;     // floats, see below: 34 NR
  // q_full[2], q_empty[2], k_full[NS], k_empty[NS], v_full[NS], v_empty[NS], s_full[2], p_full[2], ml_full[2], ml_free[2],
  // o_final[2], o_free[2], drain, seg_full[4], seg_empty[4]
  static constexpr int NBAR = 4 + 4 * NS + 12 + 1 + 8;
  static constexpr uint32_t OFF_BAR = OFF_F + 34 * NR * 4;
  static constexpr uint32_t OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr uint32_t BYTES = OFF_MISC + 32 + 1024;
  static constexpr uint32_t TMEM_COLS = 8 * NR;  // 2 NR of S^T and 4 NR of O^T, rounded up to a power of two
  // Registers move from the loading, issuing and writing warps to the softmax warpgroups.
  static constexpr int THREADS = 512, REG_LAUNCH = 128, REG_LOW = 88, REG_HIGH = 168;
  static_assert(REG_HIGH * 256 + REG_LOW * 256 <= REG_LAUNCH * 512, "register split");
  static_assert(sizeof(Scan) <= 160 && sizeof(Segment) * 4 <= 192 && NS >= 2 && OFF_BAR % 8 == 0, "layout");
  static_assert(BYTES <= kSmemMax, "shared memory budget");
};

// `or` of a predicate over the 128 threads of warpgroup h
__device__ __forceinline__ bool group_any(int h, bool v) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %2, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, 128, p;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(2 + h), "r"(int(v))
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int h) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(2 + h) : "memory"); }

// NR <= 32 values a lane, reduced over the warp: the lane ends with the result of
// the row that owned_row names, in v[0] (with 16 rows, two lanes hold each).
// Halves the rows with each exchange, so NR + 5 exchanges in place of 5 NR.
template <int NR, class Op>
__device__ __forceinline__ void warp_reduce_rows(float (&v)[NR], int lane, Op op) {
  int n = NR;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < NR / 2; ++i)
        if (i < n) {
          const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
          v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
    } else {
      v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    }
  }
}
// The row that a lane holds after warp_reduce_rows.
template <int NR>
__device__ __forceinline__ int owned_row(int lane) {
  int n = NR, r = 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (n > 1) {
      n >>= 1;
      if (lane & o) r += n;
    }
  return r;
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&r)[N]) {
  static_assert(N == 16 || N == 32, "columns");
  if constexpr (N == 16) tc::tmem_ld16(at, r);
  else tc::tmem_ld32(at, r);
}

template <int D, int NR, bool TREE>
__global__ void __launch_bounds__(512, 1)
    paged_few_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const Params p) {
  using C = FewCfg<D, NR>;
  constexpr int NCH = C::NCH, NS = C::NS, NQ = C::NQ;
  constexpr uint32_t TILE = C::TILE;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sV = smem + C::OFF_V;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sQ = smem + C::OFF_Q;
  Scan* sc = reinterpret_cast<Scan*>(smem + C::OFF_SCAN);
  volatile Segment* seg_ring = reinterpret_cast<volatile Segment*>(smem + C::OFF_SEG);
  float* f_s = reinterpret_cast<float*>(smem + C::OFF_F);
  // handed to the writing warpgroup, by parity of the segment: maxima [2][2][NR], sums [2][2][4 warps][NR]
  float* xm_s = f_s + 12 * NR;
  float* xl_s = f_s + 16 * NR;
  float* coef_s = f_s + 32 * NR;  // [2][NR] what the two O^T are multiplied by
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_empty = q_full + 2;
  uint64_t* k_full = q_full + 4;
  uint64_t* k_empty = k_full + NS;
  uint64_t* v_full = k_empty + NS;
  uint64_t* v_empty = v_full + NS;
  uint64_t* s_full = v_empty + NS;  // [2]
  uint64_t* p_full = s_full + 2;    // [2]
  uint64_t* ml_full = p_full + 2;   // [2]
  uint64_t* ml_free = ml_full + 2;  // [2]
  uint64_t* o_final = ml_free + 2;  // [2]
  uint64_t* o_free = o_final + 2;   // [2]
  uint64_t* drain = o_free + 2;
  uint64_t* seg_full = drain + 1;   // [4]
  uint64_t* seg_empty = drain + 5;  // [4]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  volatile int* dead_s = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 8);  // [3]

  const int warp = threadIdx.x >> 5;
  constexpr int W_K = 8, W_MMA = 9, W_V = 10, W_Q = 11;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NQ; ++s) {
      tc::mbar_init(q_full + s, 1);
      tc::mbar_init(q_empty + s, 1);
    }
    for (int s = 0; s < NS; ++s) {
      tc::mbar_init(k_full + s, 1);
      tc::mbar_init(k_empty + s, 1);
      tc::mbar_init(v_full + s, 1);
      tc::mbar_init(v_empty + s, 1);
    }
    for (int h = 0; h < 2; ++h) {
      tc::mbar_init(s_full + h, 1);
      tc::mbar_init(p_full + h, 128);
      tc::mbar_init(ml_full + h, 256);
      tc::mbar_init(ml_free + h, 128);
      tc::mbar_init(o_final + h, 1);
      tc::mbar_init(o_free + h, 128);
    }
    for (int s = 0; s < 4; ++s) {
      tc::mbar_init(seg_full + s, 1);
      tc::mbar_init(seg_empty + s, 1 + 256 + 128);
    }
    for (int h = 0; h < 3; ++h) dead_s[h] = 0;
    tc::mbar_init(drain, 1);
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (threadIdx.x == 32) {
    tc::tma_prefetch_desc(&tm_k);
    tc::tma_prefetch_desc(&tm_v);
    tc::tma_prefetch_desc(&tm_q);
  }
  // query rows that the loads do not reach are zero: their scores then do not move a maximum
  for (int i = threadIdx.x; i < int(NQ * NCH * C::QCH / 16); i += blockDim.x)
    reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0, 0, 0, 0);
  tc::fence_proxy_async_smem();
  if (warp == W_MMA) tc::tmem_alloc(tmem_slot, C::TMEM_COLS);
  tc::tc_fence_before();
  // From here on memory is read and written that the kernel before may write and read.
  tc::grid_wait_prior();
  tc::grid_launch_dependents();  // the joining kernel waits for this one's end by itself
  const Shares shares = scan_batch<TREE>(p.b, sc, &g_status_pfew);
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;  // columns: S^T of the two warpgroups, then two sets of their O^T
  auto o_col = [](int k, int h) { return uint32_t(2 * NR + ((k & 1) * 2 + h) * NR); };  // of segment k

  if (int(blockIdx.x) >= shares.n) {  // nothing to do here
    if (threadIdx.x == 0) write_split(p, sc, shares, &g_status_pfew);
  } else if (warp >= 8 && warp < 12) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REG_LOW));
  if (warp == W_K || warp == W_V) {
    // ------------------------------------------------------------ producers: one thread for the keys (and the
    // segments that the other roles read), one for the values.  Each walks the steps.  With 16-token pages a
    // step is 16 boxes a side; one thread alone for both took longer to issue them than HBM to deliver.
    const bool keys = warp == W_K;
    if (tc::elect_one()) {
      const CUtensorMap* tm = keys ? &tm_k : &tm_v;
      auto wait1 = [&](uint64_t* b_, uint32_t par) { return tc::mbar_wait(b_, par, abort_flag, &g_status_pfew); };
      LoadRing ring{keys ? k_full : v_full, keys ? k_empty : v_empty, keys ? sK : sV};
      Walk<TREE> w;
      w.start(p.b, sc, shares);
      bool ok = true, more = w.end > w.begin;
      for (int k = 0; ok; ++k) {
        const int n_it = more ? w.end - w.begin : -1;
        const int key0 = (w.t.step0 + w.begin) * kStep;
        if (keys) {
          if (!(ok = wait1(seg_empty + (k & 3), ((k >> 2) & 1) ^ 1))) break;
          volatile Segment* sg = seg_ring + (k & 3);
          sg->n_it = n_it;
          sg->head = w.head;
          sg->first = w.t.first;
          sg->n = w.t.n;
          sg->pos0 = w.t.pos0;
          sg->lo = w.t.lo;
          sg->hi = w.t.hi;
          sg->key0 = key0;
          if (TREE) sg->at = w.i * p.b.tile_tok;
          sg->whole = w.begin == 0 && w.end == w.t.steps;
          sg->slot = blockIdx.x * 2 + (w.begin == 0 ? 1 : 0);
          tc::mbar_arrive(seg_full + (k & 3));
        }
        if (!more) break;
        const int32_t* row = p.b.pages + int64_t(w.seq) * p.b.page_stride;
        const int lo = w.t.lo, hi = w.t.hi, head = w.head;
        ok = load_steps<NS, NCH>(p.b, ring, tm, row, head, key0, n_it, lo, hi, &g_status_pfew, wait1);
        if (ok) more = w.next(p.b);
      }
      if (*abort_flag) {  // let the copies already issued land before the CTA exits
        volatile int never = 0;
        for (int j = (ring.t > NS ? ring.t - NS : 0); j < ring.t; ++j)
          tc::mbar_wait(ring.full + (j % NS), (j / NS) & 1, &never, &g_status_pfew, 100000000ull);
      }
    }
    __syncwarp();
  } else if (warp == W_MMA) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc_s = tc::idesc_bf16(128, NR, false, false);
    constexpr uint32_t idesc_o = tc::idesc_bf16(128, NR, true, false);
    const uint64_t dK = tc::smem_desc(tc::smem_u32(sK), 16, 1024);
    const uint64_t dQ = tc::smem_desc(tc::smem_u32(sQ), 16, 1024);
    const uint64_t dV = tc::smem_desc(tc::smem_u32(sV), kChunk, 1024);
    const uint64_t dP = tc::smem_desc(tc::smem_u32(smem + C::OFF_P), 16, 1024);
    auto issue_s = [&](int h, int s, int qb) {  // S^T_h = K(s) Q^T
      const uint64_t kb = dK + ((s * TILE) >> 4), q = dQ + ((qb * NCH * C::QCH) >> 4);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        tc::mma_ss(tmem + h * NR, kb + (((k >> 2) * kChunk + (k & 3) * 32) >> 4),
                   q + (((k >> 2) * C::QCH + (k & 3) * 32) >> 4), idesc_s, k > 0);
      tc::mma_commit(s_full + h);
    };
    auto issue_o = [&](int k_, int h, int s, bool first) {  // O^T_h (+)= V(s)^T P^T_h
      const uint64_t vb = dV + ((s * TILE) >> 4), pb = dP + ((h * C::PT) >> 4);
#pragma unroll
      for (int k = 0; k < kStep / 16; ++k)
        tc::mma_ss(tmem + o_col(k_, h), vb + ((k * 2048) >> 4),
                   pb + (((k >> 2) * C::QCH + (k & 3) * 32) >> 4), idesc_o, (!first || k > 0) ? 1u : 0u);
    };
    auto wait1 = [&](uint64_t* b_, uint32_t par) { return tc::mbar_wait(b_, par, abort_flag, &g_status_pfew); };
    if (tc::elect_one()) {
      // The scores run two steps ahead of the products with V, over the ends of tiles: a tile of one or two steps
      // would else go all the way from its scores to its products alone.
      int ks = 0, ns = 0, js = 0, ts = 0, qb = 0;  // for the scores: segments begun, steps and step of the last, steps so far
      bool ended = false;
      auto start = [&] {  // S^T of the next step, when its keys are there
        if (ended) return true;
        if (js == ns) {
          if (!wait1(seg_full + (ks & 3), (ks >> 2) & 1)) return false;
          ns = seg_ring[ks & 3].n_it;
          ended = ns < 0;
          if (ended) return true;
          qb = ks % NQ;
          if (!wait1(q_full + qb, (ks / NQ) & 1)) return false;
          js = 0;
          ++ks;
        }
        const int s = ts % NS;
        if (!wait1(k_full + s, (ts / NS) & 1)) return false;
        tc::tc_fence_after();
        issue_s(ts & 1, s, qb);
        tc::mma_commit(k_empty + s);
        if (++js == ns) tc::mma_commit(q_empty + qb);  // the segment's last S^T
        ++ts;
        return true;
      };
      int t = 0;             // steps so far
      int uses[2] = {0, 0};  // steps of each warpgroup so far
      bool ok = start() && start();
      for (int k = 0; ok && t < ts; ++k) {
        const int n_it = seg_ring[k & 3].n_it;
        tc::mbar_arrive(seg_empty + (k & 3));
        for (int j = 0; ok && j < n_it; ++j) {
          const int h = t & 1, s = t % NS;
          if (!(ok = wait1(v_full + s, (t / NS) & 1) && wait1(p_full + h, uses[h] & 1))) break;
          if (j == 0 && !(ok = wait1(o_free + (k & 1), ((k >> 1) & 1) ^ 1))) break;
          ++uses[h];
          tc::tc_fence_after();
          issue_o(k, h, s, j < 2);
          tc::mma_commit(v_empty + s);
          if (j + 1 == n_it) tc::mma_commit(o_final + (k & 1));
          ++t;
          // this warpgroup's S^T was read before the p_full just waited for
          ok = start();
        }
      }
      if (*abort_flag) {  // let issued MMAs finish before TMEM is released
        volatile int never = 0;
        tc::mma_commit(drain);
        tc::mbar_wait(drain, 0, &never, &g_status_pfew, 100000000ull);
      }
    }
    __syncwarp();
  } else if (warp == W_Q) {
    // ------------------------------------------------------------ one thread for the queries of each segment (the
    // thread for the keys would stop at them until the segment before is done)
    if (tc::elect_one()) {
      const uint32_t q_bytes = uint32_t(NCH) * p.b.tile_tok * p.b.group * 128;
      Walk<TREE> w;
      w.start(p.b, sc, shares);
      int nq = 0;
      bool more = w.end > w.begin;
      while (more && tc::mbar_wait(q_empty + nq % NQ, ((nq / NQ) & 1) ^ 1, abort_flag, &g_status_pfew)) {
        const int qb = nq % NQ;
        tc::mbar_arrive_expect_tx(q_full + qb, q_bytes);
        for (int c = 0; c < NCH; ++c)
          tc::tma_load_3d(sQ + (qb * NCH + c) * C::QCH, &tm_q, q_full + qb, c * 64, w.head * p.b.group, w.t.first);
        if (nq++ == 0) write_split(p, sc, shares, &g_status_pfew);
        more = w.next(p.b);
      }
      if (*abort_flag) {
        volatile int never = 0;
        for (int j = (nq > NQ ? nq - NQ : 0); j < nq; ++j)
          tc::mbar_wait(q_full + j % NQ, (j / NQ) & 1, &never, &g_status_pfew, 100000000ull);
      }
    }
    __syncwarp();
  }
  } else if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REG_HIGH));
    // ------------------------------------------------------------ softmax of every other step
    const int h = warp >> 2, lane = threadIdx.x & 31;
    const int r = threadIdx.x & 127;  // key of the step, then head dimension = TMEM lane
    const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + h * NR;
    uint8_t* sP = smem + C::OFF_P + h * C::PT + (r >> 6) * C::QCH + (r & 7) * 2;
    const uint32_t p_chunk = (r >> 3) & 7;  // of the 128-byte piece of a row
    float* m_s = f_s + h * NR;                  // running maxima
    float* warp_s = f_s + 2 * NR + h * 4 * NR;  // the four warps' maxima
    float* alpha_s = f_s + 10 * NR + h * NR;    // rescaling
    auto wait_thread = [&](uint64_t* b_, uint32_t par) { return tc::mbar_wait(b_, par, abort_flag, &g_status_pfew); };
    // The warps of a warpgroup meet in barriers, so they leave together or not at all: a failed wait is passed on
    // through dead_s at the next vote.
    bool fine = true;
    auto note = [&](bool ok) {
      if (!ok) {
        fine = false;
        dead_s[h] = 1;
      }
    };
    int t = 0, uses = 0;
    for (int k = 0;; ++k) {
      note(wait_thread(seg_full + (k & 3), (k >> 2) & 1));
      if (group_any(h, !fine)) break;
      const volatile Segment* sg = seg_ring + (k & 3);
      const int n_it = sg->n_it, n_tok = sg->n, lo = sg->lo, hi = sg->hi, key_first = sg->key0, pos_first = sg->pos0;
      const int row_first = TREE ? sg->first : 0, at_first = TREE ? sg->at : 0;
      tc::mbar_arrive(seg_empty + (k & 3));
      if (n_it < 0) break;
      const uint32_t tO = tmem + lane_base + o_col(k, h);
      // every row in use sees the keys in [all_lo, all_hi)
      const int base = pos_first - at_first;  // (TREE) the sequence's tokens before its tree
      const int all_hi = TREE ? base : pos_first + 1;
      const int all_lo = p.b.window > 0 ? pos_first + n_tok - p.b.window : 0;
      // Rows behind the tile's own (the load brings the next sequence's queries, or padding) never pass an infinite
      // maximum, so they have no say in when the others' are moved, and no bit of those depends on what they hold.  Their
      // own sums may then be no numbers; nobody reads them.
      const float floor_r = r < n_tok * p.b.group ? kNoMax : INFINITY;
      float l[NR];
#pragma unroll
      for (int i = 0; i < NR; ++i) l[i] = 0.f;
      bool dead = false;
      const int j0 = (t ^ h) & 1;  // this warpgroup's first step: the two take all steps in turn
      for (int j = j0; j < n_it; j += 2) {
        const int key0 = key_first + j * kStep;
        note(wait_thread(s_full + h, uses & 1));
        ++uses;
        if (key0 < lo || key0 + kStep > hi) {
          // slots that no row sees may hold anything: zero their values, so that 0 x NaN does not come in.  This S^T
          // was issued behind the products with V of every step up to j - 2, so those V have landed and the wait can
          // only end with this step's; before S^T, the stage's last V could still be under way, whose end has the
          // parity that a wait for this one takes for its own.
          static_assert(NS >= 2, "the stage's last V is of a step before j - 1");
          const int s = (t + j) % NS;
          const bool there = wait_thread(v_full + s, ((t + j) / NS) & 1);
          note(there);
          if (there && fine) {
            const int head_rows = min(max(lo - key0, 0), kStep), live_rows = min(max(hi - key0, 0), kStep);
#pragma unroll
            for (int c = 0; c < NCH; ++c) {
              uint4* v = reinterpret_cast<uint4*>(sV + s * TILE + c * kChunk);
              for (int i = r; i < head_rows * 8; i += 128) v[i] = make_uint4(0, 0, 0, 0);
              for (int i = live_rows * 8 + r; i < kStep * 8; i += 128) v[i] = make_uint4(0, 0, 0, 0);
            }
          }
        }
        __syncwarp();
        tc::tc_fence_after();
        uint32_t raw[NR];
        tmem_ld(tS, raw);
        tc::tmem_ld_wait();
        float x[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) x[i] = __uint_as_float(raw[i]) * p.scale_log2;
        if (key0 + kStep > all_hi || key0 < all_lo) {
          if constexpr (TREE) {
            // the rows that see this thread's key, a bit each
            const int key = key0 + r, drafted = key - base;
            const uint32_t heads = p.b.group < 32 ? (1u << p.b.group) - 1 : ~0u;
            uint32_t rows = 0;
            if (key < hi)
              for (int t_ = 0; t_ < n_tok; ++t_) {
                bool sees;
                if (drafted < 0)
                  sees = p.b.window == 0 || key > tree_position(p.b, row_first + t_, base, at_first + t_) - p.b.window;
                else
                  sees = drafted <= at_first + t_ &&
                         (p.b.masks[int64_t(row_first + t_) * p.b.mask_words + (drafted >> 5)] >> (drafted & 31) & 1);
                if (sees) rows |= heads << (t_ * p.b.group);
              }
#pragma unroll
            for (int i = 0; i < NR; ++i)
              if (!(rows >> i & 1)) x[i] = -INFINITY;
          } else {
          // rows [first_row, last_row) see this thread's key
          const int rel = key0 + r - pos_first;
          int first_row = max(rel, 0) * p.b.group, last_row = NR;
          if (p.b.window > 0) last_row = min(max(rel + p.b.window, 0), NR) * p.b.group;
          if (key0 + r >= hi) last_row = 0;
#pragma unroll
          for (int i = 0; i < NR; ++i)
            if (i < first_row || i >= last_row) x[i] = -INFINITY;
          }
        }
        bool grow = j == j0;
#pragma unroll
        for (int i = 0; i < NR; i += 4) {
          const float4 m = *reinterpret_cast<const float4*>(m_s + i);
          grow |= x[i] > m.x + kRescale || x[i + 1] > m.y + kRescale || x[i + 2] > m.z + kRescale ||
                  x[i + 3] > m.w + kRescale;
        }
        if (group_any(h, grow || !fine)) {
          if (dead_s[h]) {
            dead = true;
            break;
          }
          float v[NR];
#pragma unroll
          for (int i = 0; i < NR; ++i) v[i] = x[i];
          warp_reduce_rows<NR>(v, lane, [](float a, float b) { return fmaxf(a, b); });
          warp_s[(warp & 3) * NR + owned_row<NR>(lane)] = v[0];
          group_sync(h);
          if (r < NR) {
            const float before = j == j0 ? floor_r : m_s[r];
            const float top = fmaxf(fmaxf(warp_s[r], warp_s[NR + r]), fmaxf(warp_s[2 * NR + r], warp_s[3 * NR + r]));
            const float m = fmaxf(before, top);
            m_s[r] = m;
            alpha_s[r] = tc::ex2(before - m);
          }
          group_sync(h);
          if (j != j0) {
#pragma unroll
            for (int i = 0; i < NR; ++i) l[i] *= alpha_s[i];
            // O^T of this warpgroup is complete up to its step before: that product was issued before this S^T
            uint32_t ov[NR];
            tmem_ld(tO, ov);
            tc::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < NR; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha_s[i]);
#pragma unroll
            for (int c = 0; c < NR / 16; ++c)
              tc::tmem_st16(tO + c * 16, *reinterpret_cast<const uint32_t(*)[16]>(ov + c * 16));
            tc::tmem_st_wait();
          }
        }
#pragma unroll
        for (int i = 0; i < NR; i += 4) {
          const float4 m = *reinterpret_cast<const float4*>(m_s + i);
          const float mm[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float e = tc::ex2(x[i + u] - mm[u]);
            l[i + u] += e;
            // P^T enters the second product as bf16, its operand type; row i + u, key r
            *reinterpret_cast<__nv_bfloat16*>(sP + (i + u) * 128 + ((p_chunk ^ ((i + u) & 7)) << 4)) =
                __float2bfloat16_rn(e);
          }
        }
        tc::fence_proxy_async_smem();
        tc::tc_fence_before();
        tc::mbar_arrive(p_full + h);
      }
      if (dead) break;

      // -------- the tile's end: the maxima and this warp's sums go to the writing warpgroup
      warp_reduce_rows<NR>(l, lane, [](float a, float b) { return a + b; });
      note(wait_thread(ml_free + (k & 1), ((k >> 1) & 1) ^ 1));
      if (fine) {
        float* xm = xm_s + (k & 1) * 2 * NR + h * NR;
        float* xl = xl_s + (k & 1) * 8 * NR + (h * 4 + (warp & 3)) * NR;
        xl[owned_row<NR>(lane)] = l[0];
        if (r < NR) xm[r] = j0 < n_it ? m_s[r] : kNoMax;  // (a warpgroup without a step has no maxima)
      }
      tc::mbar_arrive(ml_full + (k & 1));
      t += n_it;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REG_LOW));
    // ------------------------------------------------------------ the tile's end: the two O^T joined and written
    const int r = threadIdx.x & 127;  // head dimension = TMEM lane, and row of the coefficients
    const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
    bool fine = true;
    auto note = [&](bool ok) {
      if (!ok) {
        fine = false;
        dead_s[2] = 1;
      }
    };
    auto wait_thread = [&](uint64_t* b_, uint32_t par) { return tc::mbar_wait(b_, par, abort_flag, &g_status_pfew); };
    int t = 0;
    for (int k = 0;; ++k) {
      note(wait_thread(seg_full + (k & 3), (k >> 2) & 1));
      if (group_any(2, !fine)) break;
      const volatile Segment* sg = seg_ring + (k & 3);
      const int n_it = sg->n_it, first = sg->first, live = sg->n * p.b.group;
      const int slot = sg->whole ? -1 : sg->slot, head0 = sg->head * p.b.group;
      tc::mbar_arrive(seg_empty + (k & 3));
      if (n_it < 0) break;
      note(wait_thread(ml_full + (k & 1), (k >> 1) & 1));
      note(wait_thread(o_final + (k & 1), (k >> 1) & 1));
      // (of the tile's own rows: the quotient of a sum that is no number takes a long way, 5 us for 256 short sequences)
      if (r < live && fine) {
        const float* xm = xm_s + (k & 1) * 2 * NR;
        const float* xl = xl_s + (k & 1) * 8 * NR;
        const float m0 = xm[r], m1 = xm[NR + r];
        const float l0 = (xl[r] + xl[NR + r]) + (xl[2 * NR + r] + xl[3 * NR + r]);
        const float l1 = (xl[4 * NR + r] + xl[5 * NR + r]) + (xl[6 * NR + r] + xl[7 * NR + r]);
        const float top = fmaxf(m0, m1);
        float a0 = tc::ex2(m0 - top), a1 = tc::ex2(m1 - top);
        const float sum = l0 * a0 + l1 * a1;
        if (slot < 0) {
          const float inv = sum > 0.f ? 1.f / sum : 0.f;
          a0 *= inv;
          a1 *= inv;
        }
        coef_s[r] = a0;
        coef_s[NR + r] = a1;
        if (slot < 0) {
          const int tok = r / p.b.group;
          p.lse[int64_t(first + tok) * p.hq + head0 + r - tok * p.b.group] =
              sum > 0.f ? (top + __log2f(sum)) * kLn2 : -INFINITY;
        } else {
          p.part_ml[int64_t(slot) * p.rows + r] = make_float2(top, sum);
        }
      }
      if (group_any(2, !fine)) break;  // (the coefficients are there)
      tc::tc_fence_after();
      // with one step, one of the two O^T was not written
      const bool has0 = n_it > 1 || (t & 1) == 0, has1 = n_it > 1 || (t & 1) == 1;
      int tok = 0, gh = 0;
#pragma unroll
      for (int c = 0; c < NR; c += 16) {
        uint32_t x[16], y[16];
        tc::tmem_ld16(tmem + lane_base + o_col(k, 0) + c, x);
        tc::tmem_ld16(tmem + lane_base + o_col(k, 1) + c, y);
        tc::tmem_ld_wait();
        if (c + 16 == NR) {  // the segment after next may have the maxima's, sums' and O^T's places
          tc::tc_fence_before();
          tc::mbar_arrive(ml_free + (k & 1));
          tc::mbar_arrive(o_free + (k & 1));
        }
        if (r < D) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (c + i < live) {
              float v = has0 ? __uint_as_float(x[i]) * coef_s[c + i] : 0.f;
              if (has1) v = fmaf(__uint_as_float(y[i]), coef_s[NR + c + i], v);
              if (slot < 0)
                p.o[(int64_t(first + tok) * p.hq + head0 + gh) * D + r] = __float2bfloat16_rn(v);
              else
                p.part_o[(int64_t(slot) * p.rows + c + i) * D + r] = v;
              if (++gh == p.b.group) {
                gh = 0;
                ++tok;
              }
            }
          }
        }
      }
      t += n_it;
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == W_MMA) tc::tmem_dealloc(tmem, C::TMEM_COLS);
}

template <int D, int NR, bool TREE>
int launch_few(const tpa_paged_view* c, Params& p, int grid, cudaStream_t st) {
  using C = FewCfg<D, NR>;
  CUtensorMap tq, tk, tv;
  p.b.tile_tok = NR / p.b.group;
  const uint64_t rows = uint64_t(c->n_pages) * c->n_heads_kv * c->page_size;
  if (!query_map(&tq, c, p, p.b.tile_tok) || !cache_map(&tk, c->k_cache, rows, D, c->page_size) ||
      !cache_map(&tv, c->v_cache, rows, D, c->page_size))
    return TPA_ERR_CUDA;
  TPA_CUDA_TRY(cudaFuncSetAttribute(paged_few_kernel<D, NR, TREE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES));
  cudaFuncAttributes fa;
  TPA_CUDA_TRY(cudaFuncGetAttributes(&fa, paged_few_kernel<D, NR, TREE>));
  if (fa.numRegs != C::REG_LAUNCH) return TPA_ERR_BAD_BUILD;  // the setmaxnreg split would not add up
  return launch_overlapped(paged_few_kernel<D, NR, TREE>, dim3(grid), C::THREADS, C::BYTES, st, tq, tk, tv,
                           static_cast<const Params>(p));
}

}  // namespace

TPA_DEFINE_STATUS_READER(tpa_internal_status_pfew, g_status_pfew)

int tpa_internal_paged_few(const tpa_paged_view* c, Params& p, int rows, int grid, cudaStream_t st) {
  auto launch = [&](auto d, auto nr) {
    constexpr int D = decltype(d)::value, NR = decltype(nr)::value;
    return p.b.masks ? launch_few<D, NR, true>(c, p, grid, st) : launch_few<D, NR, false>(c, p, grid, st);
  };
  using std::integral_constant;
  if (c->head_dim == 128)
    return rows == 16 ? launch(integral_constant<int, 128>(), integral_constant<int, 16>())
                      : launch(integral_constant<int, 128>(), integral_constant<int, 32>());
  return rows == 16 ? launch(integral_constant<int, 64>(), integral_constant<int, 16>())
                    : launch(integral_constant<int, 64>(), integral_constant<int, 32>());
}
