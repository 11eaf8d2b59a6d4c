// What the paged attention kernels share: a batch's tiles (runs of one
// sequence's new tokens with one key/value head's queries), how their steps of
// 128 keys are dealt to the CTAs, and the record of a tile whose steps went to
// several CTAs.
//
// The steps of all tiles stand in one line, key/value head by head, sequence by
// sequence, tile by tile, and CTA c of n takes the part [c T / n, (c + 1) T / n)
// of its T steps: every CTA has the same work whatever the lengths, a long
// sequence is split along its keys by as much as that needs, and a CTA has at
// most two tiles that it shares with others (its first and its last).  The
// lengths are read from device memory by every CTA (a scan over the
// sequences), so nothing of the partition is computed on the host.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "device_common.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace paged {

constexpr uint32_t kSmemMax = 232448;  // 227 KB opt-in per CTA
constexpr int kMaxGrid = 160;  // CTAs of a launch, at most (one an SM)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kStepShift = 7, kStep = 1 << kStepShift;  // keys of a step
constexpr float kRescale = 8.0f;  // log2 units: the running maximum is kept while the new one is not this much larger

struct Batch {
  const int32_t* pages;
  const int32_t* offsets;
  const int32_t* kv_lens;
  int32_t n_pages, page_shift, n_seqs, max_pages, page_stride, hkv, n_rows;
  int32_t group;     // query heads of a key/value head
  int32_t tile_tok;  // tokens of a tile
  int32_t window;    // 0: none
};

struct Seq {
  int first, n, kv;  // first row, new tokens, cached tokens
};

// A sequence whose numbers are out of range has no tokens (and is reported).
__device__ __forceinline__ Seq load_seq(const Batch& b, int s, unsigned int* status) {
  const int o0 = __ldg(b.offsets + s), o1 = __ldg(b.offsets + s + 1), kv = __ldg(b.kv_lens + s);
  if (o0 < 0 || o1 < o0 || o1 > b.n_rows || kv < 0 || kv > (int64_t(b.max_pages) << b.page_shift)) {
    if (status) atomicOr(status, TPA_DEV_BAD_INPUT);
    return Seq{0, 0, 0};
  }
  return Seq{o0, o1 - o0, kv};
}

// Tile i of a sequence: n tokens from row `first`, the first of them at
// position pos0 (negative where there are more new tokens than cached ones).
// Keys outside [lo, hi) are seen by none of its tokens; those from hi to `end`,
// the sequence's cached tokens, by later ones.  At least one step, so that a tile
// that sees nothing still has its rows written.
struct Tile {
  int first, n, pos0, lo, hi, end, step0, steps;
};

__device__ __forceinline__ int tiles_of(const Batch& b, int n) { return (n + b.tile_tok - 1) / b.tile_tok; }

__device__ __forceinline__ Tile make_tile(const Batch& b, const Seq& q, int i) {
  Tile t;
  const int t0 = i * b.tile_tok;
  t.first = q.first + t0;
  t.n = min(b.tile_tok, q.n - t0);
  t.pos0 = q.kv - q.n + t0;
  t.hi = max(t.pos0 + t.n, 0);
  t.end = q.kv;
  t.lo = b.window > 0 ? max(t.pos0 - b.window + 1, 0) : 0;
  t.step0 = t.lo >> kStepShift;
  t.steps = max(((t.hi + kStep - 1) >> kStepShift) - t.step0, 1);
  return t;
}

// Quotient below 2^20.  Integer division is a long chain of dependent
// instructions, and every CTA's first load waits for three of them.
__device__ __forceinline__ int small_quot(long long a, long long b) {
  if (((a | b) >> 31) != 0) return int(a / b);
  int q = int(__fdividef(float(int(a)), float(int(b))));  // off by one at most
  const int r = int(uint32_t(a) - uint32_t(q) * uint32_t(b));  // in [-b, 2 b), whatever q * b passes
  if (r < 0) --q;
  else if (r >= int(b)) ++q;
  return q;
}

// How the CTAs share `total` steps: n of them, the first `rem` with size + 1 and the others with `size`.
struct Shares {
  int n;
  long long size, rem;
  __device__ __forceinline__ Shares(long long total, int grid) {
    n = int(total < grid ? total : grid);
    if (total < grid) {
      size = 1;
    } else if ((total >> 20) == 0) {
      size = small_quot(total, grid);
    } else {
      size = total / grid;
    }
    rem = total - size * n;
  }
  __device__ __forceinline__ long long begin(int c) const { return size * c + (c < rem ? c : rem); }
  __device__ __forceinline__ int of(long long f) const {
    const long long edge = rem * (size + 1);
    return f < edge ? small_quot(f, size + 1) : int(rem) + small_quot(f - edge, size);
  }
};

// What the scan finds out: the sums of its warps, and where this CTA begins.
struct Scan {
  long long warp_sum[8];
  long long item;            // flat step at which the first tile begins
  int head, seq, i, begin;   // key/value head, sequence, tile of it, step of the tile
  int n_tiles;
  Seq q;
  Tile t;
};

// Every thread of the CTA (256 of them or more; the first 256 work, a share of
// the sequences each): adds up the steps and finds this CTA's first one; the
// thread that has it among its sequences writes it down.  Reports bad
// sequences once (CTA 0).
__device__ inline Shares scan_batch(const Batch& b, Scan* sc, unsigned int* status) {
  const int tid = threadIdx.x, chunk = (b.n_seqs + 255) >> 8;
  const int s0 = tid * chunk, s1 = min(s0 + chunk, b.n_seqs);
  long long mine = 0, incl = 0;
  Seq q{0, 0, 0};
  if (tid < 256) {
    for (int s = s0; s < s1; ++s) {
      q = load_seq(b, s, blockIdx.x == 0 ? status : nullptr);
      const int n = tiles_of(b, q.n);
      for (int i = 0; i < n; ++i) mine += make_tile(b, q, i).steps;
    }
    incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if ((tid & 31) >= o) incl += v;
    }
    if ((tid & 31) == 31) sc->warp_sum[tid >> 5] = incl;
  }
  __syncthreads();
  long long per_head = 0, before = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    if (w < (tid >> 5)) before += sc->warp_sum[w];
    per_head += sc->warp_sum[w];
  }
  const Shares shares(per_head * b.hkv, gridDim.x);
  if (int(blockIdx.x) < shares.n) {
    const long long f = shares.begin(blockIdx.x), head = small_quot(f, per_head);
    long long r = f - head * per_head - (before + incl - mine);  // step among this thread's sequences
    if (tid < 256 && r >= 0 && r < mine) {
      for (int s = s0; s < s1; ++s) {
        if (chunk > 1) q = load_seq(b, s, nullptr);
        const int n = tiles_of(b, q.n);
        for (int i = 0; i < n; ++i) {
          const Tile t = make_tile(b, q, i);
          const int steps = t.steps;
          if (r >= 0 && r < steps) {
            // the page table's row is about to be read
            asm volatile("prefetch.global.L1 [%0];" ::"l"(b.pages + int64_t(s) * b.page_stride +
                                                          min(((t.step0 + int(r)) << kStepShift) >> b.page_shift, b.max_pages - 1)));
            sc->t = t;
            sc->n_tiles = n;
            sc->item = f - r;
            sc->head = int(head);
            sc->seq = s;
            sc->i = i;
            sc->begin = int(r);
            sc->q = q;
          }
          r -= steps;
        }
      }
    }
  }
  __syncthreads();
  return shares;
}

// Walks the tiles of this CTA's steps.
struct Walk {
  long long left;     // steps from `begin` of the current tile on
  int head, seq, i;   // key/value head, sequence, tile of the sequence
  int n_tiles;
  Seq q;
  Tile t;
  int begin, end;     // this CTA's steps of the tile

  __device__ __forceinline__ void take() {
    const long long e = begin + left;
    end = e < t.steps ? int(e) : t.steps;
  }
  __device__ inline void start(const Batch& b, const Scan* sc, const Shares& shares) {
    left = shares.size + (int(blockIdx.x) < shares.rem ? 1 : 0);
    head = sc->head;
    seq = sc->seq;
    i = sc->i;
    begin = sc->begin;
    q = sc->q;
    n_tiles = sc->n_tiles;
    t = sc->t;
    take();
  }
  // To the next tile; false when this CTA's steps are done.
  __device__ inline bool next(const Batch& b) {
    left -= end - begin;
    if (left <= 0) return false;
    if (++i >= n_tiles) {
      i = 0;
      int tries = 0;
      do {
        if (++seq >= b.n_seqs) {
          seq = 0;
          ++head;
        }
        q = load_seq(b, seq, nullptr);
        n_tiles = tiles_of(b, q.n);
      } while (n_tiles == 0 && ++tries <= b.n_seqs);
      if (n_tiles == 0 || head >= b.hkv) return false;  // not reached with the lengths that were scanned
    }
    t = make_tile(b, q, i);
    begin = 0;
    take();
    return true;
  }
};

// A tile whose steps went to the CTAs c0 .. c1, written by CTA c0 + 1.  Its
// part from CTA c0 is in that CTA's slot 1, the others' parts in their slot 0.
struct Split {
  int32_t valid, head, first, n, c0, c1, pad_[2];
};

struct Params {
  Batch b;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  float* part_o;    // [2 grid][R][D]: sums relative to the row's own maximum
  float2* part_ml;  // [2 grid][R]: maximum (log2 units) and sum
  Split* split;     // [grid]
  int64_t q_stride;
  int32_t hq, rows;  // rows: R, of a part
  float scale_log2;
};

// 2-D tiled load: a box of 64 columns into 128-byte swizzled rows
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(tc::smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}

// One CTA's part of a tile, as the producer hands it to the other roles.
struct Segment {
  int32_t n_it;  // steps; -1: no more
  int32_t head, first, n, pos0, lo, hi, key0, whole, slot;
  int32_t pad_[2];
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// O (+)= P V with P read from TMEM
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Writes the record of the tile that this CTA's first segment is a part of: one thread of each CTA, behind its first
// loads.  Rows before the first sequence are reported here, where nothing waits for it.
__device__ __forceinline__ void write_split(const Params& p, const Scan* sc, const Shares& sh, unsigned int* status) {
  if (blockIdx.x == 0 && __ldg(p.b.offsets) != 0) atomicOr(status, TPA_DEV_BAD_INPUT);
  Split s = {};
  if (int(blockIdx.x) < sh.n && sc->begin > 0) {  // the tile began in an earlier CTA
    const Tile t = sc->t;
    const int c0 = sh.of(sc->item), c1 = sh.of(sc->item + t.steps - 1);
    if (c0 + 1 == int(blockIdx.x)) s = Split{1, sc->head, t.first, t.n, c0, c1, {0, 0}};
  }
  p.split[blockIdx.x] = s;
}

// The ring of stages that one thread fills with the keys (or the values) of this CTA's steps.
struct LoadRing {
  uint64_t* full;
  uint64_t* empty;
  uint8_t* tiles;
  int t = 0, s = 0;  // steps loaded, the next stage
  uint32_t par = 1;  // and the parity of its `empty`
};

// Loads steps [0, n_it) of a segment from key0 on, the pages that hold keys of [lo, hi) of them: a page
// is a box for each 64 columns.  Unrolled for the number of pages of a step.  The entries of the page table come from
// L1, a line of them fetched ahead.  False when a wait gave up.
template <int NS, int NCH, class Wait>
__device__ __forceinline__ bool load_steps(const Batch& b, LoadRing& ring, const CUtensorMap* tm, const int32_t* row,
                                           int head, int key0, int n_it, int lo, int hi, unsigned int* status, Wait wait1) {
  auto load_step = [&](int j, auto n_pages) {
    constexpr int N = decltype(n_pages)::value;
    int at[N];  // first cache row of each page that is needed
    uint32_t needed = 0;
    const int first_page = (key0 + j * kStep) >> b.page_shift;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int ki = key0 + j * kStep + i * (kStep / N);
      const bool need = ki < hi && ki + kStep / N > lo;
      at[i] = need ? __ldg(row + first_page + i) : 0;
      needed |= uint32_t(need) << i;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (uint32_t(at[i]) >= uint32_t(b.n_pages)) {  // never followed: page 0 is read in its place
        atomicOr(status, TPA_DEV_BAD_INPUT);
        at[i] = 0;
      }
      at[i] = (at[i] * b.hkv + head) * (kStep / N);
    }
    if (!wait1(ring.empty + ring.s, ring.par)) return false;
    constexpr uint32_t kBytes = 128 * (kStep / N);  // a 64-column piece of a page
    tc::mbar_arrive_expect_tx(ring.full + ring.s, __popc(needed) * NCH * kBytes);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (needed >> i & 1)
#pragma unroll
        for (int c = 0; c < NCH; ++c)
          tma_load_2d(ring.tiles + ring.s * (NCH * kStep * 128) + c * (kStep * 128) + i * kBytes, tm, ring.full + ring.s, c * 64,
                      at[i]);
    if (first_page + 32 < b.max_pages) asm volatile("prefetch.global.L1 [%0];" ::"l"(row + first_page + 32));
    ++ring.t;
    if (++ring.s == NS) {
      ring.s = 0;
      ring.par ^= 1;
    }
    return true;
  };
  auto all = [&](auto n_pages) {
    bool ok = true;
    for (int j = 0; ok && j < n_it; ++j) ok = load_step(j, n_pages);
    return ok;
  };
  switch (kStep >> b.page_shift) {
    case 1: return all(std::integral_constant<int, 1>());
    case 2: return all(std::integral_constant<int, 2>());
    case 4: return all(std::integral_constant<int, 4>());
    default: return all(std::integral_constant<int, 8>());
  }
}

// Launches a kernel that may begin while the one before it in the stream ends;
// it waits for that one itself (tc::grid_wait_prior) before it touches memory.
template <class... Args>
inline int launch_overlapped(void (*kernel)(Args...), dim3 grid, int threads, uint32_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  TPA_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, args...));
  return TPA_OK;
}

// Cache rows as a matrix [n_pages * Hkv * page_size, d]: boxes of 64 columns x `rows` rows.
inline bool cache_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t d, uint32_t box_rows) {
  tmap::EncodeTiledFn fn = tmap::encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {d, rows};
  const cuuint64_t strides[1] = {d * 2};
  const cuuint32_t box[2] = {64, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries [n_rows, Hq, d]: boxes of 64 columns x the group's heads x a sub-tile's tokens.
inline bool query_map(CUtensorMap* m, const tpa_paged_view* c, const Params& p, int sub_tok) {
  tmap::EncodeTiledFn fn = tmap::encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cuuint64_t(c->head_dim), cuuint64_t(p.hq), cuuint64_t(c->n_rows)};
  const cuuint64_t strides[2] = {cuuint64_t(c->head_dim) * 2, cuuint64_t(p.q_stride) * 2};
  const cuuint32_t box[3] = {64, cuuint32_t(p.b.group), cuuint32_t(sub_tok)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(p.q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace paged

// Launch the attention kernel (the caller joins split tiles afterwards): for
// tiles of `rows` = 16 or 32 rows (paged_few.cu), and of 256 (paged_tile.cu).
// Either may find that it was not compiled with the registers that its warps
// divide up; it then launches nothing (TPA_ERR_BAD_BUILD).
int tpa_internal_paged_few(const tpa_paged_view* cache, paged::Params& p, int rows, int grid, cudaStream_t stream);
int tpa_internal_paged_tile(const tpa_paged_view* cache, paged::Params& p, int grid, cudaStream_t stream);
