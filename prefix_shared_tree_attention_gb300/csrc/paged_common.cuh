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

#include "device_common.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace paged {

constexpr int kStep = 128;     // keys of a step
constexpr uint32_t kSmemMax = 232448;  // 227 KB opt-in per CTA
constexpr int kMaxGrid = 160;  // CTAs of a launch, at most (one an SM)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;  // log2 units: the running maximum is kept while the new one is not this much larger

struct Batch {
  const int32_t* pages;
  const int32_t* offsets;
  const int32_t* kv_lens;
  int32_t n_pages, page_size, page_shift, n_seqs, max_pages, page_stride, hkv, n_rows;
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
// Keys outside [lo, hi) are seen by none of its tokens.  At least one step, so
// that a tile that sees nothing still has its rows written.
struct Tile {
  int first, n, pos0, lo, hi, step0, steps;
};

__device__ __forceinline__ int tiles_of(const Batch& b, int n) { return (n + b.tile_tok - 1) / b.tile_tok; }

__device__ __forceinline__ Tile make_tile(const Batch& b, const Seq& q, int i) {
  Tile t;
  const int t0 = i * b.tile_tok;
  t.first = q.first + t0;
  t.n = min(b.tile_tok, q.n - t0);
  t.pos0 = q.kv - q.n + t0;
  t.hi = max(t.pos0 + t.n, 0);
  t.lo = b.window > 0 ? max(t.pos0 - b.window + 1, 0) : 0;
  t.step0 = t.lo / kStep;
  t.steps = max((t.hi + kStep - 1) / kStep - t.step0, 1);
  return t;
}

struct Scan {
  long long prefix[257];  // steps of one head before the chunk of sequences of each thread
};

// Every thread of the CTA (256 of them or more; the first 256 work): fills the
// scan, returns the steps of one head.  Reports bad sequences once (CTA 0).
__device__ inline long long scan_batch(const Batch& b, Scan* sc, unsigned int* status) {
  const int tid = threadIdx.x, chunk = (b.n_seqs + 255) >> 8;
  if (tid < 256) {
    long long mine = 0;
    const int s1 = min((tid + 1) * chunk, b.n_seqs);
    for (int s = tid * chunk; s < s1; ++s) {
      const Seq q = load_seq(b, s, blockIdx.x == 0 ? status : nullptr);
      const int n = tiles_of(b, q.n);
      for (int i = 0; i < n; ++i) mine += make_tile(b, q, i).steps;
    }
    long long v = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, v, o);
      if ((tid & 31) >= o) v += t;
    }
    sc->prefix[tid + 1] = v;
  }
  __syncthreads();
  if (tid < 256) {
    long long before = 0;
    for (int w = 0; w < (tid >> 5); ++w) before += sc->prefix[(w + 1) * 32];
    const long long v = sc->prefix[tid + 1];
    __syncwarp();
    // all warps have read the warp totals before any overwrites them
    asm volatile("bar.sync 1, 256;" ::: "memory");
    sc->prefix[tid + 1] = before + v;
    if (tid == 0) sc->prefix[0] = 0;
  }
  __syncthreads();
  return sc->prefix[256];
}

// How many CTAs share `total` steps, and the first step of CTA c.
__device__ __forceinline__ int used_ctas(long long total, int grid, int min_steps) {
  const long long want = (total + min_steps - 1) / min_steps;
  return int(want < grid ? want : grid);
}
__device__ __forceinline__ long long cta_begin(long long total, int n, int c) { return total * c / n; }
__device__ __forceinline__ int cta_of(long long total, int n, long long f) { return int(((f + 1) * n - 1) / total); }

// Walks the tiles of the steps [f, f + left).
struct Walk {
  long long left;     // steps from `begin` of the current tile on
  long long item;     // flat step at which the current tile begins
  int head, seq, i;   // key/value head, sequence, tile of the sequence
  int n_tiles;
  Seq q;
  Tile t;
  int begin, end;     // this CTA's steps of the tile

  __device__ __forceinline__ void take() {
    const long long e = begin + left;
    end = e < t.steps ? int(e) : t.steps;
  }
  // f < total
  __device__ inline void start(const Batch& b, const Scan* sc, long long per_head, long long f, long long count) {
    left = count;
    head = int(f / per_head);
    long long r = f - head * per_head;
    int lo = 0, hi = 256;  // the last chunk that begins at r or before
    while (hi - lo > 1) {
      const int m = (lo + hi) >> 1;
      if (sc->prefix[m] <= r) lo = m;
      else hi = m;
    }
    const int chunk = (b.n_seqs + 255) >> 8;
    long long at = sc->prefix[lo];
    for (seq = lo * chunk;; ++seq) {  // ends: the chunk holds step r
      q = load_seq(b, seq, nullptr);
      n_tiles = tiles_of(b, q.n);
      for (i = 0; i < n_tiles; ++i) {
        t = make_tile(b, q, i);
        if (at + t.steps > r) {
          begin = int(r - at);
          item = f - begin;
          take();
          return;
        }
        at += t.steps;
      }
      if (seq + 1 >= b.n_seqs) {  // not reached with the lengths that were scanned
        left = 0;
        begin = end = 0;
        return;
      }
    }
  }
  // To the next tile; false when this CTA's steps are done.
  __device__ inline bool next(const Batch& b) {
    left -= end - begin;
    if (left <= 0) return false;
    item += t.steps;
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
  int32_t hq, min_steps, rows;  // rows: R, of a part
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

// Writes the record of the tile that this CTA's first segment is a part of.
__device__ __forceinline__ void write_split(const Params& p, const Walk& w, long long total, int n_ctas) {
  Split s = {};
  if (w.begin > 0) {  // the tile began in an earlier CTA
    const int c0 = cta_of(total, n_ctas, w.item), c1 = cta_of(total, n_ctas, w.item + w.t.steps - 1);
    if (c0 + 1 == int(blockIdx.x)) s = Split{1, w.head, w.t.first, w.t.n, c0, c1, {0, 0}};
  }
  p.split[blockIdx.x] = s;
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

}  // namespace paged

// paged_tile.cu: launches the attention kernel for tiles of `rows` (128 or 256)
// rows; the caller joins split tiles afterwards.
int tpa_internal_paged_tile(const tpa_paged_view* cache, paged::Params& p, int rows, int grid, cudaStream_t stream);
