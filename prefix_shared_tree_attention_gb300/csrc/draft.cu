// What surrounds the model in a sampling step that drafts trees: positions and
// masks from the parents, the path that the sampled tokens follow, and the
// cache with that path's keys and values moved to where the sequence goes on.
//
// All three move a few hundred bytes a sequence (the last, 4 d Hkv bytes a layer
// for a moved token), so what counts is the number of dependent reads and the
// launches: a CTA a sequence, trees in shared memory, chains followed there.
#include <cuda_runtime.h>

#include <initializer_list>

#include "device_common.cuh"
#include "internal.h"
#include "paged_common.cuh"
#include "tc.cuh"

namespace {

__device__ unsigned int g_status_draft = 0;

constexpr int kMostDrafted = 1024;  // tokens of a tree
constexpr int kThreads = 128;

__device__ __forceinline__ void report() { atomicOr(&g_status_draft, TPA_DEV_BAD_INPUT); }

// First row and number of a sequence's new tokens; none (and reported) where its numbers are out of range.
// (Inputs are read by plain loads, here and below: the kernel before, which may still run when this one starts, may write them.)
struct Rows {
  int first, n;
};
__device__ __forceinline__ Rows load_rows(const int32_t* offsets, int s, int n_rows, int most) {
  const int o0 = offsets[s], o1 = offsets[s + 1];
  if (o0 < 0 || o1 < o0 || o1 > n_rows || o1 - o0 > most || (s == 0 && o0 != 0)) {
    if (threadIdx.x == 0) report();
    return Rows{0, 0};
  }
  return Rows{o0, o1 - o0};
}

// A thread a token: it walks up to the root and sets its ancestors' bits, which come in falling order.
__global__ void __launch_bounds__(kThreads) masks_kernel(const int32_t* parents, const int32_t* offsets, const int32_t* kv_lens,
                                                         int n_rows, int window, int32_t* positions, uint32_t* masks, int words) {
  __shared__ int16_t up_s[kMostDrafted];
  tc::grid_launch_dependents();
  tc::grid_wait_prior();
  const int s = blockIdx.x;
  const int kv = kv_lens[s];  // under way beside the offsets
  const Rows q = load_rows(offsets, s, n_rows, 32 * words);
  if (kv < 0 && threadIdx.x == 0) report();
  if (q.n == 0 || kv < 0) return;
  const int base = kv - q.n;
  for (int i = threadIdx.x; i < q.n; i += kThreads) {
    int p = parents[q.first + i];
    if (p < -1 || p >= i) {
      report();
      p = -1;
    }
    up_s[i] = int16_t(p);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < q.n; i += kThreads) {
    uint32_t* out = masks + int64_t(q.first + i) * words;
    for (int w = (i >> 5) + 1; w < words; ++w) out[w] = 0;
    int depth = 0, word = i >> 5;
    uint32_t bits = 0;
    for (int j = i; j >= 0; j = up_s[j]) {
      for (; word > j >> 5; --word) {
        out[word] = bits;
        bits = 0;
      }
      if (window == 0 || depth < window) bits |= 1u << (j & 31);
      ++depth;
    }
    for (; word >= 0; --word) {
      out[word] = bits;
      bits = 0;
    }
    positions[q.first + i] = base + depth - 1;
  }
}

// Every token that is the first of its parent's children with the token sampled behind the parent becomes that one's
// next (a negative token, padding of a tree or a row with nothing to draw, is nobody's); then one thread follows the path from row 0.
__global__ void __launch_bounds__(kThreads) accept_kernel(const int32_t* parents, const int32_t* offsets, const int32_t* drafted,
                                                          const int32_t* sampled, int n_rows, int32_t* tokens, int32_t* path,
                                                          int32_t* n_accepted, int most) {
  __shared__ int next_s[kMostDrafted], sampled_s[kMostDrafted];
  __shared__ int16_t path_s[kMostDrafted];
  __shared__ int count_s;
  tc::grid_launch_dependents();
  tc::grid_wait_prior();
  const int s = blockIdx.x;
  const Rows q = load_rows(offsets, s, n_rows, kMostDrafted);
  for (int i = threadIdx.x; i < q.n; i += kThreads) {
    next_s[i] = q.n;
    sampled_s[i] = sampled[q.first + i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < q.n; i += kThreads) {
    const int p = parents[q.first + i], x = drafted[q.first + i];
    if (p < -1 || p >= i) report();
    else if (p >= 0 && x >= 0 && sampled_s[p] == x) atomicMin(next_s + p, i);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int n = 0;
    for (int i = 0; i < q.n && n < most; i = next_s[i]) path_s[n++] = int16_t(i);
    count_s = n;
    n_accepted[s] = n;
  }
  __syncthreads();
  const int n = count_s;
  for (int i = threadIdx.x; i < most; i += kThreads) {
    const int at = i < n ? path_s[i] : -1;
    path[int64_t(s) * most + i] = at;
    tokens[int64_t(s) * most + i] = at >= 0 ? sampled_s[at] : -1;
  }
}

struct CompactParams {
  uint4* k_cache;
  uint4* v_cache;
  const int32_t* pages;
  const int32_t* offsets;
  const int32_t* kv_lens;
  const int32_t* path;
  const int32_t* n_accepted;
  int32_t* new_lens;
  int64_t layer_pieces;  // 16-byte pieces of a layer's cache
  int32_t n_pages, page_shift, max_pages, page_stride, hkv, pieces, n_rows, most;  // pieces: of a token's head
};

// One CTA for a sequence and a layer's keys or values.  A thread keeps to its pieces of a token and takes the path's tokens in
// order, kAhead of them read before they are written: place i is never read for a later token (path[j] >= j > i), and
// what an earlier one reads from it has been read.
constexpr int kAhead = 8;
__global__ void __launch_bounds__(256) compact_kernel(const CompactParams p) {
  tc::grid_launch_dependents();
  tc::grid_wait_prior();
  const int s = blockIdx.x, layer = blockIdx.y >> 1;
  const Rows q = load_rows(p.offsets, s, p.n_rows, 1 << 30);
  const int kv = p.kv_lens[s], base = kv - q.n;
  const int32_t* path = p.path + int64_t(s) * p.most;
  int n = p.n_accepted[s];
  bool bad = n < 0 || n > p.most || n > q.n || base < 0 || kv > (int64_t(p.max_pages) << p.page_shift);
  if (!bad) {
    int wrong = 0;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const int at = path[i];
      wrong |= at < i || at >= q.n || (i > 0 && at <= path[i - 1]);
    }
    bad = __syncthreads_or(wrong);
  }
  if (blockIdx.y == 0 && threadIdx.x == 0) {
    if (bad) report();
    p.new_lens[s] = bad ? kv : base + n;
  }
  if (bad) return;
  uint4* cache = (blockIdx.y & 1 ? p.v_cache : p.k_cache) + layer * p.layer_pieces;
  const int32_t* row = p.pages + int64_t(s) * p.page_stride;
  auto piece_of = [&](int slot, int head, int c) -> int64_t {  // -1: no such page
    const int page = row[slot >> p.page_shift];
    if (uint32_t(page) >= uint32_t(p.n_pages)) {
      report();
      return -1;
    }
    return (((int64_t(page) * p.hkv + head) << p.page_shift) + (slot & ((1 << p.page_shift) - 1))) * p.pieces + c;
  };
  for (int e = threadIdx.x; e < p.hkv * p.pieces; e += blockDim.x) {
    const int head = e / p.pieces, c = e - head * p.pieces;
    for (int i0 = 0; i0 < n; i0 += kAhead) {
      uint4 v[kAhead];
      int64_t to[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        to[u] = -1;
        const int i = i0 + u, at = i < n ? path[i] : i;
        if (at == i) continue;  // it is there (or there is none)
        const int64_t from = piece_of(base + at, head, c);
        if (from < 0) continue;
        to[u] = piece_of(base + i, head, c);
        v[u] = cache[from];
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (to[u] >= 0) cache[to[u]] = v[u];
    }
  }
}

bool aligned4(std::initializer_list<const void*> list) {
  uintptr_t a = 0;
  for (const void* x : list) a |= reinterpret_cast<uintptr_t>(x);
  return (a & 3) == 0;
}

}  // namespace

TPA_DEFINE_STATUS_READER(tpa_internal_status_draft, g_status_draft)

extern "C" int tpa_draft_masks(const int32_t* parents, const int32_t* offsets, const int32_t* kv_lens, int32_t n_seqs,
                               int32_t n_rows, int32_t window, int32_t* positions, int32_t* masks, int32_t mask_words,
                               void* stream) {
  TPA_NVTX_RANGE("tpa_draft_masks");
  if (n_seqs < 0 || n_rows < 0 || n_rows >= (1 << 30) || window < 0 || mask_words < 1 || mask_words > kMostDrafted / 32)
    return TPA_ERR_INVALID_ARG;
  if (n_seqs == 0) return n_rows == 0 ? TPA_OK : TPA_ERR_INVALID_ARG;
  if (!offsets || !kv_lens || !aligned4({parents, offsets, kv_lens, positions, masks})) return TPA_ERR_INVALID_ARG;
  if (n_rows == 0) return TPA_OK;
  if (!parents || !positions || !masks) return TPA_ERR_INVALID_ARG;
  return paged::launch_overlapped(masks_kernel, dim3(n_seqs), kThreads, 0, static_cast<cudaStream_t>(stream), parents, offsets, kv_lens,
                               int(n_rows), int(window), positions, reinterpret_cast<uint32_t*>(masks), int(mask_words));
}

extern "C" int tpa_accept_drafts(const int32_t* parents, const int32_t* offsets, const int32_t* draft_tokens,
                                 const int32_t* sampled, int32_t n_seqs, int32_t n_rows, int32_t* tokens, int32_t* path,
                                 int32_t* n_accepted, int32_t max_path, void* stream) {
  TPA_NVTX_RANGE("tpa_accept_drafts");
  if (n_seqs < 0 || n_rows < 0 || n_rows >= (1 << 30) || max_path < 1 || max_path > kMostDrafted) return TPA_ERR_INVALID_ARG;
  if (n_seqs == 0) return n_rows == 0 ? TPA_OK : TPA_ERR_INVALID_ARG;
  if (!offsets || !tokens || !path || !n_accepted || (n_rows > 0 && (!parents || !draft_tokens || !sampled)) ||
      !aligned4({parents, offsets, draft_tokens, sampled, tokens, path, n_accepted}))
    return TPA_ERR_INVALID_ARG;
  return paged::launch_overlapped(accept_kernel, dim3(n_seqs), kThreads, 0, static_cast<cudaStream_t>(stream), parents, offsets,
                               draft_tokens, sampled, int(n_rows), tokens, path, n_accepted, int(max_path));
}

extern "C" int tpa_paged_compact(const tpa_paged_view* cache, int32_t n_layers, const int32_t* path, const int32_t* n_accepted,
                                 int32_t max_path, int32_t* new_lens, void* stream) {
  TPA_NVTX_RANGE("tpa_paged_compact");
  const int rc = tpa_internal_check_paged(cache);
  if (rc != TPA_OK) return rc;
  if (n_layers < 1 || n_layers > 32767 || max_path < 1) return TPA_ERR_INVALID_ARG;
  if (cache->n_seqs == 0) return TPA_OK;
  if (!path || !n_accepted || !new_lens || new_lens == cache->kv_lens || new_lens == n_accepted || !aligned4({path, n_accepted, new_lens}))
    return TPA_ERR_INVALID_ARG;
  CompactParams p = {};
  p.k_cache = static_cast<uint4*>(cache->k_cache);
  p.v_cache = static_cast<uint4*>(cache->v_cache);
  p.pages = cache->pages;
  p.offsets = cache->offsets;
  p.kv_lens = cache->kv_lens;
  p.path = path;
  p.n_accepted = n_accepted;
  p.new_lens = new_lens;
  p.pieces = cache->head_dim / 8;
  p.layer_pieces = int64_t(cache->n_pages) * cache->n_heads_kv * cache->page_size * p.pieces;
  p.n_pages = cache->n_pages;
  p.page_shift = cache->page_size == 16 ? 4 : cache->page_size == 32 ? 5 : cache->page_size == 64 ? 6 : 7;
  p.max_pages = cache->max_pages;
  p.page_stride = cache->page_stride;
  p.hkv = cache->n_heads_kv;
  p.n_rows = cache->n_rows;
  p.most = max_path;
  const int pieces = p.hkv * p.pieces;
  return paged::launch_overlapped(compact_kernel, dim3(cache->n_seqs, 2 * n_layers), pieces < 256 ? (pieces + 31) / 32 * 32 : 256, 0,
                               static_cast<cudaStream_t>(stream), static_cast<const CompactParams>(p));
}
