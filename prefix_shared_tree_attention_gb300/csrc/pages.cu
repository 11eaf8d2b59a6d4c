// The pages of a cache: which are free, which sequence has them, and sequences that
// begin as copies of others.
//
// The state is a count of uses for each page and the page tables, both in device
// memory; a page is free when its count is 0, and free pages are handed out lowest
// first, in the order of the rows, so that the same calls give the same tables.  Both
// calls do their bookkeeping in one cluster of 8 CTAs, whose 256 warps take the rows and the
// counts in turn: what each row wants is told to all CTAs, the counts are read once and kept as a bit a page in
// shared memory, and each warp then hands out an equal run of the free pages, which it finds among the shares' running
// sums and whose rows it finds among those of what the rows want.  Nothing is handed out before it is known that it
// suffices.  Bound by the chain of dependent reads (a row's length, its table, the counts) and the cluster barriers; the
// bytes are 4 a page of the pool and 8 a table entry that changes.
#include <cuda_runtime.h>

#include <initializer_list>

#include "device_common.cuh"
#include "internal.h"
#include "paged_common.cuh"
#include "tc.cuh"

namespace {

__device__ unsigned int g_status_pages = 0;

constexpr int kCluster = 8;
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kShares = kCluster * kWarps;  // of the counts, one a warp
constexpr int kMostRows = 8192;             // rows of a call
constexpr int kMostTable = 1 << 18;         // rows of a table that is forked in
constexpr int kMostPages = 1 << 23;
constexpr int kU = 4;                       // entries of a row that a lane has under way together

__device__ __forceinline__ void report() { atomicOr(&g_status_pages, TPA_DEV_BAD_INPUT); }

// (Inputs are read by plain loads: the kernel before, which may still run when this one starts, may write them.)
struct Params {
  int32_t* pages;
  int32_t* kv_lens;
  int32_t* refs;
  int32_t* n_free;
  const int32_t* src;
  const int32_t* dst;
  int32_t n_pages, page_shift, n_rows, max_pages, page_stride;  // n_rows: of the table
  int32_t n_forks;
  int32_t words;  // of 32 counts, in a share
};

// Shared memory: what each row wants (and one more), the entry of the row that the first of them goes to, the free
// pages of this CTA's shares as bits, and in a fork a bit for each row that is a dst.
struct Shared {
  int64_t warp_v[kWarps];
  int32_t share[kShares + 1];  // free pages of each share; then their running sums
  int32_t bad;
};
struct View {
  Shared& sh;
  int32_t* want;
  int32_t* have;
  uint32_t* free;
  uint32_t* named;
  __device__ __forceinline__ View(uint8_t* smem, int rows, int words)
      : sh(*reinterpret_cast<Shared*>(smem)),
        want(reinterpret_cast<int32_t*>(smem + sizeof(Shared))),
        have(want + rows + 1),
        free(reinterpret_cast<uint32_t*>(have + rows)),
        named(free + kWarps * words) {}
};
// rows: of the call; table: rows of the table in a fork, else 0
uint32_t shared_bytes(int rows, int words, int table) {
  return uint32_t(sizeof(Shared)) + 4u * (2u * rows + 1 + kWarps * words + (table + 31) / 32);
}

// Entries at the head of a row that hold a page: they are not negative, and the ones behind them are.
__device__ __forceinline__ int held(const int32_t* row, int width) {
  int lo = 0, hi = width;
  while (lo < hi) {  // three entries at a time
    const int q = max((hi - lo) >> 2, 1), a = lo + q - 1, b = a + q, c = b + q;
    const bool fa = __ldcg(row + a) >= 0, fb = __ldcg(row + min(b, hi - 1)) >= 0, fc = __ldcg(row + min(c, hi - 1)) >= 0;
    if (c < hi && fc) lo = c + 1;
    else if (b < hi && fb) lo = b + 1, hi = min(c, hi);
    else if (fa) lo = a + 1, hi = min(b, hi);
    else hi = a;
  }
  return lo;
}

__device__ __forceinline__ void give_back(const Params& p, int page) {
  if (uint32_t(page) >= uint32_t(p.n_pages)) {
    if (page >= 0) report();
  } else if (atomicSub(p.refs + page, 1) <= 0) {  // it was not in use
    atomicAdd(p.refs + page, 1);
    report();
  }
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void tell_all(int32_t* at, int32_t v) {
#pragma unroll
  for (int c = 0; c < kCluster; ++c) tc::st_cluster_u32(tc::peer_addr(at, c), uint32_t(v));
}

// Running sums of v >= 0 over the CTA's threads, modulo 2^32; the whole in `total`, exactly.
__device__ __forceinline__ int cta_scan(int v, Shared& sh, int64_t& total) {  // (by all threads)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  const uint32_t high = __reduce_add_sync(0xffffffffu, uint32_t(v) >> 16), low = __reduce_add_sync(0xffffffffu, uint32_t(v) & 0xffffu);
  __syncthreads();
  if (lane == 31) sh.warp_v[warp] = (int64_t(high) << 16) + low;
  __syncthreads();
  uint32_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += uint32_t(sh.warp_v[w]);
    total += sh.warp_v[w];
  }
  return int(before + incl - uint32_t(v));
}

// This CTA's rows of n, dealt out in turn: f(row) by a thread each.
template <class F>
__device__ __forceinline__ void each_row(int n, int rank, F f) {
  for (int r = rank + kCluster * int(threadIdx.x); r < n; r += kCluster * kThreads) f(r);
}
// And by a warp each.
template <class F>
__device__ __forceinline__ void each_row_warp(int n, int rank, F f) {
  for (int r = rank + kCluster * int(threadIdx.x >> 5); r < n; r += kCluster * kWarps) f(r);
}

// Hands out free pages for v.want (n rows; row_of names the row of the table): every CTA has all of want and have.
// Returns the free pages left, or minus the number missing, and then nothing was handed out.  Ends with the cluster together.
template <class RowOf>
__device__ int hand_out(const Params& p, int n, int rank, const View& v, RowOf row_of) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, share = rank * kWarps + warp;
  {  // this warp's share of the counts
    constexpr int kWordsAhead = 8;
    const int64_t first = int64_t(share) * p.words;
    int mine = 0;
    for (int w = 0; w < p.words; w += kWordsAhead) {
      int c[kWordsAhead];
#pragma unroll
      for (int u = 0; u < kWordsAhead; ++u) {
        const int64_t i = (first + w + u) * 32 + lane;
        c[u] = w + u < p.words && i < p.n_pages ? __ldcg(p.refs + i) : 1;
      }
#pragma unroll
      for (int u = 0; u < kWordsAhead; ++u) {
        const unsigned m = __ballot_sync(0xffffffffu, c[u] == 0);
        if (w + u < p.words && lane == 0) v.free[warp * p.words + w + u] = m;
        mine += __popc(m);
      }
    }
    if (lane < kCluster) tc::st_cluster_u32(tc::peer_addr(&v.sh.share[share], lane), uint32_t(mine));
  }
  // running sums of what the rows want, a run of rows a thread (8 rows of less than 2^26 pages; the whole may pass 32
  // bits, and `room` with them: then the sums are not looked at)
  const int each = (n + kThreads - 1) / kThreads;
  const int a = min(int(threadIdx.x) * each, n), b = min(a + each, n);
  int sum = 0;
  int64_t all;
  for (int i = a; i < b; ++i) sum += v.want[i];
  int at = cta_scan(sum, v.sh, all);
  for (int i = a; i < b; ++i) {
    const int w = v.want[i];
    v.want[i] = at;
    at = int(uint32_t(at) + uint32_t(w));
  }
  tc::cluster_sync();
  const int mine = int(threadIdx.x) < kShares ? v.sh.share[threadIdx.x] : 0;
  int64_t room;
  at = cta_scan(mine, v.sh, room);
  if (int(threadIdx.x) < kShares) v.sh.share[threadIdx.x] = at;
  __syncthreads();
  if (all <= room) {
    // ranks [r0, r1) among the free pages are this warp's
    const int r0 = int(all * share / kShares), r1 = int(all * (share + 1) / kShares);
    int s = 0;  // the last share that begins at r0 or before
    for (int step = kShares / 2; step > 0; step >>= 1)
      if (v.sh.share[s + step] <= r0) s += step;
    int before = v.sh.share[s];
    const int64_t words = int64_t(kShares) * p.words;
    for (int64_t w0 = int64_t(s) * p.words; w0 < words && before < r1 && r0 < r1; w0 += 32) {
      unsigned m = 0;  // lane: a word, from the CTA that has it
      if (w0 + lane < words) {
        const int cta = int((w0 + lane) / (kWarps * p.words)), i = int(w0 + lane - int64_t(cta) * kWarps * p.words);
        m = ld_cluster_u32(tc::peer_addr(v.free + i, cta));
      }
      int incl = __popc(m);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      const int begin = before + incl - __popc(m);
      // the words that have some of the ranks, one after the other
      unsigned some = __ballot_sync(0xffffffffu, m != 0 && begin < r1 && begin + __popc(m) > r0);
      while (some) {
        const int k = __ffs(some) - 1;
        some &= some - 1;
        const unsigned word = __shfl_sync(0xffffffffu, m, k);
        const int q = __shfl_sync(0xffffffffu, begin, k) + __popc(word & ((1u << lane) - 1));
        if ((word >> lane & 1) && q >= r0 && q < r1) {
          int lo = 0, hi = n;  // the last row whose running sum is at most q
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (v.want[mid] <= q) lo = mid;
            else hi = mid;
          }
          const int page = int(w0 + k) * 32 + lane;
          p.pages[int64_t(row_of(lo)) * p.page_stride + v.have[lo] + q - v.want[lo]] = page;
          p.refs[page] = 1;
        }
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  tc::cluster_sync();  // the others' bits are read no more
  return int(max(room - all, int64_t(INT32_MIN) + 1));
}

// Rows get the pages that their lengths need: what is behind them goes back, what is missing is handed out.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1) resize_kernel(const Params p) {
  extern __shared__ uint8_t smem[];
  const View v(smem, p.n_rows, p.words);
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // this CTA runs
  tc::grid_launch_dependents();
  tc::grid_wait_prior();
  const int rank = int(tc::cta_rank()), lane = threadIdx.x & 31;
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  each_row(p.n_rows, rank, [&](int r) {
    const int len = p.kv_lens[r];
    const int have = held(p.pages + int64_t(r) * p.page_stride, p.max_pages);
    int need = have;
    if (len < 0 || len > (int64_t(p.max_pages) << p.page_shift)) report();
    else need = int((int64_t(len) + (1 << p.page_shift) - 1) >> p.page_shift);
    tell_all(&v.want[r], need - have);  // negative: pages to give back
    tell_all(&v.have[r], have);
  });
  __syncthreads();  // (this CTA's own rows)
  each_row_warp(p.n_rows, rank, [&](int r) {
    const int have = v.have[r];
    int32_t* row = p.pages + int64_t(r) * p.page_stride;
    for (int j0 = have + v.want[r] + lane; j0 - lane < have; j0 += 32 * kU) {
      int page[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) page[u] = j0 + 32 * u < have ? __ldcg(row + j0 + 32 * u) : -1;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        give_back(p, page[u]);
        if (j0 + 32 * u < have) row[j0 + 32 * u] = -1;
      }
    }
  });
  tc::cluster_sync();  // all is told, and every page that goes back has
  for (int r = threadIdx.x; r < p.n_rows; r += kThreads) v.want[r] = max(v.want[r], 0);
  __syncthreads();
  const int left = hand_out(p, p.n_rows, rank, v, [](int r) { return r; });
  if (rank == 0 && threadIdx.x == 0) *p.n_free = left;
}

// Row dst[f] becomes a copy of row src[f]: the whole pages shared, a page of its own for what is behind them.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1) fork_kernel(const Params p) {
  extern __shared__ uint8_t smem[];
  const View v(smem, p.n_forks, p.words);
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // this CTA runs
  tc::grid_launch_dependents();
  for (int i = threadIdx.x; i < (p.n_rows + 31) / 32; i += kThreads) v.named[i] = 0;
  if (threadIdx.x == 0) v.sh.bad = 0;
  tc::grid_wait_prior();
  const int rank = int(tc::cta_rank()), lane = threadIdx.x & 31;
  __syncthreads();
  // a call with a row out of range, named twice, or both copied and written is not done at all
  for (int f = threadIdx.x; f < p.n_forks; f += kThreads) {
    const int d = p.dst[f];
    if (uint32_t(d) >= uint32_t(p.n_rows) || (atomicOr(v.named + (d >> 5), 1u << (d & 31)) >> (d & 31) & 1)) v.sh.bad = 1;
  }
  __syncthreads();
  for (int f = threadIdx.x; f < p.n_forks; f += kThreads) {
    const int s = p.src[f];
    if (uint32_t(s) >= uint32_t(p.n_rows) || (v.named[s >> 5] >> (s & 31) & 1)) {
      v.sh.bad = 1;
    } else {
      const int len = p.kv_lens[s];
      if (len < 0 || len > (int64_t(p.max_pages) << p.page_shift)) v.sh.bad = 1;
    }
  }
  __syncthreads();
  const bool bad = v.sh.bad;
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  const int n = bad ? 0 : p.n_forks;
  each_row_warp(n, rank, [&](int f) {
    const int s = p.src[f], d = p.dst[f];
    const int len = p.kv_lens[s], whole = len >> p.page_shift, part = len & ((1 << p.page_shift) - 1);
    const int32_t* from = p.pages + int64_t(s) * p.page_stride;
    int32_t* to = p.pages + int64_t(d) * p.page_stride;
    for (int j0 = lane; j0 - lane < p.max_pages; j0 += 32 * kU) {
      int old[kU], page[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int j = j0 + 32 * u;
        old[u] = j < p.max_pages ? __ldcg(to + j) : -1;
        page[u] = j < whole ? __ldcg(from + j) : -1;
      }
      bool more = false;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int j = j0 + 32 * u;
        more |= j < whole || old[u] >= 0;
        if (j < whole && uint32_t(page[u]) >= uint32_t(p.n_pages)) {
          report();
          page[u] = -1;
        }
        if (old[u] != page[u]) {
          if (page[u] >= 0) atomicAdd(p.refs + page[u], 1);
          give_back(p, old[u]);
          to[j] = page[u];
        }
      }
      if (!__any_sync(0xffffffffu, more)) break;
    }
    if (lane == 0) p.kv_lens[d] = len;
    if (lane < kCluster) {
      tc::st_cluster_u32(tc::peer_addr(&v.want[f], lane), part > 0);
      tc::st_cluster_u32(tc::peer_addr(&v.have[f], lane), uint32_t(whole));
    }
  });
  tc::cluster_sync();
  const int left = hand_out(p, n, rank, v, [&](int f) { return p.dst[f]; });
  if (rank == 0 && threadIdx.x == 0) {
    *p.n_free = bad ? INT32_MIN : left;
    if (bad) report();
  }
  if (left < 0) {  // too few: the rows are left empty
    each_row_warp(n, rank, [&](int f) {
      const int d = p.dst[f];
      int32_t* to = p.pages + int64_t(d) * p.page_stride;
      for (int j = lane; j < v.have[f]; j += 32) {
        give_back(p, to[j]);
        to[j] = -1;
      }
      if (lane == 0) p.kv_lens[d] = 0;
    });
  }
}

struct CopyParams {
  uint4* k_cache;
  uint4* v_cache;
  const int32_t* pages;
  const int32_t* kv_lens;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* n_free;
  int64_t layer_pieces;
  int32_t n_pages, page_shift, n_rows, max_pages, page_stride, hkv, pieces;
};

// The tokens of each fork's last page, behind the bookkeeping: a CTA a fork and a layer's keys or values.
__global__ void __launch_bounds__(256) copy_kernel(const CopyParams p) {
  tc::grid_launch_dependents();
  tc::grid_wait_prior();
  const int f = blockIdx.x, layer = blockIdx.y >> 1;
  const int s = p.src[f], d = p.dst[f];
  if (__ldcg(p.n_free) < 0 || uint32_t(s) >= uint32_t(p.n_rows) || uint32_t(d) >= uint32_t(p.n_rows)) return;
  const int len = p.kv_lens[s], whole = len >> p.page_shift, part = len & ((1 << p.page_shift) - 1);
  if (part == 0 || len < 0 || whole >= p.max_pages) return;
  const int from = __ldcg(p.pages + int64_t(s) * p.page_stride + whole), to = __ldcg(p.pages + int64_t(d) * p.page_stride + whole);
  if (uint32_t(from) >= uint32_t(p.n_pages) || uint32_t(to) >= uint32_t(p.n_pages)) {
    if (threadIdx.x == 0) report();
    return;
  }
  uint4* cache = (blockIdx.y & 1 ? p.v_cache : p.k_cache) + layer * p.layer_pieces;
  const int64_t head = int64_t(p.pieces) << p.page_shift;  // of a page's head, in pieces of 16 bytes
  const uint4* a = cache + from * head * p.hkv;
  uint4* b = cache + to * head * p.hkv;
  const int run = part * p.pieces, all = run * p.hkv;
  for (int i0 = threadIdx.x; i0 < all; i0 += kU * blockDim.x) {
    uint4 v[kU];
    int64_t at[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int i = i0 + u * blockDim.x;
      at[u] = -1;
      if (i < all) {
        const int h = i / run;
        at[u] = h * head + (i - h * run);
        v[u] = a[at[u]];
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (at[u] >= 0) b[at[u]] = v[u];
  }
}

int check_pool(const tpa_paged_pool* c) {
  if (!c || !c->refs || c->n_seqs < 0 || c->n_pages < 1 || c->n_pages > kMostPages || c->max_pages < 0 || c->page_stride < c->max_pages ||
      (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) ||
      int64_t(c->max_pages) * c->page_size >= (int64_t(1) << 30))
    return TPA_ERR_INVALID_ARG;
  if (c->n_seqs > 0 && (!c->pages || !c->kv_lens)) return TPA_ERR_INVALID_ARG;
  const uintptr_t a = reinterpret_cast<uintptr_t>(c->refs) | reinterpret_cast<uintptr_t>(c->pages) |
                      reinterpret_cast<uintptr_t>(c->kv_lens);
  return a & 3 ? TPA_ERR_INVALID_ARG : TPA_OK;
}

Params make_params(const tpa_paged_pool* c, int32_t* n_free) {
  Params p = {};
  p.pages = c->pages;
  p.kv_lens = c->kv_lens;
  p.refs = c->refs;
  p.n_free = n_free;
  p.n_pages = c->n_pages;
  p.page_shift = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  p.n_rows = c->n_seqs;
  p.max_pages = c->max_pages;
  p.page_stride = c->page_stride;
  p.words = ((c->n_pages + 31) / 32 + kShares - 1) / kShares;
  return p;
}

// rows: of the call; table: rows of the table in a fork, else 0
int launch(void (*kernel)(Params), const Params& p, int rows, int table, cudaStream_t st) {
  const uint32_t smem = shared_bytes(rows, p.words, table);
  // (always the same limit: calls from several threads set it beside one another)
  const int most = int(shared_bytes(kMostRows, kMostPages / 32 / kShares, kMostTable));
  if (smem > 48 * 1024) TPA_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most));
  return paged::launch_overlapped(kernel, dim3(kCluster), kThreads, smem, st, Params(p));
}

}  // namespace

TPA_DEFINE_STATUS_READER(tpa_internal_status_pages, g_status_pages)

extern "C" int tpa_paged_resize(const tpa_paged_pool* pool, int32_t* n_free, void* stream) {
  TPA_NVTX_RANGE("tpa_paged_resize");
  const int rc = check_pool(pool);
  if (rc != TPA_OK) return rc;
  if (pool->n_seqs > kMostRows || !n_free || (reinterpret_cast<uintptr_t>(n_free) & 3)) return TPA_ERR_INVALID_ARG;
  return launch(resize_kernel, make_params(pool, n_free), pool->n_seqs, 0, static_cast<cudaStream_t>(stream));
}

extern "C" int tpa_paged_fork(const tpa_paged_pool* pool, const int32_t* src, const int32_t* dst, int32_t n_forks,
                              int32_t* n_free, void* stream) {
  TPA_NVTX_RANGE("tpa_paged_fork");
  const int rc = check_pool(pool);
  if (rc != TPA_OK) return rc;
  auto al16 = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; };
  if (!pool->k_cache || !pool->v_cache || !al16(pool->k_cache) || !al16(pool->v_cache) || pool->n_layers < 1 ||
      pool->n_layers > 32767 || (pool->head_dim != 64 && pool->head_dim != 128) || pool->n_heads_kv < 1 ||
      pool->n_heads_kv > 65535 || int64_t(pool->n_pages) * pool->n_heads_kv >= (int64_t(1) << 31) / pool->page_size ||
      pool->n_seqs > kMostTable || n_forks < 0 || n_forks > kMostRows || !n_free)
    return TPA_ERR_INVALID_ARG;
  if (n_forks > 0 && (!src || !dst)) return TPA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst) | reinterpret_cast<uintptr_t>(n_free)) & 3)
    return TPA_ERR_INVALID_ARG;
  Params p = make_params(pool, n_free);
  p.src = src;
  p.dst = dst;
  p.n_forks = n_forks;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int rt = launch(fork_kernel, p, n_forks, pool->n_seqs, st);
  if (rt != TPA_OK || n_forks == 0) return rt;
  CopyParams c = {};
  c.k_cache = static_cast<uint4*>(pool->k_cache);
  c.v_cache = static_cast<uint4*>(pool->v_cache);
  c.pages = p.pages;
  c.kv_lens = p.kv_lens;
  c.src = src;
  c.dst = dst;
  c.n_free = n_free;
  c.pieces = pool->head_dim / 8;
  c.layer_pieces = int64_t(pool->n_pages) * pool->n_heads_kv * pool->page_size * c.pieces;
  c.n_pages = p.n_pages;
  c.page_shift = p.page_shift;
  c.n_rows = p.n_rows;
  c.max_pages = p.max_pages;
  c.page_stride = p.page_stride;
  c.hkv = pool->n_heads_kv;
  return paged::launch_overlapped(copy_kernel, dim3(n_forks, 2 * pool->n_layers), 256, 0, st, static_cast<const CopyParams>(c));
}
