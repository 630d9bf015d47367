// k_pages.cu -- pages of the paged cache: copy-on-write reservation, sharing, release and
// compaction of a pool kept on the device, and the copies that they ask for.
//
// The pool is page_table [rows, max_pages], n_pages [rows] and refcount [num_pages].  All
// its state is integers and every result is unique: fresh pages are the lowest free ones in
// order of (row, page index), compaction pairs pages by rank.  Atomics only add, subtract
// or take a minimum, so their order does not matter.
//
// The table work is latency: a few dependent passes over 4 bytes per page (a pool of 62000
// pages, one GPU's memory at 61 layers, is 250 KB).  One cluster of CTAs does it in one
// launch, each CTA scanning its slice of the counts, with counts exchanged through
// distributed shared memory and one warp per row for the tables.  The copies are the bytes:
// 64 keys of 1152 bytes per page and layer.
#include <algorithm>
#include <climits>

#include "sm100_ptx.h"
#include "tv_internal.h"

namespace tv {
namespace {

using namespace ptx;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;

struct Workspace {
  int32_t* a;     // reserve: writers of a shared page.   compact: holes by rank
  int32_t* b;     // reserve: its lowest writer.          compact: pages that move, by rank
  int32_t* c;     // reserve: free pages by rank.         compact: where a page moves
  int32_t* head;  // compact: {pages in use, moves}
};
__host__ __device__ inline size_t ws_array(int num_pages) {
  return ((size_t)num_pages * 4 + 255) / 256 * 256;
}
Workspace split(void* ws, int num_pages) {
  char* p = (char*)ws;
  const size_t n = ws_array(num_pages);
  return {(int32_t*)p, (int32_t*)(p + n), (int32_t*)(p + 2 * n), (int32_t*)(p + 3 * n)};
}

// Loads that see what another CTA of the cluster wrote (these kernels also write the
// arrays, so the read-only path is not open to them).
__device__ __forceinline__ int ld(const int32_t* p) { return __ldcg(p); }

__device__ __forceinline__ void st_cluster_s64(const void* local, uint32_t rank, int64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(map_to_rank(smem_u32(local), rank)), "l"(v)
               : "memory");
}

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the block, for every thread.
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* part) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  int64_t s = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += part[w];
  return s;
}

// This CTA's number into slot `rank` of every CTA; the sum of the slots below this rank and
// of all of them.
struct Offsets {
  int64_t below, total;
};
__device__ __forceinline__ void post(int64_t* slots, int64_t v) {
  if (threadIdx.x < kCluster) st_cluster_s64(&slots[cluster_rank()], threadIdx.x, v);
}
__device__ __forceinline__ Offsets collect(const int64_t* slots) {
  Offsets o{0, 0};
  const int me = (int)cluster_rank();
#pragma unroll
  for (int r = 0; r < kCluster; ++r) {
    o.below += r < me ? slots[r] : 0;
    o.total += slots[r];
  }
  return o;
}

// Ranks of the flagged elements of [p0, p1): f(p, rank) for each, ranks counted from
// `base` in ascending order.  Ends early once the ranks pass `limit`.
template <typename Flag, typename Fn>
__device__ void ranked(int p0, int p1, int64_t base, int64_t limit, int64_t* part, Flag flag,
                       Fn f) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int q = p0; q < p1 && base < limit; q += kThreads) {
    const int p = q + (int)threadIdx.x;
    const bool on = p < p1 && flag(p);
    const uint32_t m = __ballot_sync(0xffffffffu, on);
    __syncthreads();
    if (lane == 0) part[warp] = __popc(m);
    __syncthreads();
    int64_t before = base, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      before += w < warp ? part[w] : 0;
      all += part[w];
    }
    if (on) f(p, before + __popc(m & ((1u << lane) - 1)));
    base += all;
  }
}

// ---- reserve --------------------------------------------------------------------------
struct RowNeed {
  bool active;
  int n, first, need;  // pages held, first page written, pages wanted
};

__device__ __forceinline__ RowNeed row_need(const tv_page_pool& P, int r,
                                            const int32_t* __restrict__ length,
                                            const int32_t* __restrict__ new_length, bool* bad) {
  RowNeed w{};
  const int len = length[r], nl = new_length[r];
  w.active = nl > len;
  if (!w.active) return w;
  w.n = ld(P.n_pages + r);
  const int64_t need = ((int64_t)nl + P.page_size - 1) / P.page_size;
  if (len < 0 || w.n < 0 || w.n > P.max_pages || (int64_t)len > (int64_t)w.n * P.page_size ||
      need > P.max_pages) {
    *bad = true;
    w.active = false;
    return w;
  }
  w.first = len / P.page_size;
  w.need = (int)need;
  return w;
}

// Whether page index k of row r gets a fresh page.  `old`: the page it holds, or -1.
__device__ __forceinline__ bool takes(const tv_page_pool& P, const Workspace& W, const RowNeed& w,
                                      int r, int k, int* old) {
  *old = -1;
  if (k >= w.n) return true;
  const int p = ld(P.page_table + (int64_t)r * P.max_pages + k);
  const int c = ld(P.refcount + p);
  if (c <= 1) return false;
  *old = p;
  return !(ld(W.a + p) == c && ld(W.b + p) == r);
}

__global__ void __cluster_dims__(kCluster) __launch_bounds__(kThreads)
    reserve_kernel(tv_page_pool P, Workspace W, const int32_t* __restrict__ length,
                   const int32_t* __restrict__ new_length, int32_t* __restrict__ copies,
                   int32_t* status) {
  __shared__ int64_t s_free[kCluster], s_need[kCluster], s_bad[kCluster], s_part[kWarps];
  __shared__ int64_t s_row[4096 / kCluster + 1];
  __shared__ int s_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank();
  const int per = (P.num_pages + kCluster - 1) / kCluster;
  const int p0 = min(P.num_pages, rank * per), p1 = min(P.num_pages, p0 + per);
  const int per_r = (P.rows + kCluster - 1) / kCluster;
  const int r0 = min(P.rows, rank * per_r), r1 = min(P.rows, r0 + per_r);
  if (tid == 0) s_flag = 0;
  // free pages of this slice; scratch of the shared ones
  int n_free = 0;
  for (int p = p0 + tid; p < p1; p += kThreads) {
    const int c = ld(P.refcount + p);
    n_free += c == 0;
    if (c > 1) {
      W.a[p] = 0;
      W.b[p] = INT_MAX;
    }
  }
  const int64_t free_here = block_sum(n_free, s_part);
  cluster_sync();
  // who writes which shared page; what is wrong with a row
  bool bad = false;
  for (int r = r0 + warp; r < r1; r += kWarps) {
    const RowNeed w = row_need(P, r, length, new_length, &bad);
    for (int k = w.first + lane; w.active && k < min(w.need, w.n); k += 32) {
      const int p = ld(P.page_table + (int64_t)r * P.max_pages + k);
      const int c = p >= 0 && p < P.num_pages ? ld(P.refcount + p) : 0;
      if (c < 1) {
        bad = true;
      } else if (c > 1) {
        atomicAdd(W.a + p, 1);
        atomicMin(W.b + p, r);
      }
    }
  }
  if (bad) s_flag = 1;
  __syncthreads();
  post(s_bad, s_flag);
  cluster_sync();
  const bool any_bad = collect(s_bad).total > 0;
  // fresh pages per row
  int64_t mine = 0;
  if (!any_bad) {
    for (int r = r0 + warp; r < r1; r += kWarps) {
      bool unused = false;
      const RowNeed w = row_need(P, r, length, new_length, &unused);
      int n = 0, old;
      for (int k = w.first + lane; w.active && k < w.need; k += 32)
        n += takes(P, W, w, r, k, &old);
      const int64_t t = warp_sum(n);
      if (lane == 0) {
        s_row[r - r0] = t;
        mine += t;
      }
    }
  }
  const int64_t need_here = block_sum(mine, s_part);
  post(s_free, free_here);
  post(s_need, need_here);
  cluster_sync();
  const Offsets of = collect(s_free), on = collect(s_need);
  if (any_bad || on.total > of.total) {  // the whole cluster alike
    for (int i = r0 * 3 + tid; i < r1 * 3; i += kThreads) copies[i] = i % 3 == 2 ? 0 : -1;
    if (rank == 0 && tid == 0) report(status, any_bad ? TV_ERR_BOUNDS : TV_ERR_NO_PAGES);
    return;
  }
  // the lowest free pages, by rank
  ranked(
      p0, p1, of.below, on.total, s_part, [&](int p) { return ld(P.refcount + p) == 0; },
      [&](int p, int64_t i) {
        if (i < on.total) W.c[i] = p;
      });
  // where each row's fresh pages start
  __syncthreads();
  if (tid == 0) {
    int64_t at = on.below;
    for (int r = 0; r < r1 - r0; ++r) {
      const int64_t n = s_row[r];
      s_row[r] = at;
      at += n;
    }
  }
  cluster_sync();
  for (int r = r0 + warp; r < r1; r += kWarps) {
    bool unused = false;
    const RowNeed w = row_need(P, r, length, new_length, &unused);
    int src = -1, dst = -1;
    int64_t at = s_row[r - r0];
    for (int k0 = w.first; w.active && k0 < w.need; k0 += 32) {
      const int k = k0 + lane;
      int old = -1;
      const bool take = k < w.need && takes(P, W, w, r, k, &old);
      const uint32_t m = __ballot_sync(0xffffffffu, take);
      if (take) {
        const int fresh = ld(W.c + at + __popc(m & ((1u << lane) - 1)));
        P.page_table[(int64_t)r * P.max_pages + k] = fresh;
        P.refcount[fresh] = 1;
        if (old >= 0 && k == w.first) {
          src = old;
          dst = fresh;
        }
      }
      at += __popc(m);
    }
    if (lane == 0) {  // lane 0 has the first page written
      const int n = w.active ? length[r] % P.page_size : 0;
      const bool copy = src >= 0 && n > 0;
      copies[r * 3] = copy ? src : -1;
      copies[r * 3 + 1] = copy ? dst : -1;
      copies[r * 3 + 2] = copy ? n : 0;
      if (w.active && w.need > w.n) P.n_pages[r] = w.need;
    }
  }
  cluster_sync();
  // shared pages lose the holders that moved off
  for (int p = p0 + tid; p < p1; p += kThreads) {
    const int c = ld(P.refcount + p);
    if (c > 1) {
      const int n = ld(W.a + p);
      if (n > 0) P.refcount[p] = n == c ? 1 : c - n;
    }
  }
}

// ---- fork, release ----------------------------------------------------------------------
__global__ void __launch_bounds__(128)
    fork_kernel(tv_page_pool P, const int32_t* __restrict__ fork_from,
                const int32_t* __restrict__ length, int32_t* status) {
  const int r = blockIdx.x, src = fork_from[r];
  if (src < 0) return;
  const int64_t want = ((int64_t)length[r] + P.page_size - 1) / P.page_size;
  bool bad = src >= P.rows || length[r] < 0 || want > P.max_pages || P.n_pages[r] != 0;
  if (!bad) bad = fork_from[src] >= 0 || want > P.n_pages[src];
  const int n = bad ? 0 : (int)want;
  const int32_t* from = P.page_table + (int64_t)src * P.max_pages;
  for (int k = threadIdx.x; k < n; k += blockDim.x) {
    const int p = from[k];
    if (p < 0 || p >= P.num_pages || ld(P.refcount + p) < 1) bad = true;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) report(status, TV_ERR_BOUNDS);
    return;
  }
  int32_t* to = P.page_table + (int64_t)r * P.max_pages;
  for (int k = threadIdx.x; k < n; k += blockDim.x) {
    const int p = from[k];
    to[k] = p;
    atomicAdd(P.refcount + p, 1);
  }
  if (threadIdx.x == 0) P.n_pages[r] = n;
}

__global__ void __launch_bounds__(128)
    release_kernel(tv_page_pool P, const int32_t* __restrict__ keep, int32_t* status) {
  const int r = blockIdx.x;
  if (keep[r] < 0) return;
  const int64_t kept = ((int64_t)keep[r] + P.page_size - 1) / P.page_size;
  const int held = P.n_pages[r], n = min(held, P.max_pages);
  if (kept >= held) return;
  bool bad = held > P.max_pages;
  int32_t* row = P.page_table + (int64_t)r * P.max_pages;
  for (int64_t k = kept + threadIdx.x; k < n; k += blockDim.x) {
    const int p = row[k];
    row[k] = -1;
    if (p < 0 || p >= P.num_pages) {
      bad = true;
    } else if (atomicSub(P.refcount + p, 1) < 1) {
      atomicAdd(P.refcount + p, 1);
      bad = true;
    }
  }
  if (__syncthreads_or(bad) && threadIdx.x == 0) report(status, TV_ERR_BOUNDS);
  if (threadIdx.x == 0) P.n_pages[r] = (int)kept;
}

// ---- compact ----------------------------------------------------------------------------
__global__ void __cluster_dims__(kCluster) __launch_bounds__(kThreads)
    compact_plan_kernel(tv_page_pool P, Workspace W, int32_t* __restrict__ moves,
                        int32_t* __restrict__ n_moves) {
  __shared__ int64_t s_used[kCluster], s_hole[kCluster], s_move[kCluster], s_part[kWarps];
  const int tid = threadIdx.x, rank = (int)cluster_rank();
  const int per = (P.num_pages + kCluster - 1) / kCluster;
  const int p0 = min(P.num_pages, rank * per), p1 = min(P.num_pages, p0 + per);
  int n = 0;
  for (int p = p0 + tid; p < p1; p += kThreads) n += ld(P.refcount + p) > 0;
  const int64_t here = block_sum(n, s_part);
  post(s_used, here);
  cluster_sync();
  const int used = (int)collect(s_used).total;
  int holes = 0, movers = 0;
  for (int p = p0 + tid; p < p1; p += kThreads) {
    const bool on = ld(P.refcount + p) > 0;
    holes += !on && p < used;
    movers += on && p >= used;
    if (!on) W.c[p] = -1;
  }
  const int64_t holes_here = block_sum(holes, s_part), movers_here = block_sum(movers, s_part);
  post(s_hole, holes_here);
  post(s_move, movers_here);
  cluster_sync();
  const Offsets oh = collect(s_hole), om = collect(s_move);
  ranked(
      p0, min(p1, used), oh.below, LLONG_MAX, s_part,
      [&](int p) { return ld(P.refcount + p) <= 0; }, [&](int p, int64_t i) { W.a[i] = p; });
  ranked(
      max(p0, used), p1, om.below, LLONG_MAX, s_part,
      [&](int p) { return ld(P.refcount + p) > 0; }, [&](int p, int64_t i) { W.b[i] = p; });
  cluster_sync();
  const int total = (int)om.total;  // as many holes as pages that move
  for (int i = rank * kThreads + tid; i < total; i += kCluster * kThreads) {
    const int from = ld(W.b + i), to = ld(W.a + i);
    W.c[from] = to;
    moves[i * 3] = from;
    moves[i * 3 + 1] = to;
    moves[i * 3 + 2] = P.page_size;
    P.refcount[to] = ld(P.refcount + from);
    P.refcount[from] = 0;
  }
  if (rank == 0 && tid == 0) {
    *n_moves = total;
    W.head[0] = used;
  }
}

__global__ void __launch_bounds__(256)
    compact_tables_kernel(tv_page_pool P, Workspace W, int32_t* status) {
  const int r = blockIdx.x, used = W.head[0];
  const int n = min(P.n_pages[r], P.max_pages);
  int32_t* row = P.page_table + (int64_t)r * P.max_pages;
  for (int k = threadIdx.x; k < n; k += blockDim.x) {
    const int p = row[k];
    const int to = p >= 0 && p < used ? p : p >= used && p < P.num_pages ? W.c[p] : -1;
    if (to < 0) report(status, TV_ERR_BOUNDS);
    else if (to != p) row[k] = to;
  }
}

// ---- copy -------------------------------------------------------------------------------
constexpr int kCopyThreads = 256;
constexpr int kCopyRows = 16;  // rows per unit of work

struct CopyParams {
  uint4 *c_kv, *k_pe;
  int64_t ckv_stride, kpe_stride, ckv_layer, kpe_layer;  // in 16-byte words
  int ckv_words, kpe_words, n_layers, page_size, chunks;
  int64_t num_rows;
  const int32_t* list;
  const int32_t* count;
  int n_list;
  int32_t* status;
};

__device__ __forceinline__ void copy_rows(uint4* x, int64_t stride, int words, int64_t src,
                                          int64_t dst, int rows) {
  const int total = rows * words;
  for (int i = threadIdx.x; i < total; i += 4 * kCopyThreads) {
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = i + u * kCopyThreads;
      if (j < total) v[u] = x[(src + j / words) * stride + j % words];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = i + u * kCopyThreads;
      if (j < total) x[(dst + j / words) * stride + j % words] = v[u];
    }
  }
}

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(CopyParams p) {
  const int n = p.count ? min(max(*p.count, 0), p.n_list) : p.n_list;
  const int64_t units = (int64_t)n * p.n_layers * p.chunks;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int chunk = (int)(u % p.chunks);
    const int64_t e = u / p.chunks;
    const int layer = (int)(e % p.n_layers);
    const int32_t* entry = p.list + e / p.n_layers * 3;
    const int64_t s = entry[0], d = entry[1];
    const int rows = entry[2];
    if (s < 0 || rows == 0) continue;
    if (d < 0 || rows < 0 || rows > p.page_size || (s + 1) * p.page_size > p.num_rows ||
        (d + 1) * p.page_size > p.num_rows) {
      if (threadIdx.x == 0) report(p.status, TV_ERR_BOUNDS);
      continue;
    }
    const int at = chunk * kCopyRows, here = min(kCopyRows, rows - at);
    if (here <= 0) continue;
    const int64_t src = s * p.page_size + at, dst = d * p.page_size + at;
    copy_rows(p.c_kv + layer * p.ckv_layer, p.ckv_stride, p.ckv_words, src, dst, here);
    if (p.kpe_words > 0)
      copy_rows(p.k_pe + layer * p.kpe_layer, p.kpe_stride, p.kpe_words, src, dst, here);
  }
}

}  // namespace

size_t pages_workspace(const tv_page_pool& p) { return 3 * ws_array(p.num_pages) + 256; }

cudaError_t launch_pages_reserve(const tv_page_pool& p, const int32_t* length,
                                 const int32_t* new_length, int32_t* copies, int32_t* status,
                                 void* ws, cudaStream_t st) {
  reserve_kernel<<<kCluster, kThreads, 0, st>>>(p, split(ws, p.num_pages), length, new_length,
                                                copies, status);
  return cudaGetLastError();
}

cudaError_t launch_pages_fork(const tv_page_pool& p, const int32_t* fork_from,
                              const int32_t* length, int32_t* status, cudaStream_t st) {
  fork_kernel<<<p.rows, 128, 0, st>>>(p, fork_from, length, status);
  return cudaGetLastError();
}

cudaError_t launch_pages_release(const tv_page_pool& p, const int32_t* keep, int32_t* status,
                                 cudaStream_t st) {
  release_kernel<<<p.rows, 128, 0, st>>>(p, keep, status);
  return cudaGetLastError();
}

cudaError_t launch_pages_compact(const tv_page_pool& p, int32_t* moves, int32_t* n_moves,
                                 int32_t* status, void* ws, cudaStream_t st) {
  const Workspace w = split(ws, p.num_pages);
  compact_plan_kernel<<<kCluster, kThreads, 0, st>>>(p, w, moves, n_moves);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  compact_tables_kernel<<<p.rows, 256, 0, st>>>(p, w, status);
  return cudaGetLastError();
}

cudaError_t launch_pages_copy(void* c_kv, void* k_pe, int64_t ckv_stride, int64_t kpe_stride,
                              int ckv_row, int kpe_row, int n_layers, int64_t ckv_layer,
                              int64_t kpe_layer, int page_size, int64_t num_rows,
                              const int32_t* list, const int32_t* count, int n_list,
                              int32_t* status, cudaStream_t st) {
  CopyParams p{};
  p.c_kv = (uint4*)c_kv;
  p.k_pe = (uint4*)k_pe;
  p.ckv_stride = ckv_stride / 16;
  p.kpe_stride = kpe_stride / 16;
  p.ckv_layer = ckv_layer / 16;
  p.kpe_layer = kpe_layer / 16;
  p.ckv_words = ckv_row / 16;
  p.kpe_words = kpe_row / 16;
  p.n_layers = n_layers;
  p.page_size = page_size;
  p.chunks = (page_size + kCopyRows - 1) / kCopyRows;
  p.num_rows = num_rows;
  p.list = list;
  p.count = count;
  p.n_list = n_list;
  p.status = status;
  const int64_t units = (int64_t)n_list * n_layers * p.chunks;
  const int64_t grid = std::min<int64_t>(units, 8ll * current_sm_count());
  copy_kernel<<<(unsigned)grid, kCopyThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace tv
