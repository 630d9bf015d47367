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
// launch, each CTA scanning its slice of the counts (a run of consecutive pages per thread,
// whose free ones it keeps as bits), with sums exchanged through distributed shared memory.
// The copies are the bytes: 64 keys of 1152 bytes per page and layer.
//
// Measured.  A cycle that forks each of 64 rows into 7 more, reserves and copies the written
// pages and releases: 45 us, overlapped by programmatic launches (55 without).  Alone, reserve
// takes 13.5 (23 with a CTA's rows one after another instead of a thread each), fork 5.5,
// release 7.5 and the copies 27.  Compaction of 1.16 GB: plan 10, tables 4, copies 172.
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

// Every kernel here is launched as a programmatic dependent of the one before it on the
// stream, so that its launch overlaps that one, and waits for it before anything else.  It
// lets the next kernel start only then: one that works before its own wait (an attention
// call's preparation under overlap_prev, which reads the page table) overlaps this kernel
// alone, and not the writers of the table before it.
__device__ __forceinline__ void begin() {
  griddep_wait();
  griddep_launch_dependents();
}
template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), int64_t grid, int block, cudaStream_t st,
                   Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

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
  return warp_sum(part[threadIdx.x & 31]);
}
static_assert(kWarps == 32, "one part per lane");

// The same, with the sum of the threads before this one.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* part, int64_t* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t up_to = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t below = __shfl_up_sync(0xffffffffu, up_to, o);
    if (lane >= o) up_to += below;
  }
  __syncthreads();
  if (lane == 31) part[warp] = up_to;
  __syncthreads();
  const int64_t mine = part[lane];
  const int64_t before = warp_sum(lane < warp ? mine : 0);
  *total = warp_sum(mine);
  return before + up_to - v;
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

// A thread's run of consecutive pages of this CTA's slice, with a bit for each flagged one
// where the run has at most 64 pages (a pool of half a million); longer runs are read again.
struct Run {
  int p0, p1;
  uint64_t bits;
};
__device__ __forceinline__ Run run_of(int num_pages) {
  const int per = (num_pages + kCluster - 1) / kCluster;
  const int s0 = min(num_pages, (int)cluster_rank() * per), s1 = min(num_pages, s0 + per);
  const int each = (per + kThreads - 1) / kThreads;
  const int p0 = min(s1, s0 + (int)threadIdx.x * each);
  return {p0, min(s1, p0 + each), 0ull};
}
template <typename Flag>
__device__ __forceinline__ int mark(Run& r, Flag flag) {
  int n = 0;
  r.bits = 0;
#pragma unroll 4
  for (int p = r.p0; p < r.p1; ++p)
    if (flag(p)) {
      ++n;
      r.bits |= 1ull << ((p - r.p0) & 63);
    }
  return n;
}
// f(p, rank) for each flagged page of the run, ranks from `rank` on and below `limit`.
template <typename Flag, typename Fn>
__device__ __forceinline__ void emit(const Run& r, int64_t rank, int64_t limit, Flag flag, Fn f) {
  const bool known = r.p1 - r.p0 <= 64;
  if (known && r.bits == 0) return;
  for (int p = r.p0; p < r.p1 && rank < limit; ++p)
    if (known ? (r.bits >> (p - r.p0)) & 1 : flag(p)) f(p, rank++);
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

__global__ void __cluster_dims__(kCluster) __launch_bounds__(kThreads)
    reserve_kernel(tv_page_pool P, Workspace W, const int32_t* __restrict__ length,
                   const int32_t* __restrict__ new_length, int32_t* __restrict__ copies,
                   int32_t* status) {
  constexpr int kRows = 4096 / kCluster;  // of a CTA at most: one per thread
  static_assert(kRows <= kThreads, "a thread per row");
  __shared__ int64_t s_flags[kCluster], s_free[kCluster], s_need[kCluster], s_part[kWarps];
  __shared__ int s_new[kRows], s_at[kRows], s_k[kRows];  // of the pages behind those held
  cluster_arrive();  // a CTA's shared memory may be written once it is known to have started
  begin();
  const int tid = threadIdx.x;
  const int per_r = (P.rows + kCluster - 1) / kCluster;
  const int r0 = min(P.rows, (int)cluster_rank() * per_r), r1 = min(P.rows, r0 + per_r);
  const int r = r0 + tid;
  // the row, and its pages that are written again: [first, held)
  RowNeed w{};
  bool bad = false, shared = false;
  if (r < r1) w = row_need(P, r, length, new_length, &bad);
  int32_t* row = P.page_table + (int64_t)r * P.max_pages;
  const int held = w.active ? min(w.need, w.n) : 0;
  for (int k = w.first; k < held; ++k) {
    const int p = ld(row + k);
    const int c = p >= 0 && p < P.num_pages ? ld(P.refcount + p) : 0;
    if (c < 1) {
      bad = true;
    } else if (c > 1) {
      shared = true;
      W.a[p] = 0;  // every writer the same
      W.b[p] = INT_MAX;
    }
  }
  // free pages of this slice
  Run run = run_of(P.num_pages);
  const auto is_free = [&](int p) { return ld(P.refcount + p) == 0; };
  int64_t free_here;
  const int64_t free_before = block_scan(mark(run, is_free), s_part, &free_here);
  const int64_t flags = __syncthreads_or(bad) ? 1ll << 32 : 0;
  cluster_wait();
  post(s_flags, flags + (__syncthreads_or(shared) ? 1 : 0));
  post(s_free, free_here);
  cluster_sync();
  const int64_t all_flags = collect(s_flags).total;
  const Offsets of = collect(s_free);
  const bool any_bad = all_flags >> 32;
  int swaps = 0;
  if (!any_bad && all_flags) {  // somewhere a shared page is written
    for (int k = w.first; k < held; ++k) {
      const int p = ld(row + k);
      if (ld(P.refcount + p) > 1) {
        atomicAdd(W.a + p, 1);
        atomicMin(W.b + p, r);
      }
    }
    cluster_sync();
    for (int k = w.first; k < held; ++k) {
      const int p = ld(row + k), c = ld(P.refcount + p);
      if (c > 1 && !(ld(W.a + p) == c && ld(W.b + p) == r)) {
        row[k] = ~p;  // to be replaced
        ++swaps;
      }
    }
  }
  const int fresh_k = max(w.n, w.first);  // the first page index that the row does not hold
  const int news = w.active ? max(0, w.need - fresh_k) : 0;
  int64_t need_here, news_here;
  const int64_t need_before = block_scan((int64_t)swaps + news, s_part, &need_here);
  const int64_t news_before = block_scan(news, s_part, &news_here);
  post(s_need, need_here);
  cluster_sync();
  const Offsets on = collect(s_need);
  if (any_bad || on.total > of.total) {  // the whole cluster alike
    for (int k = w.first; swaps > 0 && k < held; ++k) {
      const int p = ld(row + k);
      if (p < 0) row[k] = ~p;
    }
    for (int i = r0 * 3 + tid; i < r1 * 3; i += kThreads) copies[i] = i % 3 == 2 ? 0 : -1;
    if (cluster_rank() == 0 && tid == 0) report(status, any_bad ? TV_ERR_BOUNDS : TV_ERR_NO_PAGES);
    return;
  }
  // the lowest free pages, by rank
  emit(run, of.below + free_before, on.total, is_free, [&](int p, int64_t i) { W.c[i] = p; });
  int at = (int)(on.below + need_before);  // below num_pages
  if (r < r1) {
    s_new[tid] = (int)news_before;
    s_at[tid] = at + swaps - (int)news_before;
    s_k[tid] = fresh_k - (int)news_before;
  }
  cluster_sync();
  if (r < r1) {
    int src = -1, dst = -1;
    for (int k = w.first; swaps > 0 && k < held; ++k) {
      const int p = ld(row + k);
      if (p >= 0) continue;
      const int fresh = ld(W.c + at++);
      row[k] = fresh;
      P.refcount[fresh] = 1;
      atomicSub(P.refcount + ~p, 1);
      if (k == w.first) {
        src = ~p;
        dst = fresh;
      }
    }
    const int n = w.active ? length[r] % P.page_size : 0;
    const bool copy = src >= 0 && n > 0;
    copies[r * 3] = copy ? src : -1;
    copies[r * 3 + 1] = copy ? dst : -1;
    copies[r * 3 + 2] = copy ? n : 0;
    if (news > 0) P.n_pages[r] = w.need;
  }
  // pages behind the ones held, all threads alike: their number differs from row to row
  for (int i = tid; i < (int)news_here; i += kThreads) {
    int x = 0, y = r1 - r0;  // the row x with s_new[x] <= i < s_new[x + 1]
    while (y - x > 1) {
      const int mid = (x + y) / 2;
      if (s_new[mid] <= i) x = mid;
      else y = mid;
    }
    const int fresh = ld(W.c + s_at[x] + i);
    P.page_table[(int64_t)(r0 + x) * P.max_pages + s_k[x] + i] = fresh;
    P.refcount[fresh] = 1;
  }
}

// ---- fork, release ----------------------------------------------------------------------
__global__ void __launch_bounds__(128)
    fork_kernel(tv_page_pool P, const int32_t* __restrict__ fork_from,
                const int32_t* __restrict__ length, int32_t* status) {
  begin();
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
  begin();
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
  cluster_arrive();  // (as above)
  begin();
  const int tid = threadIdx.x, rank = (int)cluster_rank();
  Run run = run_of(P.num_pages);
  const auto is_used = [&](int p) { return ld(P.refcount + p) > 0; };
  const int64_t here = block_sum(mark(run, is_used), s_part);
  cluster_wait();
  post(s_used, here);
  cluster_sync();
  const int used = (int)collect(s_used).total;
  const auto is_hole = [&](int p) { return p < used && ld(P.refcount + p) <= 0; };
  const auto moves_on = [&](int p) { return p >= used && ld(P.refcount + p) > 0; };
  Run holes = run, movers = run;
  if (run.p1 - run.p0 <= 64) {  // from the bits: those below `used`, and the others
    const int n = max(0, min(run.p1, used) - run.p0);
    const uint64_t low = n >= 64 ? ~0ull : (1ull << n) - 1;
    const int m = run.p1 - run.p0;
    holes.bits = ~run.bits & low & (m >= 64 ? ~0ull : m > 0 ? (1ull << m) - 1 : 0ull);
    movers.bits = run.bits & ~low;
  }
  const bool known = run.p1 - run.p0 <= 64;
  int64_t holes_here, movers_here;
  const int64_t hole0 = block_scan(known ? __popcll(holes.bits) : mark(holes, is_hole), s_part,
                                   &holes_here);
  const int64_t move0 = block_scan(known ? __popcll(movers.bits) : mark(movers, moves_on), s_part,
                                   &movers_here);
  // where a page goes: -1 for the free ones (a table that names one is wrong)
  for (int p = max(run.p0, used); p < run.p1; ++p)
    if (known ? !((run.bits >> (p - run.p0)) & 1) : !is_used(p)) W.c[p] = -1;
  post(s_hole, holes_here);
  post(s_move, movers_here);
  cluster_sync();
  const Offsets oh = collect(s_hole), om = collect(s_move);
  emit(holes, oh.below + hole0, LLONG_MAX, is_hole, [&](int p, int64_t i) { W.a[i] = p; });
  emit(movers, om.below + move0, LLONG_MAX, moves_on, [&](int p, int64_t i) { W.b[i] = p; });
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
  begin();
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
// A unit of 16 rows of 512 + 64 bf16 elements is four 16-byte words a thread.
constexpr int kCopyThreads = 288;
constexpr int kCopyRows = 16;  // rows per unit of work
constexpr int kCopyUnroll = 4;

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

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(CopyParams p) {
  begin();
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
    uint4* const c = p.c_kv + layer * p.ckv_layer;
    uint4* const k = p.kpe_words > 0 ? p.k_pe + layer * p.kpe_layer : c;
    // the rows' words, both arrays' in one
    const int words = p.ckv_words + p.kpe_words, total = here * words;
    for (int i = threadIdx.x; i < total; i += kCopyUnroll * kCopyThreads) {
      uint4 v[kCopyUnroll];
      uint4* to[kCopyUnroll];
#pragma unroll
      for (int e = 0; e < kCopyUnroll; ++e) {
        const int j = i + e * kCopyThreads;
        if (j >= total) continue;
        const int r = j / words, x = j - r * words;
        const bool latent = x < p.ckv_words;
        uint4* const base = latent ? c + x : k + (x - p.ckv_words);
        const int64_t stride = latent ? p.ckv_stride : p.kpe_stride;
        v[e] = __ldcs(base + (src + r) * stride);
        to[e] = base + (dst + r) * stride;
      }
#pragma unroll
      for (int e = 0; e < kCopyUnroll; ++e)
        if (i + e * kCopyThreads < total) __stcs(to[e], v[e]);
    }
  }
}

}  // namespace

size_t pages_workspace(const tv_page_pool& p) { return 3 * ws_array(p.num_pages) + 256; }

cudaError_t launch_pages_reserve(const tv_page_pool& p, const int32_t* length,
                                 const int32_t* new_length, int32_t* copies, int32_t* status,
                                 void* ws, cudaStream_t st) {
  return launch(reserve_kernel, kCluster, kThreads, st, p, split(ws, p.num_pages), length,
                new_length, copies, status);
}

cudaError_t launch_pages_fork(const tv_page_pool& p, const int32_t* fork_from,
                              const int32_t* length, int32_t* status, cudaStream_t st) {
  return launch(fork_kernel, p.rows, 128, st, p, fork_from, length, status);
}

cudaError_t launch_pages_release(const tv_page_pool& p, const int32_t* keep, int32_t* status,
                                 cudaStream_t st) {
  return launch(release_kernel, p.rows, 128, st, p, keep, status);
}

cudaError_t launch_pages_compact(const tv_page_pool& p, int32_t* moves, int32_t* n_moves,
                                 int32_t* status, void* ws, cudaStream_t st) {
  const Workspace w = split(ws, p.num_pages);
  cudaError_t e = launch(compact_plan_kernel, kCluster, kThreads, st, p, w, moves, n_moves);
  if (e != cudaSuccess) return e;
  return launch(compact_tables_kernel, p.rows, 256, st, p, w, status);
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
  // 24 CTAs per SM, several waves of them: 3.9k pages of two layers (1.16 GB moved) took 192 us
  // with 7, 179 with 12, 172 with 24 and 217 with a CTA per unit of the list's capacity
  const int64_t grid = std::min<int64_t>(units, 24ll * current_sm_count());
  return launch(copy_kernel, grid, kCopyThreads, st, p);
}

}  // namespace tv
