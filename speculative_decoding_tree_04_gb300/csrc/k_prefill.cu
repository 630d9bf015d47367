// k_prefill.cu -- causal latent attention of prompts in its expanded form (tv_prefill_attn).
//
// For head h, key j of a sequence is k_j = W_uk[h] c_j (d_nope) with the rope part k_pe_j
// that all heads share, and value j is v_j = W_uv[h] c_j.  Query i (at key P + i) takes
//   out_i = sum_{j <= P+i} softmax_j( scale (q_nope.k_j + q_pe.k_pe_j) ) v_j.
// Per (query, key) pair and head that is 2 (128 + 64 + 128) = 640 flop, against
// 2 (2*512 + 64) = 2176 with the query absorbed into the latent space (tv_verify_attn);
// the expansion costs 2*512*256 flop per key and head once, whatever the number of queries.
// So it pays from about 170 queries per key sweep on; below that the absorbed form is
// cheaper.
//
// Four kernels:
//   plan     one block: where each sequence's expanded keys go, the tiles of the others;
//   expand   [K | V] = C W^T for every sequence and head, a GEMM of 128 keys x 256 outputs
//            x d_latent, rounded into the workspace to 16 bits (what the tensor cores read):
//            K to bf16, the type of the queries it meets, V to fp16 (three bits more); rows
//            behind a sequence's last key are zero, so that masked weights (zero) times them
//            is zero;
//   attend   per head and 256 queries, an online softmax over 128 keys at a time; where that
//            leaves SMs idle, the keys are cut into pieces that
//   join     puts together.
//
// Both tensor-core kernels are warp-specialised: one thread issues TMA loads into a ring of
// 128-byte-swizzled tiles, one (attend: two in turns) issues tcgen05.mma with accumulators in
// TMEM, whole warps read TMEM.  Every wait is bounded by a deadline, after which the kernel
// records TV_ERR_TIMEOUT, waits for its own copies and MMAs, frees TMEM and returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>
#include <mutex>

#include "sm100_ptx.h"
#include "tv_internal.h"

namespace tv {
namespace {

using namespace ptx;

constexpr int kDN = 128, kDR = 64, kDV = 128;   // per-head widths
static_assert(kDN == kDV, "K and V of the workspace have one shape");
constexpr int kKV = kDN + kDV;                  // outputs of the expansion per head
constexpr int kBlock = 128;                     // keys per block, queries per tile
constexpr int kPair = 2 * kBlock;               // queries per CTA
constexpr int kChunk = kBlock * 128;            // 128 rows of 64 bf16: 16 KB
constexpr long long kDeadline = 4000000000ll;   // clocks of a wait: about 2 s
constexpr int kAllLoads = INT_MAX;
constexpr float kLift = 7.0f, kRescale = 15.0f;  // log2: see attend_kernel
constexpr float kMaxV = 65504.f;                // the largest fp16

// ---- workspace --------------------------------------------------------------------------
// counts {query tiles, key tiles, pieces, whether any tile is cut}; query tiles {first row of
// q, rows left, position of the first row, first expanded key}; key tiles {sequence, first key,
// expanded row, rows left}; where items may be cut, pieces {query tile, number, of how many}
// and each query tile's {first piece, pieces}; then K [H][cap][128] in bf16, V [H][cap][128] in fp16 and the rope keys [cap][64]; and,
// where items may be cut, a piece's unnormalised output [256][128] and its rows' maximum and
// sum [256][2], in floats, for each SM.
struct Layout {
  int64_t cap;               // expanded key rows
  int64_t max_q, max_k;      // tiles at most
  bool cut;                  // few items: their keys may be cut into pieces
  size_t q_tiles, k_tiles, pieces, tile_pieces, k, v, kr, part_o, part_ml, total;
};
size_t align1k(size_t n) { return (n + 1023) / 1024 * 1024; }
Layout layout(const tv_prefill_args* a, int sm_count) {
  Layout l{};
  l.cap = (a->total_kv + (int64_t)(kBlock - 1) * a->B + kBlock - 1) / kBlock * kBlock;
  l.max_k = l.cap / kBlock;
  l.max_q = a->T / kPair + a->B;
  size_t n = 1024;
  l.q_tiles = n;
  n += align1k((size_t)l.max_q * sizeof(int4));
  l.k_tiles = n;
  n += align1k((size_t)l.max_k * sizeof(int4));
  l.cut = l.max_q * a->H < sm_count;
  l.pieces = n;
  if (l.cut) n += align1k((size_t)sm_count * sizeof(int4));
  l.tile_pieces = n;
  if (l.cut) n += align1k((size_t)sm_count * sizeof(int2));
  l.k = n;
  n += (size_t)l.cap * a->H * kDN * 2;
  l.v = n;
  n += (size_t)l.cap * a->H * kDV * 2;
  l.kr = n;
  n += (size_t)l.cap * kDR * 2;
  l.part_o = n;
  if (l.cut) n += (size_t)sm_count * kPair * kDV * 4;
  l.part_ml = n;
  if (l.cut) n += (size_t)sm_count * kPair * 2 * 4;
  l.total = n;
  return l;
}

// ---- plan -------------------------------------------------------------------------------
struct PlanArgs {
  const int32_t* q_start;
  const int32_t* prefix_len;
  int32_t B, T, max_q_len, max_kv_len;
  int32_t max_q, max_k, H, slots;  // slots: SMs if items may be cut, else 0
  int32_t* counts;
  int4* q_tiles;
  int4* k_tiles;
  int4* pieces;
  int2* tile_pieces;
  int32_t* status;
};

// Key blocks that a query tile's rows see.
__device__ __forceinline__ int blocks_of(int4 q_tile) {
  return (q_tile.z + min(q_tile.y, kPair) + kBlock - 1) / kBlock;
}

__global__ void __launch_bounds__(1024) plan_kernel(PlanArgs p) {
  __shared__ int s_q[32], s_k[32], s_max[32], s_base_q, s_base_k, s_base_max, s_lost;
  __shared__ int s_weight[1024];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_launch_dependents();  // the expansion may set itself up meanwhile
  if (tid == 0) {
    s_base_q = s_base_k = 0;
    s_base_max = INT_MIN;
  }
  for (int b0 = 0; b0 < p.B; b0 += 1024) {
    const int b = b0 + tid;
    int nq = 0, nk = 0, q0 = 0, n = 0, P = 0;
    // a sequence that starts below an earlier start would share rows with another one
    int top = b < p.B ? p.q_start[b] : INT_MIN;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) top = max(top, __shfl_up_sync(0xffffffffu, top, o));
    if (lane == 31) s_max[warp] = top;
    __syncthreads();
    top = max(top, s_base_max);
    for (int w = 0; w < warp; ++w) top = max(top, s_max[w]);
    __syncthreads();
    if (tid == 1023) s_base_max = top;
    if (b < p.B) {
      const int64_t s = p.q_start[b], e = p.q_start[b + 1], pre = p.prefix_len[b];
      // a bad sequence is left out: its rows stay as they were
      if (s < 0 || s < top || e < s || e > p.T || pre < 0 || e - s > p.max_q_len ||
          (e > s && pre + e - s > p.max_kv_len)) {
        report(p.status, TV_ERR_BOUNDS);
      } else if (e > s) {
        q0 = (int)s;
        n = (int)(e - s);
        P = (int)pre;
        nq = (n + kPair - 1) / kPair;
        nk = (int)((pre + n + kBlock - 1) / kBlock);  // (of up to 2^31 - 1 keys)
      }
    }
    int cq = nq, ck = nk;  // inclusive sums within the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int uq = __shfl_up_sync(0xffffffffu, cq, o), uk = __shfl_up_sync(0xffffffffu, ck, o);
      if (lane >= o) {
        cq += uq;
        ck += uk;
      }
    }
    if (lane == 31) {
      s_q[warp] = cq;
      s_k[warp] = ck;
    }
    __syncthreads();
    int bq = s_base_q + cq - nq, bk = s_base_k + ck - nk;
    for (int w = 0; w < warp; ++w) {
      bq += s_q[w];
      bk += s_k[w];
    }
    __syncthreads();
    if (tid == 1023) {
      s_base_q = bq + nq;
      s_base_k = bk + nk;
    }
    // past the caller's bounds: left out (and, counts being cumulative, all after it too)
    const bool fits = bq + nq <= p.max_q && bk + nk <= p.max_k;
    if (nq > 0 && !fits) report(p.status, TV_ERR_BOUNDS);
    if (nq > 0 && fits) {
      for (int i = 0; i < nq; ++i)
        p.q_tiles[bq + i] = make_int4(q0 + i * kPair, n - i * kPair, P + i * kPair, bk * kBlock);
      for (int i = 0; i < nk; ++i)
        p.k_tiles[bk + i] =
            make_int4(b, i * kBlock, (bk + i) * kBlock, P + n - i * kBlock);
    }
    const uint32_t lost = __ballot_sync(0xffffffffu, nq > 0 && !fits);
    // the counts end at the first sequence that does not fit
    if (tid == 0) s_lost = INT_MAX;
    __syncthreads();
    if (lost && lane == __ffs(lost) - 1) atomicMin(&s_lost, b);
    __syncthreads();
    if (s_lost != INT_MAX) {
      if (b == s_lost) {
        s_base_q = bq;
        s_base_k = bk;
      }
      __syncthreads();
      break;
    }
  }
  __syncthreads();
  const int total_q = s_base_q, total_k = s_base_k;
  if (tid == 0) {
    p.counts[0] = total_q;
    p.counts[1] = total_k;
    if (!p.slots) {
      p.counts[2] = total_q;
      p.counts[3] = 0;
    }
  }
  // longest sweeps first, so that the short ones fill the end (up to 1024 tiles)
  if (total_q > 1024) return;
  int4 mine = make_int4(0, 0, 0, 0);
  __syncthreads();
  if (tid < total_q) {
    mine = p.q_tiles[tid];
    s_weight[tid] = mine.z + min(mine.y, kPair);
  }
  __syncthreads();
  int rank = 0;
  if (tid < total_q) {
    const int w = s_weight[tid];
    for (int i = 0; i < total_q; ++i)
      rank += s_weight[i] > w || (s_weight[i] == w && i < tid);
    p.q_tiles[rank] = mine;
  }
  if (!p.slots) return;
  // Few items (total_q * H < slots): the least length, of four blocks at least, at which all
  // pieces have an SM each; then every tile in equal pieces of that length at most.  (The same
  // number of pieces for every tile left the longest one's twice the mean: 4 chunks of 256
  // queries after 2048 to 6000 keys, 16 heads: attend 62 us, 47 with this.)
  __syncthreads();
  if (tid < total_q) s_weight[rank] = blocks_of(mine);
  __syncthreads();
  if (warp > 0) return;
  const int most = p.slots / p.H;
  auto count = [&](int length) {
    int n = 0;
    for (int i = lane; i < total_q; i += 32) n += (s_weight[i] + length - 1) / length;
    return __reduce_add_sync(0xffffffffu, n);
  };
  int lo = 4, hi = max(4, total_q > 0 ? s_weight[0] : 0);  // at hi, a piece per tile
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (count(mid) <= most) hi = mid;
    else lo = mid + 1;
  }
  int first = 0;
  for (int i0 = 0; i0 < total_q; i0 += 32) {
    const int i = i0 + lane, n = i < total_q ? (s_weight[i] + hi - 1) / hi : 0;
    int up_to = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int below = __shfl_up_sync(0xffffffffu, up_to, o);
      if (lane >= o) up_to += below;
    }
    if (i < total_q) p.tile_pieces[i] = make_int2(first + up_to - n, n);
    for (int k = 0; k < n; ++k) p.pieces[first + up_to - n + k] = make_int4(i, k, n, 0);
    first += __shfl_sync(0xffffffffu, up_to, 31);
  }
  if (lane == 0) {
    p.counts[2] = first;
    p.counts[3] = first > total_q;
  }
}

// ---- bounded waits ------------------------------------------------------------------------
// What a test may change (tv_testing_set_prompt_fault): how many loads a CTA issues, the
// waits' deadline, and where CTAs count as they leave, {all, those that gave up}.
struct WaitFault {
  int32_t loads;
  long long deadline;
  int32_t* exits;
};
struct Abort {
  volatile int flag;
  int32_t* status;
  long long deadline;
};
__device__ __forceinline__ void count_exit(const WaitFault& f, const Abort& ab) {
  if (!f.exits || threadIdx.x != 0) return;
  atomicAdd(f.exits, 1);
  if (ab.flag) atomicAdd(f.exits + 1, 1);
}

__device__ __noinline__ bool wait_slow(Abort& ab, uint32_t a, uint32_t parity) {
  // the SM's own clock: reading the global timer takes about as long as these waits do
  const long long t0 = clock64();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait_plain(a, parity)) return true;
    if (ab.flag) return false;
    if (clock64() - t0 > ab.deadline) {
      ab.flag = 1;
      report(ab.status, TV_ERR_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_for(Abort& ab, uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait_plain(a, parity)) return true;
  return wait_slow(ab, a, parity);
}
// Whether or not the kernel is giving up: a copy or MMA in flight has to land first.
__device__ __noinline__ void drain(Abort& ab, uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  const long long t0 = clock64();
  while (!mbar_try_wait_plain(a, parity))
    if (clock64() - t0 > kDeadline) {
      report(ab.status, TV_ERR_TIMEOUT);
      return;
    }
}
__device__ __forceinline__ void drain_ring(Abort& ab, uint64_t* full, uint32_t stages,
                                           uint32_t count) {
  for (uint32_t k = 0; k < stages && k < count; ++k) {
    const uint32_t u = count - 1 - k;
    drain(ab, &full[u % stages], (u / stages) & 1);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
// 32 bytes in one store (sm_100)
__device__ __forceinline__ void st_global_32(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// ---- expand -------------------------------------------------------------------------------
// 128 keys x 256 outputs per tile, the contraction in steps of 64 through four stages, two
// accumulators so that a tile's rounding and stores run beside the next one's MMAs; tiles go
// head by head, so that a head's 256 KB of weights stay in L2.  4096 keys, 64 heads (69 GFLOP):
// 57 us, 61 % of the measured cuBLAS rate.  Without its stores 45, without its loads 45: operand
// reads, incoming tiles and outgoing rows share one limit, the SM's path to shared memory and
// L1.  Slower: pairs of SMs on one tile (61), key rows kept in shared memory (62), a 256 x 256
// tile with a single accumulator (74).
constexpr int kExpThreads = 256;
constexpr int kExpStages = 4;
constexpr int kExpA = kChunk, kExpB = kKV * 128;  // 16 KB of keys, 32 KB of weights
constexpr int kExpStage = kExpA + kExpB;
constexpr uint32_t kIdescExp = idesc_bf16_f32(kBlock, kKV, 0, 0);

struct ExpandShared {
  uint64_t full[kExpStages], empty[kExpStages], acc_full[2], acc_empty[2], last;
  uint32_t tmem;
  Abort abort;
};
constexpr int kExpSmem = kExpStages * kExpStage + (int)sizeof(ExpandShared);

struct ExpandArgs {
  const int32_t* counts;
  const int4* k_tiles;
  const int32_t* page_table;  // null: contiguous
  int32_t max_pages, H, k_chunks;
  int64_t kv_stride_b, num_rows, cap;
  const __nv_bfloat16* k_pe;
  int64_t kpe_stride;
  __nv_bfloat16 *K, *KR;
  __half* V;
  int32_t* status;
  WaitFault fault;
};

// First cache row of 64 keys, or a row past the end (TMA then reads zeros) for a page that
// is not in the cache.
__device__ __forceinline__ int64_t cache_row64(const ExpandArgs& p, int b, int64_t key) {
  if (!p.page_table) return (int64_t)b * p.kv_stride_b + key;
  const int64_t row = (int64_t)__ldg(p.page_table + (int64_t)b * p.max_pages + key / 64) * 64;
  return row >= 0 && row + 64 <= p.num_rows ? row : p.num_rows;
}

__global__ void __launch_bounds__(kExpThreads, 1)
    expand_kernel(ExpandArgs p, const __grid_constant__ CUtensorMap map_c,
                  const __grid_constant__ CUtensorMap map_w) {
  extern __shared__ __align__(1024) unsigned char smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles need it
    if (threadIdx.x == 0) report(p.status, TV_ERR_UNSUPPORTED);
    return;
  }
  ExpandShared& sh = *(ExpandShared*)(smem + kExpStages * kExpStage);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kExpStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.acc_full[i], 1);
      mbar_init(&sh.acc_empty[i], 4);
    }
    mbar_init(&sh.last, 1);
    sh.abort.flag = 0;
    sh.abort.status = p.status;
    sh.abort.deadline = p.fault.deadline;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  griddep_launch_dependents();
  griddep_wait();  // the plan
  const int n_k = p.counts[1];
  const int64_t n_tiles = (int64_t)n_k * p.H;

  if (warp == 0 && lane == 0) {
    fence_proxy_async_global();
    uint32_t u = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; ok && t < n_tiles; t += gridDim.x) {
      const int h = (int)(t / n_k);
      const int4 kt = p.k_tiles[t - (int64_t)h * n_k];
      // the second half may hold no key: read past the end then (its page may not exist)
      const int row0 = (int)min(cache_row64(p, kt.x, kt.y), p.num_rows);
      const int row1 = kt.w > 64 ? (int)min(cache_row64(p, kt.x, kt.y + 64), p.num_rows)
                                 : (int)p.num_rows;
      for (int c = 0; c < p.k_chunks; ++c, ++u) {
        const uint32_t s = u % kExpStages;
        if (u >= (uint32_t)p.fault.loads ||
            !wait_for(sh.abort, &sh.empty[s], ((u / kExpStages) & 1) ^ 1)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&sh.full[s], kExpStage);
        unsigned char* a = smem + s * kExpStage;
        tma_load_2d(a, &map_c, 64 * c, row0, &sh.full[s]);
        tma_load_2d(a + kExpA / 2, &map_c, 64 * c, row1, &sh.full[s]);
        tma_load_2d(a + kExpA, &map_w, 64 * c, h * kKV, &sh.full[s]);
      }
    }
    drain_ring(sh.abort, sh.full, kExpStages, u);
  } else if (warp == 1 && lane == 0) {
    uint32_t u = 0, i = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; ok && t < n_tiles; t += gridDim.x, ++i) {
      const uint32_t buf = i & 1;
      ok = wait_for(sh.abort, &sh.acc_empty[buf], ((i >> 1) & 1) ^ 1);
      tc_fence_after();
      for (int c = 0; ok && c < p.k_chunks; ++c, ++u) {
        const uint32_t s = u % kExpStages;
        if (!wait_for(sh.abort, &sh.full[s], (u / kExpStages) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a = smem_u32(smem + s * kExpStage);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ss(tmem + buf * kKV, smem_desc(a + 32 * k, 16, 1024, 2),
                 smem_desc(a + kExpA + 32 * k, 16, 1024, 2), kIdescExp, (c | k) != 0);
        mma_commit(&sh.empty[s]);
      }
      if (ok) mma_commit(&sh.acc_full[buf]);
    }
    mma_commit(&sh.last);
    drain(sh.abort, &sh.last, 0);
  } else if (warp >= 4) {
    const int r = tid - 128;  // row of the tile = TMEM lane
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // 32 lanes per warp, lane field << 16
    uint32_t i = 0;
    for (int64_t t = blockIdx.x; t < n_tiles; t += gridDim.x, ++i) {
      const int h = (int)(t / n_k);
      const int4 kt = p.k_tiles[t - (int64_t)h * n_k];
      const bool live = r < kt.w;
      if (h == 0) {  // the rope keys, once per key tile
        uint4 v[8] = {};
        if (live) {
          const int64_t row = cache_row64(p, kt.x, kt.y + (r & 64)) + (r & 63);
          if (row < p.num_rows) {
            const uint4* src = reinterpret_cast<const uint4*>(p.k_pe + row * p.kpe_stride);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = __ldg(src + k);
          } else {
            report(p.status, TV_ERR_BOUNDS);
          }
        }
        uint4* dst = reinterpret_cast<uint4*>(p.KR + ((int64_t)kt.z + r) * kDR);
#pragma unroll
        for (int k = 0; k < 8; ++k) dst[k] = v[k];
      }
      const uint32_t buf = i & 1;
      if (!__all_sync(0xffffffffu, wait_for(sh.abort, &sh.acc_full[buf], (i >> 1) & 1))) break;
      tc_fence_after();
      const int64_t at = (int64_t)h * p.cap + kt.z + r;
      float big = 0.f;
#pragma unroll
      for (int c = 0; c < kKV; c += 32) {
        uint32_t x[32];
        tmem_ld32(tmem + lanes + buf * kKV + c, x);
        tmem_wait_ld_regs(x);
        uint32_t y[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          float a = __uint_as_float(x[2 * k]), b = __uint_as_float(x[2 * k + 1]);
          if (c >= kDN) {
            big = abs_max3_nan(big, a, b);
            a = fminf(fmaxf(a, -kMaxV), kMaxV);
            b = fminf(fmaxf(b, -kMaxV), kMaxV);
          }
          y[k] = !live ? 0u : c < kDN ? pack_bf16(a, b) : pack_f16(a, b);
        }
        void* dst = c < kDN ? (void*)(p.K + at * kDN + c) : (void*)(p.V + at * kDV + (c - kDN));
        st_global_32(dst, y);
        st_global_32((char*)dst + 32, y + 8);
      }
      if (live && !(big <= kMaxV)) report(p.status, TV_ERR_BOUNDS);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.acc_empty[buf]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
  count_exit(p.fault, sh.abort);
}

// ---- attend -------------------------------------------------------------------------------
// Persistent CTAs; an item of work is one head and up to 256 queries as two 128-row tiles
// that share every key block.  TMEM (512 columns): S0, S1 (128 each; P, in fp16, overwrites
// the first half of its S) and O0, O1.  The tiles take turns at the tensor cores: a tile's MMAs
// run while the other tile's softmax does.  Per tile and block these
// are 12 of 128x128x16 for S and 8 for O, 1280 clocks at the full rate, against 16384
// exponentials.  Sixteen warps do the softmax, eight per tile, 16 rows each: the 16x256b
// TMEM shape spreads a row over four lanes, which meet in two shuffles.
//   4096 queries, 64 heads (344 GFLOP, causal): 253-260 us, 68 % of the measured cuBLAS rate.
// With one issuing thread for both tiles its waits and commits stood between the MMAs; with two
// that do not take turns the tiles fall into step and wait on the tensor cores together.
constexpr int kAttThreads = 640;
constexpr int kRing = 8;  // 16 KB chunks, 5 per key block: K and V of 1.6 blocks
constexpr int kQBytes = 3 * kChunk;
constexpr int kPassAt = 2;  // of the three chunks of a block of scores
constexpr uint32_t kTmS = 0, kTmO = 256;
constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, 0, 0);
// the same with fp16 operands (type fields 0)
constexpr uint32_t kIdescO = idesc_bf16_f32(128, 128, 0, 1) & ~((1u << 7) | (1u << 10));

struct AttendShared {
  uint64_t k_full[2], v_full[2], k_done[2], v_done[2];  // of a block, by its parity
  uint64_t q_full, s_full[2], p_full[2], o_full[2], o_free[2], turn[2], last[2];
  uint32_t tmem;
  Abort abort;
};
constexpr int kAttSmem = 2 * kQBytes + kRing * kChunk + (int)sizeof(AttendShared);
static_assert(kAttSmem <= 232448, "shared memory of an SM");

struct AttendArgs {
  const int32_t* counts;
  const int4* q_tiles;
  const int4* pieces;  // null: a piece per tile
  const int2* tile_pieces;
  int32_t H;
  float scale_log2;
  __nv_bfloat16* out;
  float* part_o;   // [piece][256][128]
  float* part_ml;  // [piece][256][2]
  int32_t* status;
  WaitFault fault;
};

// The r-th item of this CTA: a head of a query tile's piece.  Items are listed longest first
// and dealt in rounds of alternating direction.  (Dealt from a counter as CTAs become free, a
// ragged batch's attend took 134 us instead of 136, but 4096 queries of 64 heads 265 instead of
// 257.)
struct Item {
  bool some;
  int slot;                       // its place in the list
  int pieces;                     // of its query tile
  int h, row0, rows, pos0, key0, tiles;
  int j0, n0, n1;                 // first key block; blocks from there that a tile's rows see
};
__device__ __forceinline__ Item item_of(const AttendArgs& p, int total, int r) {
  Item it;
  const int64_t i =
      (int64_t)r * gridDim.x + ((r & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  it.some = i < total;
  if (!it.some) return it;
  it.slot = (int)i;
  int tile = it.slot / p.H, piece = 0;
  it.h = it.slot - tile * p.H;
  it.pieces = 1;
  if (p.pieces) {
    const int4 e = p.pieces[tile];
    tile = e.x;
    piece = e.y;
    it.pieces = e.z;
  }
  const int4 qt = p.q_tiles[tile];
  it.row0 = qt.x;
  it.rows = min(qt.y, kPair);
  it.pos0 = qt.z;
  it.tiles = it.rows > kBlock ? 2 : 1;
  const int n0 = (it.pos0 + min(it.rows, kBlock) + kBlock - 1) / kBlock;
  const int n1 = it.tiles > 1 ? (it.pos0 + it.rows + kBlock - 1) / kBlock : 0;
  const int n = max(n0, n1), j1 = (int)((int64_t)n * (piece + 1) / it.pieces);
  it.j0 = (int)((int64_t)n * piece / it.pieces);
  it.n0 = max(0, min(n0, j1) - it.j0);
  it.n1 = max(0, min(n1, j1) - it.j0);
  it.key0 = qt.w + it.j0 * kBlock;
  return it;
}

// Among the four lanes that share rows: lane q gives its words x[2 d], x[2 d + 1] to lane d
// and gets y[r], y[4 + r] from lane r.
__device__ __forceinline__ void exchange4(uint32_t* x, uint32_t* y) {
  const int q = threadIdx.x & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int a = (i & 2) * 2 + (i & 1), b = a + 2;
    const uint32_t got = __shfl_xor_sync(0xffffffffu, (q & 1) ? x[a] : x[b], 1);
    if (q & 1) x[a] = got;
    else x[b] = got;
  }
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int b = a + 4;
    const uint32_t got = __shfl_xor_sync(0xffffffffu, (q & 2) ? x[a] : x[b], 2);
    if (q & 2) x[a] = got;
    else x[b] = got;
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    y[r] = x[2 * r];
    y[4 + r] = x[2 * r + 1];
  }
}

__global__ void __launch_bounds__(kAttThreads, 1)
    attend_kernel(AttendArgs p, const __grid_constant__ CUtensorMap map_q,
                  const __grid_constant__ CUtensorMap map_qr,
                  const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v,
                  const __grid_constant__ CUtensorMap map_kr) {
  extern __shared__ __align__(1024) unsigned char smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles need it
    if (threadIdx.x == 0) report(p.status, TV_ERR_UNSUPPORTED);
    return;
  }
  unsigned char* ring = smem + 2 * kQBytes;
  AttendShared& sh = *(AttendShared*)(ring + kRing * kChunk);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(&sh.q_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.v_full[i], 1);
      mbar_init(&sh.k_done[i], 2);  // one for each tile
      mbar_init(&sh.v_done[i], 2);
      mbar_init(&sh.turn[i], 1);
      mbar_init(&sh.last[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 8);
      mbar_init(&sh.o_full[i], 1);
      mbar_init(&sh.o_free[i], 8);
    }
    sh.abort.flag = 0;
    sh.abort.status = p.status;
    sh.abort.deadline = p.fault.deadline;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  // Only the join may start beside this kernel.  Where none follows, the next kernel is another
  // call's, and one that works before its own wait (an attention call's preparation under
  // overlap_prev) may have been given the same workspace.
  if (p.pieces) griddep_launch_dependents();
  griddep_wait();  // the plan and the expanded keys
  const int total = p.counts[2] * p.H;

  if (warp == 0 && lane == 0) {
    fence_proxy_async_global();
    // Block g (counted over all items) has the ring entries 5g .. 5g+4: K nope, K nope, K
    // rope (128 keys of 64 elements each), V, V (64 keys of 128 elements each, as two
    // 64-wide column pieces).  An entry is free again when the block it last held a part of
    // is done with.
    bool ok = true;
    int g = 0, items = 0, armed_k = 0, armed_v = 0;
    for (int r = 0; ok; ++r) {
      const Item it = item_of(p, total, r);
      if (!it.some) break;
      // the last block of scores of the item before frees the queries
      if (g > 0) ok = wait_for(sh.abort, &sh.k_done[(g - 1) & 1], ((g - 1) >> 1) & 1);
      if (!ok) break;
      mbar_arrive_expect_tx(&sh.q_full, it.tiles * kQBytes);
      ++items;
      for (int t = 0; t < it.tiles; ++t) {
        unsigned char* q = smem + t * kQBytes;
        const int row = it.row0 + t * kBlock;
        tma_load_3d(q, &map_q, 0, it.h, row, &sh.q_full);
        tma_load_3d(q + kChunk, &map_q, 64, it.h, row, &sh.q_full);
        tma_load_3d(q + 2 * kChunk, &map_qr, 0, it.h, row, &sh.q_full);
      }
      const int n = max(it.n0, it.n1);
      for (int j = 0; ok && j < n; ++j, ++g) {
        const int key = it.key0 + j * kBlock;
        uint64_t* kb = &sh.k_full[g & 1];
        uint64_t* vb = &sh.v_full[g & 1];
#pragma unroll 1
        for (int c = 0; c < 5; ++c) {
          const uint32_t u = 5u * g + c;
          if ((c == 0 || c == 3) && armed_k + armed_v >= p.fault.loads) ok = false;
          if (ok && u >= (uint32_t)kRing) {
            const uint32_t before = u - kRing, gb = before / 5;
            uint64_t* done = before - 5 * gb < 3 ? &sh.k_done[gb & 1] : &sh.v_done[gb & 1];
            ok = wait_for(sh.abort, done, (gb >> 1) & 1);
          }
          // giving up, but what a barrier has been armed for still has to come
          if (!ok && (c == 0 || c == 3)) break;
          unsigned char* dst = ring + (u % kRing) * kChunk;
          if (c == 0) {
            mbar_arrive_expect_tx(kb, 3 * kChunk);
            ++armed_k;
          } else if (c == 3) {
            mbar_arrive_expect_tx(vb, 2 * kChunk);
            ++armed_v;
          }
          if (c < 2) tma_load_3d(dst, &map_k, 64 * c, key, it.h, kb);
          else if (c == 2) tma_load_2d(dst, &map_kr, 0, key, kb);
          else tma_load_4d(dst, &map_v, 0, key + 64 * (c - 3), 0, it.h, vb);
        }
      }
    }
    if (items > 0) drain(sh.abort, &sh.q_full, (items - 1) & 1);
    drain_ring(sh.abort, sh.k_full, 2, armed_k);
    drain_ring(sh.abort, sh.v_full, 2, armed_v);
  } else if (warp == 1 || warp == 2) {
    // One issuing warp per tile; they hand each other the turn, so that a tile's MMAs run
    // while the other tile's softmax does, and a warp's own waits and commits fall into the
    // other's turn.  The warp stays in step, its counters and descriptors uniform; one lane
    // issues.
    const int t = warp - 1;
    const uint32_t lead = lane == 0;
    const uint32_t q = smem_u32(smem) + t * kQBytes, ring0 = smem_u32(ring);
    const uint32_t ts = kTmS + 128 * t, to = kTmO + 128 * t;
    int g = 0;      // blocks before this item
    int sc = 0;     // this tile's softmax turns before this item
    int oc = 0;     // items with this tile
    int turns = 0;  // turns taken
    auto chunk = [&](uint32_t u) { return ring0 + (u % kRing) * kChunk; };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wait_for(sh.abort, bar, parity)) != 0;
    };
    auto take_turn = [&](bool shared) {
      if (!shared) return true;
      ++turns;
      return t == 0 ? turns == 1 || wait(&sh.turn[0], (turns - 2) & 1)
                    : wait(&sh.turn[1], (turns - 1) & 1);
    };
    auto pass_turn = [&](bool shared) {
      if (shared && lead) mbar_arrive(&sh.turn[t ^ 1]);
    };
    auto scores = [&](int gj, bool both) {
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        if (c == kPassAt) pass_turn(both);  // its way there takes about as long as the rest
        const uint64_t dq = smem_desc(q + c * kChunk, 16, 1024, 2);
        const uint64_t dk = smem_desc(chunk(5u * gj + c), 16, 1024, 2);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ss_lead(lead, ts, dq + 2 * k, dk + 2 * k, kIdescS, (c | k) != 0);
      }
      mma_commit_lead(lead, &sh.s_full[t]);
    };
    // this tile is done with a block's keys or values (an item's only tile counts twice)
    auto done = [&](uint64_t* bar, bool only) {
      mma_commit_lead(lead, bar);
      if (only) mma_commit_lead(lead, bar);
    };
    bool ok = tmem == 0;  // 512 of 512 columns: the addresses above are absolute
    for (int r = 0; ok; ++r) {
      const Item it = item_of(p, total, r);
      if (!it.some) break;
      const int n0 = __reduce_max_sync(0xffffffffu, it.n0);
      const int n1 = __reduce_max_sync(0xffffffffu, it.n1);
      const int nt = t ? n1 : n0, n = max(n0, n1);
      const bool both = n1 > 0;
      if (t == 0 ? n > 0 : both) {
        ok = wait(&sh.q_full, r & 1) && wait(&sh.k_full[g & 1], (g >> 1) & 1) && take_turn(both);
        if (!ok) break;
        tc_fence_after();
        if (nt > 0) {
          scores(g, both);
          done(&sh.k_done[g & 1], !both);
        } else {
          pass_turn(both);
        }
        for (int j = 0; ok && j < nt; ++j) {
          const int gj = g + j;
          ok = wait(&sh.v_full[gj & 1], (gj >> 1) & 1) &&
               (j > 0 || oc == 0 || wait(&sh.o_free[t], (oc - 1) & 1)) &&
               wait(&sh.p_full[t], (sc + j) & 1) && take_turn(both);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dv0 = smem_desc(chunk(5u * gj + 3), kChunk / 2, 1024, 2);
          const uint64_t dv1 = smem_desc(chunk(5u * gj + 4), kChunk / 2, 1024, 2);
#pragma unroll
          for (int k = 0; k < 8; ++k)  // the keys are the contraction: V is an MN-major B
            mma_ts_lead(lead, to, ts + 8 * k, (k < 4 ? dv0 : dv1) + 128 * (k & 3), kIdescO,
                        (j | k) != 0);
          if (j + 1 < nt) {
            done(&sh.v_done[gj & 1], !both);
            ok = wait(&sh.k_full[(gj + 1) & 1], ((gj + 1) >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            scores(gj + 1, both);
            done(&sh.k_done[(gj + 1) & 1], !both);
          } else {
            mma_commit_lead(lead, &sh.o_full[t]);
            pass_turn(both);
            done(&sh.v_done[gj & 1], !both);
          }
        }
        // The first tile may end before the second: it passes its turns and lets go of those
        // blocks.  Their barriers' phase before (two blocks back) has to be over, or the
        // arrival would count for that one.
        for (int j = nt; ok && j < n; ++j) {
          const int gj = g + j;
          ok = take_turn(both) &&
               (gj < 2 || (wait(&sh.k_done[gj & 1], ((gj >> 1) & 1) ^ 1) &&
                           wait(&sh.v_done[gj & 1], ((gj >> 1) & 1) ^ 1)));
          if (!ok) break;
          pass_turn(both);
          if (lead) {
            mbar_arrive(&sh.k_done[gj & 1]);
            mbar_arrive(&sh.v_done[gj & 1]);
          }
        }
      }
      g += n;
      sc += nt;
      oc += nt > 0;
    }
    if (tmem != 0 && lane == 0) {
      report(p.status, TV_ERR_CUDA);
      sh.abort.flag = 1;
    }
    mma_commit_lead(lead, &sh.last[t]);
    if (lane == 0) drain(sh.abort, &sh.last[t], 0);
    __syncwarp();
  } else if (warp >= 4) {
    const int t = (warp - 4) >> 3, sub = ((warp - 4) >> 2) & 1;
    const int base = (warp & 3) * 32 + 16 * sub;  // first of this warp's rows = TMEM lanes
    const int ra = base + (lane >> 2);            // this thread's rows: ra and ra + 8
    const int col = 2 * (lane & 3);               // its columns: 8 i + col, 8 i + col + 1
    const uint32_t ts = tmem + ((uint32_t)base << 16) + kTmS + 128 * t;
    const uint32_t to = tmem + ((uint32_t)base << 16) + kTmO + 128 * t;
    const float c = p.scale_log2;
    const uint64_t c2 = f2_pack(c, c);
    int sc = 0, oc = 0;
    bool ok = true;
    for (int r = 0; ok; ++r) {
      int nt, tile_first;  // every row of the tile sees the sweep's keys 0 .. tile_first
      {
        const Item it = item_of(p, total, r);
        if (!it.some) break;
        nt = t ? it.n1 : it.n0;
        tile_first = it.pos0 + (t - it.j0) * kBlock;
        if (nt == 0) {
          if (it.pieces > 1 && t < it.tiles && (lane & 3) == 0) {  // nothing of these rows here
            float* ml = p.part_ml + ((int64_t)it.slot * kPair + t * kBlock + ra) * 2;
            ml[1] = ml[17] = 0.f;  // rows ra and ra + 8
          }
          continue;
        }
      }
      float ma = 0.f, mb = 0.f;                     // 2^ma is one unit of a row's weights
      float la = 0.f, lb = 0.f;                     // sums over this thread's columns
      for (int j = 0; j < nt; ++j, ++sc) {
        ok = __all_sync(0xffffffffu, wait_for(sh.abort, &sh.s_full[t], sc & 1));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[64];  // s[4 i + e]: row ra (e < 2) or ra + 8, column 8 i + col + (e & 1)
        tmem_ld_16x256b_x8(ts, s);
        tmem_ld_16x256b_x8(ts + 64, s + 32);
        tmem_wait_ld_regs(s);
        tmem_wait_ld_regs(s + 32);
        const int k0 = j * kBlock;
        if (k0 + kBlock - 1 > tile_first) {
          const int lim = tile_first + ra - k0 - col;  // row ra sees columns 8 i + e up to it
#pragma unroll
          for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (8 * i + (e & 1) > lim + 8 * (e >> 1)) s[4 * i + e] = 0xFF800000u;
        }
        float xa = -INFINITY, ya = -INFINITY, xb = -INFINITY, yb = -INFINITY;
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          xa = fmax3(xa, __uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1]));
          xb = fmax3(xb, __uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3]));
          ya = fmax3(ya, __uint_as_float(s[4 * i + 4]), __uint_as_float(s[4 * i + 5]));
          yb = fmax3(yb, __uint_as_float(s[4 * i + 6]), __uint_as_float(s[4 * i + 7]));
        }
        xa = fmaxf(xa, ya);
        xb = fmaxf(xb, yb);
        xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 1));
        xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 1));
        xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 2)) * c;
        xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 2)) * c;
        // Weights are 2^(x - m) with m a maximum's 2^-7, so that the largest is 2^7 or more and
        // those below fp16's normal range are held to 2^-32 of it (with m the maximum itself
        // they vanished below 2^-25).  m only moves when a block's weights would exceed 2^15:
        // fp16 holds them, and the accumulator is rescaled rarely.  (A piece's first block may
        // hide all its keys from a row: m is -inf then, and taken as 0 for the weights, all
        // zero.)
        if (j == 0) {
          ma = xa - kLift;
          mb = xb - kLift;
        } else if (__any_sync(0xffffffffu, xa > ma + kRescale || xb > mb + kRescale)) {
          const float na = xa > ma + kRescale ? xa - kLift : ma;
          const float nb = xb > mb + kRescale ? xb - kLift : mb;
          const float fa = na == ma ? 1.f : ex2(ma - na), fb = nb == mb ? 1.f : ex2(mb - nb);
          ma = na;
          mb = nb;
          la *= fa;
          lb *= fb;
          // S of block j was issued after the O of block j - 1: O is complete
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            uint32_t o[16];
            tmem_ld_16x256b_x4(to + 32 * k, o);
            tmem_wait_ld_regs16(o);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              o[i] = __float_as_uint(__uint_as_float(o[i]) * ((i & 2) ? fb : fa));
            tmem_st_16x256b_x4(to + 32 * k, o);
          }
        }
        const float za = ma > -INFINITY ? -ma : 0.f, zb = mb > -INFINITY ? -mb : 0.f;
        const uint64_t m2a = f2_pack(za, za), m2b = f2_pack(zb, zb);
        uint64_t l2a = 0, l2b = 0;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pk[16];  // V's type
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t* x = s + 32 * half + 4 * i;
            float a0, a1, b0, b1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(x[0]), __uint_as_float(x[1])), c2, m2a), a0,
                      a1);
            f2_unpack(f2_fma(f2_pack(__uint_as_float(x[2]), __uint_as_float(x[3])), c2, m2b), b0,
                      b1);
            a0 = ex2(a0);
            a1 = ex2(a1);
            b0 = ex2(b0);
            b1 = ex2(b1);
            l2a = f2_add(l2a, f2_pack(a0, a1));
            l2b = f2_add(l2b, f2_pack(b0, b1));
            pk[2 * i] = pack_f16(a0, a1);
            pk[2 * i + 1] = pack_f16(b0, b1);
          }
          tmem_st_16x128b_x8(ts + 32 * half, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[t]);
        float u, v;  // the sums are those of the unrounded weights
        f2_unpack(l2a, u, v);
        la += u + v;
        f2_unpack(l2b, u, v);
        lb += u + v;
      }
      if (!ok) break;
      la += __shfl_xor_sync(0xffffffffu, la, 1);
      lb += __shfl_xor_sync(0xffffffffu, lb, 1);
      la += __shfl_xor_sync(0xffffffffu, la, 2);
      lb += __shfl_xor_sync(0xffffffffu, lb, 2);
      ok = __all_sync(0xffffffffu, wait_for(sh.abort, &sh.o_full[t], oc & 1));
      if (!ok) break;
      ++oc;
      tc_fence_after();
      const Item it = item_of(p, total, r);  // (again: not kept through the sweep)
      const int q = t * kBlock + ra;                 // rows q and q + 8 of the item
      if (it.pieces > 1) {
        const int64_t at = (int64_t)it.slot * kPair + q;
        if ((lane & 3) == 0) {
          *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(ma, la);
          *reinterpret_cast<float2*>(p.part_ml + (at + 8) * 2) = make_float2(mb, lb);
        }
        float* dst = p.part_o + at * kDV + col;
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          uint32_t o[16];
          tmem_ld_16x256b_x4(to + 32 * k, o);
          tmem_wait_ld_regs16(o);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            *reinterpret_cast<uint2*>(dst + 32 * k + 8 * i) = make_uint2(o[4 * i], o[4 * i + 1]);
            *reinterpret_cast<uint2*>(dst + 8 * kDV + 32 * k + 8 * i) =
                make_uint2(o[4 * i + 2], o[4 * i + 3]);
          }
        }
        continue;  // (the CTA's only item)
      }
      const float ia = 1.f / la, ib = 1.f / lb;
      __nv_bfloat16* dst =
          p.out + ((int64_t)(it.row0 + q) * p.H + it.h) * kDV + 16 * (lane & 3);
      const int64_t down = (int64_t)8 * p.H * kDV;
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        uint32_t o[32];
        tmem_ld_16x256b_x8(to + 64 * k, o);
        tmem_wait_ld_regs(o);
        uint32_t x[8], y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          x[i] = pack_bf16(__uint_as_float(o[4 * i]) * ia, __uint_as_float(o[4 * i + 1]) * ia);
        exchange4(x, y);
        if (q < it.rows) st_global_32(dst + 64 * k, y);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          x[i] = pack_bf16(__uint_as_float(o[4 * i + 2]) * ib, __uint_as_float(o[4 * i + 3]) * ib);
        exchange4(x, y);
        if (q + 8 < it.rows) st_global_32(dst + down + 64 * k, y);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.o_free[t]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
  count_exit(p.fault, sh.abort);
}

// ---- join ---------------------------------------------------------------------------------
// A warp per (item, query): the pieces' outputs weighted by 2^(m - M).  At most 128 KB of
// partials for each SM (20 MB), from L2.
__global__ void __launch_bounds__(256) join_kernel(AttendArgs p) {
  griddep_wait();
  if (!p.counts[3]) return;
  const int lane = threadIdx.x & 31;
  const int64_t units = (int64_t)p.counts[0] * p.H * kPair;
  for (int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); u < units; u += 8 * gridDim.x) {
    const int whole = (int)(u / kPair), q = (int)(u % kPair);
    const int tile = whole / p.H, h = whole - tile * p.H;
    const int4 qt = p.q_tiles[tile];
    const int2 tp = p.tile_pieces[tile];
    const int pieces = tp.y;
    if (q >= qt.y || pieces == 1) continue;  // (a tile in one piece is written already)
    const int64_t at = ((int64_t)tp.x * p.H + h) * kPair + q, next = (int64_t)p.H * kPair;
    float M = -INFINITY;
    for (int k = 0; k < pieces; ++k) {
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + (at + k * next) * 2);
      if (ml.y != 0.f) M = fmaxf(M, ml.x);
    }
    float l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < pieces; ++k) {
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + (at + k * next) * 2);
      if (ml.y == 0.f) continue;  // nothing visible there (its output may not exist)
      const float f = ex2(ml.x - M);
      const float4 x =
          *reinterpret_cast<const float4*>(p.part_o + (at + k * next) * kDV + 4 * lane);
      l = fmaf(ml.y, f, l);
      o[0] = fmaf(x.x, f, o[0]);
      o[1] = fmaf(x.y, f, o[1]);
      o[2] = fmaf(x.z, f, o[2]);
      o[3] = fmaf(x.w, f, o[3]);
    }
    const float inv = 1.f / l;
    *reinterpret_cast<uint2*>(p.out + ((int64_t)(qt.x + q) * p.H + h) * kDV + 4 * lane) =
        make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
  }
}

// ---- host ---------------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;
std::mutex g_mu;
bool g_ready[64] = {};
// Testing hook (tv_testing_set_prompt_fault): off unless a test turns it on.
std::mutex g_fault_mu;
WaitFault g_expand_fault = {kAllLoads, kDeadline, nullptr};
WaitFault g_attend_fault = {kAllLoads, kDeadline, nullptr};

cudaError_t setup() {
  std::call_once(g_encode_once, [] {
    cudaDriverEntryPointQueryResult q;
    void* fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (!g_encode) return cudaErrorNotSupported;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorNotSupported;
  std::lock_guard<std::mutex> lock(g_mu);
  if (!g_ready[dev]) {
    e = cudaFuncSetAttribute(expand_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kExpSmem);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(attend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kAttSmem);
    if (e != cudaSuccess) return e;
    g_ready[dev] = true;
  }
  return cudaSuccess;
}

// A 2-D to 4-D view of bf16 data, inner extent 64 per box, 128-byte swizzle.
bool make_map(CUtensorMap* m, const void* base, int rank, const uint64_t* dims,
              const uint64_t* stride_bytes, const uint32_t* box) {
  cuuint64_t d[4], s[3];
  cuuint32_t b[4], e[4] = {1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    if (i + 1 < rank) s[i] = stride_bytes[i];
  }
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), d, s, b, e,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool map2(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint64_t stride,
          uint32_t box_rows) {
  const uint64_t d[2] = {inner, rows}, s[1] = {stride};
  const uint32_t b[2] = {64, box_rows};
  return make_map(m, base, 2, d, s, b);
}

}  // namespace

size_t prefill_workspace(const tv_prefill_args* a, int sm_count) {
  return layout(a, sm_count).total;
}

cudaError_t launch_prefill(const tv_prefill_args* a, void* ws, int sm_count, cudaStream_t st) {
  cudaError_t e = setup();
  if (e != cudaSuccess) return e;
  const Layout l = layout(a, sm_count);
  char* base = (char*)ws;
  int32_t* counts = (int32_t*)base;
  int4* q_tiles = (int4*)(base + l.q_tiles);
  int4* k_tiles = (int4*)(base + l.k_tiles);
  const uint64_t H = a->H, T = a->T, cap = (uint64_t)l.cap;

  PlanArgs pa{a->q_start, a->prefix_len, a->B,    a->T,    a->max_q_len, a->max_kv_len,
              (int)l.max_q, (int)l.max_k, a->H, l.cut ? sm_count : 0, counts, q_tiles, k_tiles,
              (int4*)(base + l.pieces), (int2*)(base + l.tile_pieces), a->status};
  plan_kernel<<<1, 1024, 0, st>>>(pa);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;

  CUtensorMap m_c, m_w, m_q, m_qr, m_k, m_v, m_kr;
  const uint64_t dq[3] = {kDN, H, T}, sq[2] = {kDN * 2, H * kDN * 2};
  const uint64_t dqr[3] = {kDR, H, T}, sqr[2] = {kDR * 2, H * kDR * 2};
  const uint32_t bq[3] = {64, 1, kBlock};
  const uint64_t dk[3] = {kDN, cap, H}, sk[2] = {kDN * 2, cap * kDN * 2};
  const uint32_t bk[3] = {64, kBlock, 1};
  const uint64_t dv[4] = {64, cap, kDV / 64, H}, sv[3] = {kDV * 2, 128, cap * kDV * 2};
  const uint32_t bv[4] = {64, 64, kDV / 64, 1};
  if (!map2(&m_c, a->c_kv, a->d_latent, (uint64_t)a->cache.num_rows,
            (uint64_t)a->ckv_row_stride * 2, 64) ||
      !map2(&m_w, a->w_kv, a->d_latent, H * kKV, (uint64_t)a->d_latent * 2, kKV) ||
      !make_map(&m_q, a->q_nope, 3, dq, sq, bq) || !make_map(&m_qr, a->q_pe, 3, dqr, sqr, bq) ||
      !make_map(&m_k, base + l.k, 3, dk, sk, bk) || !make_map(&m_v, base + l.v, 4, dv, sv, bv) ||
      !map2(&m_kr, base + l.kr, kDR, cap, kDR * 2, kBlock))
    return cudaErrorInvalidValue;

  ExpandArgs xa{};
  xa.counts = counts;
  xa.k_tiles = k_tiles;
  xa.page_table = a->cache.page_table;
  xa.max_pages = a->cache.max_pages;
  xa.H = a->H;
  xa.k_chunks = a->d_latent / 64;
  xa.kv_stride_b = a->cache.kv_stride_b;
  xa.num_rows = a->cache.num_rows;
  xa.k_pe = (const __nv_bfloat16*)a->k_pe;
  xa.kpe_stride = a->kpe_row_stride;
  xa.cap = l.cap;
  xa.K = (__nv_bfloat16*)(base + l.k);
  xa.V = (__half*)(base + l.v);
  xa.KR = (__nv_bfloat16*)(base + l.kr);
  xa.status = a->status;
  AttendArgs aa{counts, q_tiles, l.cut ? (const int4*)(base + l.pieces) : nullptr,
                (const int2*)(base + l.tile_pieces), a->H, (float)((double)a->scale * 1.4426950408889634),
                (__nv_bfloat16*)a->out, (float*)(base + l.part_o), (float*)(base + l.part_ml),
                a->status, {}};
  {
    std::lock_guard<std::mutex> lock(g_fault_mu);
    xa.fault = g_expand_fault;
    aa.fault = g_attend_fault;
  }

  // each kernel's set-up runs beside the one before it (programmatic dependent launch)
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(l.max_k * a->H, sm_count));
  cfg.blockDim = dim3(kExpThreads);
  cfg.dynamicSmemBytes = kExpSmem;
  e = cudaLaunchKernelEx(&cfg, expand_kernel, xa, m_c, m_w);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(l.cut ? sm_count : std::min<int64_t>(l.max_q * a->H, sm_count)));
  cfg.blockDim = dim3(kAttThreads);
  cfg.dynamicSmemBytes = kAttSmem;
  e = cudaLaunchKernelEx(&cfg, attend_kernel, aa, m_q, m_qr, m_k, m_v, m_kr);
  if (e != cudaSuccess || !l.cut) return e;
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(l.max_q * a->H * (kPair / 8), 4 * sm_count));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, join_kernel, aa);
}

}  // namespace tv

extern "C" int tv_testing_set_prompt_fault(int expand_loads, int attend_loads,
                                           uint64_t deadline_ns, int32_t* exit_counts) {
  if (deadline_ns > 2000000000ull) return TV_ERR_INVALID_ARG;
  // two clocks a nanosecond
  const long long deadline = deadline_ns ? 2ll * (long long)deadline_ns : tv::kDeadline;
  std::lock_guard<std::mutex> lock(tv::g_fault_mu);
  tv::g_expand_fault = {expand_loads < 0 ? tv::kAllLoads : expand_loads, deadline, exit_counts};
  tv::g_attend_fault = {attend_loads < 0 ? tv::kAllLoads : attend_loads, deadline,
                        exit_counts ? exit_counts + 2 : nullptr};
  return TV_OK;
}
