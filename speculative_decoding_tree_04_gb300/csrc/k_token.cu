// k_token.cu -- next tokens with temperature, top-k, top-p and min-p (tv_token_sample).
//
// All filters keep a beginning of one order, falling logit and then index, so what they leave
// ends at one token, the cut: top_k's is the k-th; top_p's the token at which the running sum of
// weights reaches p W, W the sum of what top_k keeps; min_p bounds the weight itself.  The token
// is then drawn in index order from what is kept.
//
// Weights are integers in units of 2^-44 of the largest (sample_math.h), and all decisions are
// taken on exact sums of them.  A weight costs 31 float operations, so the passes over a row are
// arranged to take each about once at most:
//   1. the maximum;
//   2. counts of the tokens in kBins bins that are linear in the logit (kSpan units of log2 of
//      the weight, the last bin for all below);
//   top_k: the counts say in which bin the k-th token lies;
//   top_p: a bin's weights lie within a factor 2^(kSpan / kBins), so the counts bound the running
//      sums to about 1 %, and the cut to a window of bins;
//   3. (top_p) exact sums of the row and, by warp, of the tokens above the window; the warps keep
//      the window's tokens (where they are too many, the row is read again instead), which are
//      summed in kFine finer bins, one of which holds the cut;
//   4. the tokens of the cut's bin go into a list, and are compared with one another; a bf16
//      row's bin is one value, whose tokens are counted by warp, to find the cut's index;
//   5. the kept tokens' sums by warp, unless 3 has left them, and the draw within one warp's
//      slice.
// Where the bins down to the cut hold few tokens altogether (top_k of common sizes, peaked
// distributions) all of them go into the list and the rest happens there.  Where the cut's own
// bin holds too many for the list (equal logits) it is cut by ordered bit patterns, level by
// level, until a bin is one value.
//
// Work.  A cluster of CTAs shares a row, each CTA a contiguous slice, each warp a part of it;
// after the first pass the row comes from L2.  Bins are added up over the cluster through
// distributed shared memory, each CTA the same share of them, and given to every CTA, which all
// take the same decisions from the same numbers.  Sums are of integers: no result depends on the
// order they are taken in, or on how a row is split.
//
// A bf16 row has few values: where it is long their weights are taken once, into a table, and the
// passes look them up.
//
// Measured, in a graph of such calls (64 rows of 163840 floats; 256 of 50257 bf16; 1 of 32000 bf16):
// greedy 9.7, 5.3 and 4.2 us (4.3 TB/s of the first's 42 MB); top_k 40 31, 30 and 16; no filter 36, 28
// and 10; top_p 0.95 72, 62 and 29 (8 rows of 163840 bf16: 36).  What bounds it with a filter: a
// CTA's own chain of passes.  A float's weight takes 31 float operations and some 15 integer ones, 12
// us for a CTA's 40960 (73 % of the issue slots while it lasts); a table's look-up half of that, its
// window tests and sums included; a count five, and 6.5 cycles for the atomics' conflicts; then
// barriers, a cluster's about 1 us each, and what a thread does once.  Over a whole call no unit is
// full (issue slots 48 % in the bf16 batch, 60 % on the busiest SM): its 256 CTAs are two side by side
// on 104 of the 152 SMs and one on the others, which take nine tenths of the time of two.
// Mixed filters: the rows with top_p alone take two to three times the others' time, and the others'
// SMs wait (SMs active 61 % of the call, issue slots 24 %).  Greedy rows wait for memory (12 of 26
// cycles between a warp's instructions) and the cluster's start and end.  Packed float operations gave
// the same times (their lanes are the same), and so did counting during the first pass below a
// guessed maximum.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "sample_math.h"
#include "sm100_ptx.h"
#include "tv_internal.h"

namespace tv {
namespace {

using namespace ptx;

constexpr int kMaxCluster = 16;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 4096, kFine = 2048;
constexpr float kSpan = 48.f;  // log2 units of the linear bins: below, weights are zero
constexpr int kList = 512;     // tokens of a list at most
constexpr int kSmall = 256;    // of one that holds every kept token
constexpr int kWindow = 256;   // of a window's tokens that a warp keeps
constexpr int kSome = 4;       // values of a vector that the passes with weights take at once
constexpr int kValues = 4096;  // values of a bf16 row whose weights are taken once, where a thread has
constexpr int kTabled = 28;    // so many tokens (256 rows, top_p, 8192 tokens: 31.0 us without the
                               // table, 32.9 with it; 16384: 39.3 and 37.7)
constexpr int kHold = 64;      // of these whose weights' parts, of 2^22, are added as ints
constexpr int kAhead = 2;      // vectors of a lane's that are on their way

struct TokenParams {
  const void* logits;
  int64_t V, stride;
  int B, sorted;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* uniforms;
  int32_t* tokens;
  int32_t* kept;
  int32_t* status;
};

struct Shared {
  ScaledTable exp2;
  union {
    struct {
      alignas(16) uint32_t bins[kBins];  // this CTA's: counts, or sums (kFine low halves, then high ones)
      alignas(16) int64_t all[kFine];    // the cluster's: counts (kBins of 32 bits), or sums
    };
    int64_t values[kValues + 1];  // between these uses: the weights of a bf16 row's values, and 0
  };
  uint64_t window_of[kWarps][kWindow];  // the warps' tokens of the window
  uint64_t list[kList];           // this CTA's tokens: key, complemented index
  uint64_t merged[kList];         // the cluster's,
  int64_t merged_w[kList];        // and their weights
  int32_t list_n;
  uint64_t keys[kMaxCluster];     // exchanged: the slices' maxima,
  int32_t lists[kMaxCluster];     // lengths of lists,
  int64_t mass[4][kMaxCluster];   // sums,
  int32_t count[kMaxCluster];     // and counts
  uint64_t warp_key[kWarps];
  int64_t warp_mass[kWarps], warp_three[3][kWarps];
  int32_t warp_count[kWarps];
  float warp_up[4][kWarps];       // of the window's search
  int32_t warp_n[kWarps], n_before[3];
  int64_t found[2];               // a bin, and the total before it
  int32_t window[4], too_many;
  uint64_t cut;
  uint32_t is_long[kWarps];
};
static_assert(kBins == 2 * kFine && kFine / 4 >= kThreads && kBins % kThreads == 0 && kFine % kThreads == 0, "bins");

__device__ __forceinline__ uint4 ld_cluster_v4(const void* local, uint32_t rank) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(map_to_rank(smem_u32(local), rank))
               : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_v4(const void* local, uint32_t rank, uint4 v) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(map_to_rank(smem_u32(local), rank)),
               "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
// Four words of the C CTAs of the cluster (a power of two), lane r of a group of C holding CTA r's,
// added up: the sum in every lane.
__device__ __forceinline__ uint4 add_up(uint4 v, int C) {
  for (int o = C / 2; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
    v.w += __shfl_xor_sync(0xffffffffu, v.w, o);
  }
  return v;
}
__device__ __forceinline__ uint4 get(const uint32_t* local, int C, int r) {
  return C == 1 ? *reinterpret_cast<const uint4*>(local) : ld_cluster_v4(local, (uint32_t)r);
}
__device__ __forceinline__ void give(void* local, int C, int r, uint4 v) {
  if (C == 1) *reinterpret_cast<uint4*>(local) = v;
  else st_cluster_v4(local, (uint32_t)r, v);
}
__device__ __forceinline__ uint64_t ld_cluster_u64(const void* local, uint32_t rank) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(map_to_rank(smem_u32(local), rank)) : "memory");
  return v;
}

// Exclusive prefix sum of one value a thread over the block; *total is the sum.
template <typename S>
__device__ __forceinline__ S block_scan(S v, S* warps, S* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  S up_to = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const S below = __shfl_up_sync(0xffffffffu, up_to, o);
    if (lane >= o) up_to += below;
  }
  __syncthreads();
  if (lane == 31) warps[warp] = up_to;
  __syncthreads();
  const S mine = lane < kWarps ? warps[lane] : (S)0;
  *total = warp_sum(mine);
  return up_to - v + warp_sum(lane < warp ? mine : (S)0);
}

// 2^-x of a bin's width, from the exponential's series.
constexpr float bin_ratio(double x) {
  const double y = -kLn2 * x * (double)kSpan / (kBins - 1);
  return (float)(1.0 + y * (1.0 + y / 2 * (1.0 + y / 3 * (1.0 + y / 4))));
}
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
// The largest of a vector's values, NaN where one is.
template <typename T>
__device__ __forceinline__ float largest(const uint4& w) {
  if constexpr (sizeof(T) == 4) {
    return max_or_nan(max_or_nan(__uint_as_float(w.x), __uint_as_float(w.y)),
                      max_or_nan(__uint_as_float(w.z), __uint_as_float(w.w)));
  } else {
    auto two = [](uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); };
    const __nv_bfloat162 y = __hmax2_nan(__hmax2_nan(two(w.x), two(w.y)), __hmax2_nan(two(w.z), two(w.w)));
    return max_or_nan(__low2float(y), __high2float(y));
  }
}
// A vector of a row at one of its ends (out of line: the passes are many and code is dear).
template <typename T>
__device__ __noinline__ uint4 end_vector(const T* x, int64_t V, int64_t a) {
  constexpr int N = Vec<T>::N;
  alignas(16) T v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = a + i >= 0 && a + i < V ? x[a + i] : (T)-INFINITY;
  return *reinterpret_cast<const uint4*>(v);
}
// One exact weight, out of line too (m: the maximum).
__device__ __noinline__ int64_t one_weight(float v, float m, float lowest, const RowScale& scale,
                                           const ScaledTable& table) {
  if (lowest != lowest) return v == m ? (int64_t)kUnit : 0;
  return units(scaled_weight(fmaxf(v, lowest), scale, table));
}

// The i-th row to start: those with a top_p and no top_k, which take two to three times as long as
// others, before the others, so that no SM is given two of them while another has none (64 rows x
// 163840, a quarter of them long and 36 rows apart: 75 us in order of rows, 63 sorted; rows alike:
// 0.7 us more).
constexpr int kSorted = 32 * kWarps;  // rows at most
__device__ __forceinline__ int row_in_order(const TokenParams& p, int i, uint32_t* is_long) {
  const int lane = threadIdx.x & 31, r = threadIdx.x;
  bool is = false;
  if (r < p.B) {
    const int k = p.top_k ? p.top_k[r] : 0;
    is = p.top_p[r] < 1.f && !(k > 0 && k < p.V) && (!p.temperature || p.temperature[r] != 0.f);
  }
  const uint32_t bits = __ballot_sync(0xffffffffu, is);
  if (lane == 0) is_long[r / 32] = bits;
  __syncthreads();
  uint32_t mine = lane < kWarps ? is_long[lane] : 0u;
  const int n_long = warp_sum(__popc(mine));
  if (i >= n_long) {
    i -= n_long;
    mine = ~mine;
  }
  const int c = locate(__popc(mine), 32, &i);
  uint32_t left = __shfl_sync(0xffffffffu, mine, c);
  for (; i > 0; --i) left &= left - 1;
  return 32 * c + __ffs(left) - 1;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) token_sample_kernel(const TokenParams p, int log2_C) {
  constexpr int N = Vec<T>::N;
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = 1 << log2_C;
  const int rank = C > 1 ? (int)cluster_rank() : 0;
  griddep_wait();
  const int place_of_row = blockIdx.x >> log2_C;
  // (a reduction's result is seen to be the same in the whole warp, and needs no registers)
  const int b = (int)__reduce_max_sync(
      0xffffffffu, (uint32_t)(p.sorted ? row_in_order(p, place_of_row, sh.is_long) : place_of_row));
  const float T0 = p.temperature ? p.temperature[b] : 1.f;
  const int top_k = p.top_k ? p.top_k[b] : 0;
  const float top_p = p.top_p ? p.top_p[b] : 1.f, min_p = p.min_p ? p.min_p[b] : 0.f;
  const float u = fminf(fmaxf(p.uniforms[b], 0.f), 0x1.fffffep-1f);  // (NaN: 0)
  const bool greedy = T0 == 0.f;
  if (!(T0 >= 0.f) || (!greedy && (top_p != top_p || min_p != min_p))) {  // the cluster alike
    if (rank == 0 && tid == 0) {
      p.tokens[b] = -1;
      if (p.kept) p.kept[b] = 0;
      report(p.status, TV_ERR_INVALID_ARG);
    }
    return;
  }
  // (a CTA's shared memory may be written once it is known to have started)
  if (C > 1) cluster_arrive();
  auto sync = [&]() {
    if (C > 1) cluster_sync();
    else __syncthreads();
  };

  // This warp's vectors, and what it does with every one of them: fn(values, index of the first).
  const Row<T> row((const T*)p.logits + (int64_t)b * p.stride, p.V);
  const int per = (row.n_vec + C - 1) >> log2_C, per_w = (per + kWarps - 1) / kWarps;
  const int c0 = min(row.n_vec, rank * per), c1 = min(row.n_vec, c0 + per);
  const int w0 = min(c1, c0 + warp * per_w), w1 = min(c1, w0 + per_w);
  // (the row's first and last vector may reach past it)
  const int e0 = row.first_whole(), e1 = row.end_whole();
  const int whole0 = max(w0, e0);
  const uint32_t n_whole = (uint32_t)max(min(w1, e1) - whole0, 0);
  const uint4* vectors = reinterpret_cast<const uint4*>(row.x - row.off);
  auto vector = [&](int j) {
    return j >= e0 && j < e1 ? __ldg(vectors + j) : end_vector<T>(row.x, p.V, row.first(j));
  };
  auto fetch = [&](int j) {  // of the warp's, masked past its last one
    if ((uint32_t)(j - whole0) < n_whole) return __ldg(vectors + j);
    return j < w1 ? vector(j)
                  : make_uint4(Vec<T>::kMasked, Vec<T>::kMasked, Vec<T>::kMasked, Vec<T>::kMasked);
  };
  // All lanes call it together, those past the last vector with -inf.  `dear`: one copy of fn's
  // code for kSome values, the next vectors on their way (unrolled, such passes outgrow the
  // registers and the instruction cache).
  auto each = [&](auto dear, auto fn) {
    if constexpr (decltype(dear)::value) {
      uint4 next[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) next[k] = fetch(w0 + lane + 32 * k);
#pragma unroll 1
      for (int j0 = w0; j0 < w1; j0 += 32) {
        uint4 w = next[0];
#pragma unroll
        for (int k = 0; k + 1 < kAhead; ++k) next[k] = next[k + 1];
        next[kAhead - 1] = fetch(j0 + lane + 32 * kAhead);
#pragma unroll 1
        for (int i = 0; i < N; i += kSome) {
          float v[N];
          Vec<T>::unpack(w, v);  // (its first kSome values)
          fn(v, (j0 + lane) * N + i - row.off);
          if constexpr (N > kSome) {
            w.x = w.z;
            w.y = w.w;
          }
        }
      }
    } else {
      constexpr int kUnroll = 4;
#pragma unroll 1
      for (int j0 = w0; j0 < w1; j0 += 32 * kUnroll) {
        uint4 w[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) w[k] = fetch(j0 + lane + 32 * k);
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
          float v[N];
          Vec<T>::unpack(w[k], v);
          fn(v, (j0 + lane + 32 * k) * N - row.off);
        }
      }
    }
  };
  constexpr std::true_type kDear{};
  constexpr std::false_type kLight{};

  // ---- the row's maximum, with its first index ----
  uint64_t top;
  {
    float best = -INFINITY;  // (NaN where one is)
    int best_j = w0 + lane;
    constexpr int kUnroll = 8;
#pragma unroll 1
    for (int j0 = w0 + lane; j0 < w1; j0 += 32 * kUnroll) {
      uint4 w[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) w[k] = fetch(j0 + 32 * k);
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const float x = largest<T>(w[k]);
        if (x > best) best_j = j0 + 32 * k;
        best = max_or_nan(best, x);
      }
    }
    int best_at = 0;
    if (greedy && best > -INFINITY) {
      float v[N];
      Vec<T>::unpack(fetch(best_j), v);
#pragma unroll
      for (int i = N - 1; i >= 0; --i)
        if (v[i] == best) best_at = best_j * N - row.off + i;
    }
    for (int i = tid; i < kTable * 32; i += kThreads) {
      sh.exp2.hi[i] = d_exp_over_linear.hi[i / 32];
      sh.exp2.lo[i] = d_exp_over_linear.lo[i / 32];
    }
    // order-preserving value bits, then the complemented index; a NaN beats every value
    top = best > -INFINITY
              ? ((uint64_t)ordered(best) << 32) | (0xFFFFFFFFu - (uint32_t)best_at)
              : 0ull;
    top = warp_max(top);
    if (__any_sync(0xffffffffu, best != best)) top = ~0ull;
    if (lane == 0) sh.warp_key[warp] = top;
    if (C > 1) cluster_wait();
    __syncthreads();
    if (warp == 0) {
      top = warp_max(lane < kWarps ? sh.warp_key[lane] : 0ull);
      if (C == 1) {
        if (lane == 0) sh.keys[0] = top;
      } else if (lane < C) {
        st_cluster_u64(&sh.keys[rank], (uint32_t)lane, top);
      }
    }
    sync();
    top = warp_max(lane < C ? sh.keys[lane] : 0ull);
  }
  const float m = unordered((uint32_t)(top >> 32));
  const bool none = top == 0 || top == ~0ull || m == INFINITY;
  if (none || greedy) {
    if (rank == 0 && tid == 0) {
      p.tokens[b] = none ? -1 : (int)(0xFFFFFFFFu - (uint32_t)top);
      if (p.kept) p.kept[b] = none ? 0 : 1;
      if (none) report(p.status, TV_ERR_INVALID_ARG);
    }
    if (C > 1) cluster_sync();  // no CTA leaves while another may still write to it
    return;
  }

  float lowest;
  const RowScale scale(m, T0, &lowest);
  const float ch = scale.k64 * (1.f / kTable), per_bin = ch * ((float)(kBins - 1) / kSpan);
  const bool apart = lowest != lowest;
  auto weight_of = [&](float v) { return one_weight(v, m, lowest, scale, sh.exp2); };
  // The weights of kSome values.
  auto weights_of = [&](const float* v, Weight* w) {
    if (apart) {
#pragma unroll
      for (int i = 0; i < kSome; ++i) w[i] = {v[i] == m ? 1 << 22 : 0, 0};
      return;
    }
#pragma unroll
    for (int i = 0; i < kSome; ++i) w[i] = scaled_weight(fmaxf(v[i], lowest), scale, sh.exp2);
  };
  // bf16: the weights of all values from the maximum down to `lowest`, but those next to 0, in a
  // table: the negative ones by falling magnitude (its bits a <= low_a), then the others (a <= high_a),
  // both of them down to cut_a, which is where they, or one of them alone, fill the table (for logits
  // of ordinary size 2^-13 or less).
  const int low_a = lowest <= 0.f ? (int)(__float_as_uint(lowest) >> 16 & 0x7FFFu) + 1 : -1;
  const int high_a = m >= 0.f ? (int)(__float_as_uint(m) >> 16 & 0x7FFFu) : -1;
  const int alone = max(low_a, high_a) + 1 - kValues;
  const int cut_a = max(max(alone, low_a < 0 || high_a < 0 ? 0 : (low_a + high_a + 3 - kValues) >> 1), 0);
  const int n_negative = max(low_a - cut_a + 1, 0), top_a = n_negative + high_a;
  const bool tabled = sizeof(T) == 2 && !apart && per * N >= kTabled * kThreads;
  auto make_values = [&]() {
    for (int i = tid; i <= kValues; i += kThreads) {
      const bool negative = i < n_negative;
      const int a = (negative ? low_a : top_a) - i;
      const float v = __uint_as_float((uint32_t)max(a, 0) << 16 | (negative ? 0x80000000u : 0u));
      const bool is = a >= cut_a && i < kValues && v >= lowest && v <= m;
      sh.values[i] = is ? units(scaled_weight(v, scale, sh.exp2)) : 0;
    }
    __syncthreads();
  };
  // (what lies past either end of the table weighs nothing; a value next to 0 is seen by the caller,
  // who finds the smallest magnitude below next_to_0)
  const float next_to_0 = __uint_as_float((uint32_t)cut_a << 16);
  auto value_weight = [&](float v) {
    const uint32_t u = __float_as_uint(v);
    const int i = ((int)u < 0 ? low_a : top_a) - (int)(u >> 16 & 0x7FFFu);
    return sh.values[min((uint32_t)i, (uint32_t)kValues)];
  };
  auto value_weights = [&](const float* v, int64_t* w) {
    float least_of = fabsf(v[0]);
#pragma unroll
    for (int i = 1; i < kSome; ++i) least_of = fminf(least_of, fabsf(v[i]));
    if (least_of < next_to_0) {
#pragma unroll
      for (int i = 0; i < kSome; ++i) w[i] = weight_of(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kSome; ++i) w[i] = value_weight(v[i]);
    }
  };
  // A token's place in the order, larger first; a value's bin, rising as the value falls (so that
  // a bin is a range of keys).
  auto place = [&](float v, int index) {
    return ((uint64_t)ordered(v) << 32) | (0xFFFFFFFFu - (uint32_t)index);
  };
  auto position = [&](float v) { return (m - v) * per_bin; };
  auto linear = [&](float v) { return min((int)position(v), kBins - 1); };
  constexpr uint64_t kMasked = (uint64_t)0x007FFFFFu << 32 | 0xFFFFFFFFu;  // -inf, any index
  uint64_t cut = kMasked + 1;  // tokens at or above it are kept
  const float mp = fminf(fmaxf(min_p, 0.f), 1.f);
  // (the maximum's own weight may be off by a unit, and is kept with a min_p of 1 too)
  const int64_t least = mp > 0.f ? min((int64_t)ceil((double)mp * (double)kUnit), weight_of(m)) : 0;
  // (a token this far below the maximum is lighter than min_p without more ado)
  const float far = mp > 0.f ? fminf(-__log2f(mp) * 1.0001f + 0.01f, 64.f) : INFINITY;

  auto clear = [&](int n) {
    for (int i = tid; i < n; i += kThreads) sh.bins[i] = 0u;
    __syncthreads();
  };
  auto add_mass = [&](int bin, uint64_t w) {
    const uint32_t low = (uint32_t)w, old = atomicAdd(&sh.bins[bin], low);
    const uint32_t high = (uint32_t)(w >> 32) + (old + low < old ? 1u : 0u);
    if (high) atomicAdd(&sh.bins[kFine + bin], high);
  };
  // The cluster's bins from the CTAs': every CTA adds up its share and gives it to all, a thread
  // for four bins and one CTA to read from and to give to (whole warps: kFine / 4 is at least a
  // block's threads).
  const int give_to = tid & (C - 1), first_bin = 4 * (tid >> log2_C), step = 4 * (kThreads >> log2_C);
  auto merge_counts = [&]() {
    sync();
    const int share = kBins >> log2_C;
    for (int i = first_bin; i < share; i += step) {
      const int at = rank * share + i;
      give(reinterpret_cast<uint32_t*>(sh.all) + at, C, give_to, add_up(get(&sh.bins[at], C, give_to), C));
    }
    sync();
  };
  auto merge_mass = [&]() {
    sync();
    const int share = kFine >> log2_C;
    for (int i = first_bin; i < share; i += step) {
      const int at = rank * share + i;
      const uint4 x = get(&sh.bins[at], C, give_to), y = get(&sh.bins[kFine + at], C, give_to);
      auto sum = [&](uint32_t low, uint32_t high) {
        uint64_t w = (uint64_t)high << 32 | low;
        for (int o = C / 2; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
        return w;
      };
      const uint64_t s0 = sum(x.x, y.x), s1 = sum(x.y, y.y), s2 = sum(x.z, y.z), s3 = sum(x.w, y.w);
      give(&sh.all[at], C, give_to,
           make_uint4((uint32_t)s0, (uint32_t)(s0 >> 32), (uint32_t)s1, (uint32_t)(s1 >> 32)));
      give(&sh.all[at + 2], C, give_to,
           make_uint4((uint32_t)s2, (uint32_t)(s2 >> 32), (uint32_t)s3, (uint32_t)(s3 >> 32)));
    }
    sync();
  };
  // The bin of n in which the running total of get(bin) passes target; *before: the total up to it.
  auto find = [&](int n, auto get, int64_t target, int64_t* before, int64_t* total) {
    const int each_n = n / kThreads;
    int64_t s = 0;
    for (int i = 0; i < each_n; ++i) s += get(tid * each_n + i);
    int64_t at = block_scan(s, sh.warp_mass, total);
    if (at <= target && target < at + s) {
      int i = tid * each_n;
      for (int64_t x; at + (x = get(i)) <= target; ++i) at += x;
      sh.found[0] = i;
      sh.found[1] = at;
    }
    __syncthreads();
    *before = sh.found[1];
    return (int)sh.found[0];
  };
  auto count_at = [&](int i) { return (int64_t) reinterpret_cast<const uint32_t*>(sh.all)[i]; };
  auto mass_at = [&](int i) { return sh.all[i]; };
  // The sums of three values a thread over the cluster.
  auto totals_of = [&](int64_t& x, int64_t& y, int64_t& z) {
    int64_t v[3] = {x, y, z};
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      v[i] = warp_sum(v[i]);
      if (lane == 0) sh.warp_three[i][warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      v[i] = warp_sum(lane < kWarps ? sh.warp_three[i][lane] : (int64_t)0);
      if (C > 1 && warp == i && lane < C) st_cluster_u64(&sh.mass[i][rank], (uint32_t)lane, (uint64_t)v[i]);
    }
    if (C > 1) {
      sync();
#pragma unroll
      for (int i = 0; i < 3; ++i) v[i] = warp_sum(lane < C ? sh.mass[i][lane] : (int64_t)0);
    }
    x = v[0];
    y = v[1];
    z = v[2];
  };
  // Lists: tokens are put on the CTA's (kList at most are kept, all are counted), which are then
  // joined in sh.merged with their weights, in any order.  join_lists returns how many there are.
  auto start_list = [&]() {
    __syncthreads();
    if (tid == 0) sh.list_n = 0;
    __syncthreads();
  };
  auto put_on_list = [&](float v, int index) {
    const int at = atomicAdd(&sh.list_n, 1);
    if (at < kList) sh.list[at] = place(v, index);
  };
  auto join_lists = [&]() {
    __syncthreads();
    if (C == 1) {
      if (tid == 0) sh.lists[0] = sh.list_n;
    } else if (warp == 0 && lane < C) {
      st_cluster_u32(&sh.lists[rank], (uint32_t)lane, (uint32_t)sh.list_n);
    }
    sync();
    const int n = warp_sum(lane < C ? sh.lists[lane] : 0);
    if (n <= kList) {
      int at = 0;
      for (int r = 0; r < C; ++r) {
        const int k = sh.lists[r];
        for (int i = tid; i < k; i += kThreads) {
          const uint64_t x = C == 1 ? sh.list[i] : ld_cluster_u64(&sh.list[i], (uint32_t)r);
          sh.merged[at + i] = x;
          sh.merged_w[at + i] = weight_of(unordered((uint32_t)(x >> 32)));
        }
        at += k;
      }
      __syncthreads();
    }
    return n;
  };
  // The smallest key whose linear bin is at most `bin`, by one probe a lane: first of the 32 keys
  // around the bins' inverse, which mostly hold it.
  auto first_key = [&](int bin) {
    uint32_t lo = 0x00800000u, hi = (uint32_t)(top >> 32);  // linear(hi) = 0
    const uint32_t near = min(max(ordered(m - (float)(bin + 1) / per_bin), lo + 16u), hi) - 16u;
    {
      const uint32_t in = __ballot_sync(
          0xffffffffu, near + (uint32_t)lane >= hi || linear(unordered(near + (uint32_t)lane)) <= bin);
      const int at = __ffs(in) - 1;
      if (at > 0) return min(near + (uint32_t)at, hi);
    }
    while (lo < hi) {
      const uint32_t step = (hi - lo + 31) / 32, probe = min(hi, lo + (uint32_t)lane * step);
      const uint32_t in = __ballot_sync(0xffffffffu, linear(unordered(probe)) <= bin);
      const int at = __ffs(in) - 1;  // (none: the answer lies above the last probe)
      if (at == 0) return lo;
      const uint32_t below = lo + (uint32_t)(at < 0 ? 31 : at - 1) * step;
      hi = at < 0 ? hi : min(hi, lo + (uint32_t)at * step);
      lo = min(hi, below + 1);
    }
    return lo;
  };
  // The list of the tokens from the bins first .. last that are not behind the cut.
  auto gather = [&](int first, int last) {
    const float above_it = first > 0 ? unordered(first_key(first - 1)) : INFINITY;
    const float from = unordered(first_key(last));
    start_list();
    each(kLight, [&](const float* v, int a) {
      float x = v[0];  // (few vectors have one: of those from the first bin on, by their largest)
#pragma unroll
      for (int i = 1; i < N; ++i) x = fmaxf(x, v[i]);
      if (!(x >= from)) return;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (v[i] >= from && v[i] < above_it && place(v[i], a + i) >= cut) put_on_list(v[i], a + i);
    });
    return join_lists();
  };
  // Tokens of the list, P threads each: fn(token, its part), with P a power of two within a warp.
  auto threads_per = [&](int n) {
    int P = 32;
    while (P > 1 && P * n > kThreads) P >>= 1;
    return P;
  };
  // How many of the list's tokens come before token x, and their weights' sum.
  auto before_in_list = [&](int n, int P, uint64_t x, int64_t* mass) {
    int64_t count = 0, sum = 0;
    for (int j = tid & (P - 1); j < n; j += P) {
      const bool is = sh.merged[j] > x;
      count += is;
      sum += is ? sh.merged_w[j] : 0;
    }
    for (int o = P / 2; o > 0; o >>= 1) {
      count += __shfl_xor_sync(0xffffffffu, count, o);
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    *mass = sum;
    return count;
  };
  // The cut from a list that holds it: the token with `target` tokens (or weight up to it) before.
  auto cut_in_list = [&](int n, bool mass, int64_t target) {
    const int P = threads_per(n);
    for (int e0_ = 0; e0_ < n; e0_ += kThreads / P) {
      const int e = e0_ + tid / P;
      const uint64_t x = e < n ? sh.merged[e] : ~0ull;
      int64_t sum;
      const int64_t count = before_in_list(n, P, x, &sum);
      if (e < n && (tid & (P - 1)) == 0 &&
          (mass ? sum <= target && target < sum + sh.merged_w[e] : count == target))
        sh.cut = x;
    }
    __syncthreads();
    return sh.cut;
  };
  // The cut at the n-th (from 0) of the tokens with this key, in order of index, those before the
  // limit aside; kept: how many of the warp's are in window_of, -1: they have to be looked for.
  auto nth_at = [&](uint32_t hi, int64_t n, uint64_t limit, int kept) {
    int64_t mine = 0;
    if (kept >= 0) {
      for (int i = lane; i < kept; i += 32) mine += (uint32_t)(sh.window_of[warp][i] >> 32) == hi;
    } else {
      each(kDear, [&](const float* v, int a) {
#pragma unroll
        for (int i = 0; i < kSome; ++i) mine += ordered(v[i]) == hi && place(v[i], a + i) >= limit;
      });
    }
    mine = warp_sum(mine);
    __syncthreads();
    if (lane == 0) sh.warp_count[warp] = (int)mine;
    __syncthreads();
    const int64_t all = warp_sum(lane < kWarps ? (int64_t)sh.warp_count[lane] : 0);
    if (warp == 0 && lane < C) {
      if (C == 1) sh.count[0] = (int)all;
      else st_cluster_u32(&sh.count[rank], (uint32_t)lane, (uint32_t)all);
    }
    sync();
    n -= warp_sum(lane < rank ? (int64_t)sh.count[lane] : (int64_t)0);
    n -= warp_sum(lane < warp ? (int64_t)sh.warp_count[lane & (kWarps - 1)] : (int64_t)0);
    auto found_it = [&](uint64_t x) {
      for (int r = 0; r < C; ++r) {
        if (C == 1) sh.cut = x;
        else st_cluster_u64(&sh.cut, (uint32_t)r, x);
      }
    };
    if (kept >= 0 && n >= 0 && n < mine) {  // on this warp's list
      for (int i = lane; i < kept; i += 32) {
        const uint64_t x = sh.window_of[warp][i];
        if ((uint32_t)(x >> 32) != hi) continue;
        int before = 0;
        for (int k = 0; k < kept; ++k) {
          const uint64_t y = sh.window_of[warp][k];
          before += (uint32_t)(y >> 32) == hi && y > x;
        }
        if (before == n) found_it(x);
      }
    } else if (n >= 0 && n < mine) {  // in its slice
      for (int j0 = w0; j0 < w1; j0 += 32) {
        float v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = NAN;
        if (j0 + lane < w1) Vec<T>::unpack(vector(j0 + lane), v);
        const int a = (int)row.first(j0 + lane);
        int64_t k = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) k += ordered(v[i]) == hi && v[i] == v[i] && place(v[i], a + i) >= limit;
        const int64_t here = warp_sum(k);
        if (n >= here) {
          n -= here;
          continue;
        }
        if (lane == locate(k, 32, &n)) {
          uint64_t x = 0;
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (ordered(v[i]) == hi && place(v[i], a + i) >= limit && n-- == 0) x = place(v[i], a + i);
          found_it(x);
        }
        break;
      }
    }
    sync();
    return sh.cut;
  };
  // The cut among more tokens than a list holds, of keys lo .. hi, `target` tokens (or weight)
  // into them: by key, level by level, then the first tokens at the last key by index.
  auto refine = [&](bool mass, uint32_t lo, uint32_t hi, int64_t target) {
    const uint64_t limit = cut;
    for (int step = 0; step < 3; ++step) {  // (2^32 keys, kFine bins)
      int shift = 0;
      while (((hi - lo) >> shift) >= (uint32_t)kFine) ++shift;
      clear(2 * kFine);
      each(kDear, [&](const float* v, int a) {
#pragma unroll
        for (int i = 0; i < kSome; ++i) {
          const uint32_t key = ordered(v[i]);
          if (key < lo || key > hi || place(v[i], a + i) < limit) continue;
          add_mass((int)((hi - key) >> shift), mass ? (uint64_t)weight_of(v[i]) : 1ull);
        }
      });
      merge_mass();
      int64_t before, total;
      const uint32_t at = (uint32_t)find(kFine, mass_at, target, &before, &total);
      target -= before;
      hi -= at << shift;
      if (shift == 0) break;
      const uint32_t width = (1u << shift) - 1;
      lo = hi - lo > width ? hi - width : lo;
    }
    return nth_at(hi, mass ? target / weight_of(unordered(hi)) : target, limit, -1);
  };
  // Counts of the kept tokens in the linear bins, those at positions below hi; hi 0: of all,
  // masked ones too, which are in the last bin.
  auto count = [&](bool limited, float hi) {
    clear(kBins);
    if (hi == 0.f && !limited) {  // (one atomic after another, without a branch)
      each(kLight, [&](const float* v, int) {
#pragma unroll
        for (int i = 0; i < N; ++i) atomicAdd(&sh.bins[linear(v[i])], 1u);
      });
      merge_counts();
      return;
    }
    if (limited) {
      each(kLight, [&](const float* v, int a) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (place(v[i], a + i) >= cut) atomicAdd(&sh.bins[linear(v[i])], 1u);
      });
    } else {
      each(kLight, [&](const float* v, int) {
        float x = v[0];
#pragma unroll
        for (int i = 1; i < N; ++i) x = fmaxf(x, v[i]);
        if (position(x) >= hi) return;  // (most vectors)
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (v[i] > -INFINITY && !(position(v[i]) >= hi)) atomicAdd(&sh.bins[linear(v[i])], 1u);
      });
    }
    merge_counts();
  };
  // The whole rest from a list of every token that can be kept: the first k of them, those with
  // less than `share` before (of the first k's sum, p < 1, where share is 0), the min_p ones.
  auto finish_in_list = [&](int n, int k, float q, int64_t share) {
    if (rank != 0) return;
    const int P = threads_per(n), e = tid / P;  // (n <= kSmall: a round)
    const bool is = e < n, one = is && (tid & (P - 1)) == 0;
    const uint64_t x = is ? sh.merged[e] : ~0ull;
    const int64_t w = is ? sh.merged_w[e] : 0;
    int64_t sum, total;
    bool keep = before_in_list(n, P, x, &sum) < (k > 0 ? (int64_t)k : (int64_t)n) && is;
    if (q < 1.f) {
      if (share == 0) {
        block_scan(one && keep ? w : (int64_t)0, sh.warp_mass, &total);
        share = max((int64_t)ceil((double)fmaxf(q, 0.f) * (double)total), (int64_t)1);
      }
      keep = keep && sum < share;
    }
    keep = keep && w >= least;
    int64_t n_kept;
    block_scan(one && keep ? (int64_t)1 : (int64_t)0, sh.warp_mass, &n_kept);
    block_scan(one && keep ? w : (int64_t)0, sh.warp_mass, &total);
    if (one && !keep) sh.merged_w[e] = 0;
    __syncthreads();
    const int64_t t = min((int64_t)((double)u * (double)total), total - 1);
    sum = 0;  // of the kept ones with a lower index
    for (int j = tid & (P - 1); j < n; j += P)
      sum += (uint32_t)sh.merged[j] > (uint32_t)x ? sh.merged_w[j] : 0;
    for (int o = P / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (one && keep && sum <= t && t < sum + w) p.tokens[b] = (int)(0xFFFFFFFFu - (uint32_t)x);
    if (tid == 0 && p.kept) p.kept[b] = (int)n_kept;
  };

  bool limited = false, counted = false, done = false;
  if (top_k > 0 && top_k < p.V) {
    // (mostly the first part of the span holds k tokens, and most of the others need no count)
    int64_t before, total;
    count(false, (float)(top_k <= 128 ? kBins / 6 : kBins / 3));
    int bin = find(kBins, count_at, (int64_t)top_k - 1, &before, &total);
    if (total < top_k) {
      count(false, NAN);
      bin = find(kBins, count_at, (int64_t)top_k - 1, &before, &total);
      counted = true;
    }
    if (top_k <= total) {
      const int64_t here = count_at(bin);
      if (before + here <= kSmall) {
        const int n = gather(0, bin);
        finish_in_list(n, top_k, top_p, 0);
        done = true;
      } else if (here <= kList) {
        const int n = gather(bin, bin);
        cut = cut_in_list(n, false, (int64_t)top_k - 1 - before);
      } else {
        cut = refine(false, first_key(bin), bin > 0 ? first_key(bin - 1) - 1 : (uint32_t)(top >> 32),
                     (int64_t)top_k - 1 - before);
      }
      limited = true;
      counted = false;
    }
  }
  // ---- top_p; saved: the lanes' sums of the kept tokens are there ----
  bool saved = false;
  int64_t above = 0;
  int n_above = 0, n_own = 0;  // tokens above the window, of the row; more that are kept, the lane's
  int b0 = 0, b1 = kBins - 1;
  if (top_p < 1.f && !done) {
    if (!counted) count(limited, 0.f);
    // The cut's window from the counts: bounds of the running sums (their weights lie within a
    // bin's; 1e-3: roundings of bins and of these sums), and an estimate from the bins' middles.
    // Of a float row's many tokens in a bin the errors cancel, a bf16 row's in one bin are equal:
    // five times the estimate's deviation (0.0025 of a bin's, evenly spread) are a window five to
    // twenty times narrower than the bounds.  A cut outside it (one row in a million; rows whose
    // logits lie on a grid like the bins') is seen, and the bounds taken.
    constexpr int kEach = kBins / kThreads;
    static_assert(kEach == 8, "two vectors of counts a thread");
    uint32_t n_of[kEach];
    *reinterpret_cast<uint4*>(n_of) = reinterpret_cast<const uint4*>(sh.all)[2 * tid];
    *reinterpret_cast<uint4*>(n_of + 4) = reinterpret_cast<const uint4*>(sh.all)[2 * tid + 1];
    // 2^-width: the weights at a bin's two ends; from the bin's middle
    constexpr float kRatio = bin_ratio(1.0), kMiddle = bin_ratio(0.5);
    const float first = ex2(-(kSpan / (float)(kBins - 1)) * (float)(tid * kEach));
    // prefix sums over the block, a thread for kEach bins: the masses' bounds and estimate, and the
    // counts; the variances' sum
    float up[4] = {0.f, 0.f, 0.f, 0.f}, all[4];
    int up_n = 0;
    auto add_bins = [&](auto fn) {
      float high = first;
#pragma unroll
      for (int i = 0; i < kEach; ++i, high *= kRatio) {
        const int bin = tid * kEach + i;
        const float n = (float)n_of[i], w = n * (high * kMiddle);
        up[0] += bin < kBins - 1 ? n * (high * kRatio) : 0.f;
        up[1] += n * high;
        up[2] += w;
        up[3] += sizeof(T) == 2 ? w * w : w * w / fmaxf(n, 1.f);
        up_n += (int)n_of[i];
        fn(bin);
      }
    };
    add_bins([](int) {});
    {
      float to[4];
      int to_n = up_n;
#pragma unroll
      for (int i = 0; i < 4; ++i) to[i] = up[i];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float below = __shfl_up_sync(0xffffffffu, to[i], o);
          if (lane >= o) to[i] += below;
        }
        const int below = __shfl_up_sync(0xffffffffu, to_n, o);
        if (lane >= o) to_n += below;
      }
      if (lane == 31) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sh.warp_up[i][warp] = to[i];
        sh.warp_n[warp] = to_n;
      }
      if (tid < 4) sh.window[tid] = kBins - 1;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float part = lane < kWarps ? sh.warp_up[i][lane] : 0.f;
        all[i] = warp_sum(part);
        up[i] = to[i] - up[i] + warp_sum(lane < warp ? part : 0.f);
      }
      up_n = to_n - up_n + warp_sum(lane < warp ? sh.warp_n[lane & (kWarps - 1)] : 0);
    }
    const float q = fmaxf(top_p, 0.f);
    const float margin = 5.f * 0.0025f * sqrtf(all[3]) + 1e-5f * all[2];
    // the first bins at which a running sum reaches a place: the bounds' ends, the estimate's
    const float t[4] = {q * all[0] * 0.999f, q * all[1] * 1.001f, q * all[2] - margin, q * all[2] + margin};
    int at[4] = {kBins - 1, kBins - 1, kBins - 1, kBins - 1};
    const int n_first = up_n;  // tokens before this thread's bins
    add_bins([&](int bin) {
      if (up[1] >= t[0]) at[0] = min(at[0], bin);
      if (up[0] >= t[1]) at[1] = min(at[1], bin);
      if (up[2] >= t[2]) at[2] = min(at[2], bin);
      if (up[2] >= t[3]) at[3] = min(at[3], bin);
    });
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      at[i] = __reduce_min_sync(0xffffffffu, at[i]);
      if (lane == 0) atomicMin(&sh.window[i], at[i]);
    }
    __syncthreads();
    const int bound0 = sh.window[0], bound1 = max(sh.window[1], bound0);
    b0 = min(max(sh.window[2], bound0), bound1);
    b1 = min(max(sh.window[3], b0), bound1);
    // tokens before the bounds, in front of the window and up to the bounds' end, by the threads
    // that have those bins
    const int ends[3] = {bound0, b0, bound1 + 1};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if ((ends[k] - (k == 2)) / kEach != tid) continue;
      int n = n_first;
#pragma unroll
      for (int i = 0; i < kEach; ++i) n += tid * kEach + i < ends[k] ? (int)n_of[i] : 0;
      sh.n_before[k] = n;
    }
    __syncthreads();
    const int n_bound0 = sh.n_before[0], n_cand = sh.n_before[2];
    n_above = sh.n_before[1];
    const bool small = n_cand <= kSmall;
    if (small) {
      b0 = bound0;
      b1 = bound1;
    }
    for (;;) {
      // exact sums: of the row, of the tokens above the window, and of the window's in finer bins
      // (linear over b0 .. b1).  The window as logits: over is the largest, under the smallest in it.
      const float from = (float)b0, scale = (float)kFine / (float)(b1 - b0 + 1);
      const float over = b0 > 0 ? unordered(first_key(b0 - 1) - 1) : INFINITY;
      const float under = unordered(first_key(b1));
      auto fine = [&](float v) { return min(max((int)((position(v) - from) * scale), 0), kFine - 1); };
      auto in_window = [&](float v) { return (v <= over) & (v >= under); };
      if (tid == 0) sh.too_many = 0;
      __syncthreads();
      int64_t sum = 0;
      above = 0;
      int n_window = 0;  // the warp's tokens of the window
      int all_h = 0, all_l = 0, up_h = 0, up_l = 0, held = 0;
      auto widen = [&]() {
        sum += units({all_h, all_l});
        above += units({up_h, up_l});
        all_h = all_l = up_h = up_l = 0;
      };
      auto collect = [&](const float* v, int a, bool any) {
        if (!__any_sync(0xffffffffu, any)) return;
#pragma unroll
        for (int i = 0; i < kSome; ++i) {
          bool in = in_window(v[i]);
          if (limited) in = in && place(v[i], a + i) >= cut;
          const uint32_t who = __ballot_sync(0xffffffffu, in);
          if (who == 0u) continue;
          const int place_of = n_window + __popc(who & ((1u << lane) - 1u));
          if (in && place_of < kWindow) sh.window_of[warp][place_of] = place(v[i], a + i);
          n_window += __popc(who);
        }
      };
      // (of a limited row all tokens above the window are kept: the cut lies in it)
      if (tabled) {
        make_values();
        each(kDear, [&](const float* v, int a) {
          bool any = false;
          int64_t w[kSome];
          value_weights(v, w);
          if (limited) {
#pragma unroll
            for (int i = 0; i < kSome; ++i) w[i] = place(v[i], a + i) < cut ? 0 : w[i];
          }
#pragma unroll
          for (int i = 0; i < kSome; ++i) {
            sum += w[i];
            above += v[i] > over ? w[i] : 0;
            any |= in_window(v[i]);
          }
          collect(v, a, any);
        });
      } else {
        each(kDear, [&](const float* v, int a) {
          Weight w[kSome];
          weights_of(v, w);
          if (limited) {
#pragma unroll
            for (int i = 0; i < kSome; ++i)
              if (place(v[i], a + i) < cut) w[i] = {0, 0};
          }
          if ((++held & (kHold - 1)) == 0) widen();
          bool any = false;
#pragma unroll
          for (int i = 0; i < kSome; ++i) {
            all_h += w[i].high;
            all_l += w[i].low;
            if (v[i] > over) {
              up_h += w[i].high;
              up_l += w[i].low;
            }
            any |= in_window(v[i]);
          }
          collect(v, a, any);
        });
      }
      widen();
      if (n_window > kWindow && lane == 0) sh.too_many = 1;
      int64_t W = sum, all_above = above, too_many = 0;
      __syncthreads();
      if (tid == 0) too_many = sh.too_many;
      totals_of(W, all_above, too_many);
      const int64_t share = min(max((int64_t)ceil((double)q * (double)W), (int64_t)1), W);
      if (small) {
        const int n = gather(0, b1);
        finish_in_list(n, 0, top_p, share);
        done = true;
      } else {
        // the window's tokens: what the warps have kept, or the row once more
        auto each_in_window = [&](auto fn) {
          if (too_many == 0) {
#pragma unroll 1
            for (int i = lane; i < n_window; i += 32) {
              const uint64_t x = sh.window_of[warp][i];
              fn(unordered((uint32_t)(x >> 32)), (int)(0xFFFFFFFFu - (uint32_t)x));
            }
            return;
          }
          each(kDear, [&](const float* v, int a) {
#pragma unroll
            for (int i = 0; i < kSome; ++i) {
              if (in_window(v[i]) && place(v[i], a + i) >= cut) fn(v[i], a + i);
            }
          });
        };
        int64_t target = share - 1 - all_above, before, total;
        bool listed = true;
        auto missed = [&]() { return (target < 0 || target >= total) && (b0 != bound0 || b1 != bound1); };
        if constexpr (sizeof(T) == 2) {
          // by value, one a bin (where the window holds values next to 0 in steps)
          uint32_t first16 = (b0 > 0 ? ordered(over) : (uint32_t)(top >> 32)) >> 16;
          uint32_t last16 = ordered(under) >> 16;
          bool again = false;
#pragma unroll 1
          for (int step = 0; step < 2; ++step) {  // (2^16 values, kFine bins)
            int shift = 0;
            while (((first16 - last16) >> shift) >= (uint32_t)kFine) ++shift;
            clear(2 * kFine);
            each_in_window([&](float v, int) {
              const uint32_t key16 = ordered(v) >> 16;
              if (key16 > first16 || key16 < last16) return;
              const int64_t w = weight_of(v);
              if (w > 0) add_mass((int)((first16 - key16) >> shift), (uint64_t)w);
            });
            merge_mass();
            const uint32_t at = (uint32_t)find(kFine, mass_at, target, &before, &total);
            again = missed();
            if (again) break;
            target -= before;
            first16 -= at << shift;
            if (shift == 0) break;
            last16 = max(last16, first16 - (1u << shift) + 1);
          }
          if (again) {
            b0 = bound0;
            b1 = bound1;
            n_above = n_bound0;
            continue;
          }
          const uint32_t key = first16 << 16 | (first16 & 0x8000u ? 0u : 0xFFFFu);
          cut = nth_at(key, target / max(weight_of(unordered(key)), (int64_t)1), cut,
                       too_many == 0 ? n_window : -1);
        } else {
          clear(2 * kFine);
          each_in_window([&](float v, int) {
            const int64_t w = weight_of(v);
            if (w > 0) add_mass(fine(v), (uint64_t)w);
          });
          merge_mass();
          const int bin = find(kFine, mass_at, target, &before, &total);
          if (missed()) {
            b0 = bound0;
            b1 = bound1;
            n_above = n_bound0;
            continue;
          }
          // the tokens of the cut's bin go on a list
          start_list();
          each_in_window([&](float v, int index) {
            if (fine(v) == bin) put_on_list(v, index);
          });
          const int n = join_lists();
          listed = n <= kList;
          cut = listed ? cut_in_list(n, true, target - before)
                       : refine(true, ordered(under), b0 > 0 ? ordered(over) : (uint32_t)(top >> 32), target);
        }
        saved = mp == 0.f && listed;
        if (saved) {
          each_in_window([&](float v, int index) {
            if (place(v, index) < cut) return;
            above += weight_of(v);
            ++n_own;
          });
        }
      }
      break;
    }
  }
  // (not earlier: a next call's first CTAs, the long rows', would take their places two by two on the
  // SMs that are done first; mixed rows, call after call: 78 us that way, 63 this way)
  griddep_launch_dependents();
  if (!done) {
    // ---- the kept tokens' sums by warps, then the draw in index order ----
    auto kept_weight = [&](float v, int index) {  // -1: not kept
      if (place(v, index) < cut || (m - v) * ch > far) return (int64_t)-1;
      const int64_t w = weight_of(v);
      return w >= least ? w : (int64_t)-1;
    };
    int64_t mass = saved ? above : 0;
    int n_kept = saved ? n_own : 0;
    if (!saved && cut == kMasked + 1 && mp == 0.f && tabled) {  // no filter
      make_values();
      each(kDear, [&](const float* v, int) {
        int64_t w[kSome];
        value_weights(v, w);
#pragma unroll
        for (int i = 0; i < kSome; ++i) {
          mass += w[i];
          n_kept += v[i] > -INFINITY;
        }
      });
    } else if (!saved && cut == kMasked + 1 && mp == 0.f) {
      int h = 0, l = 0, held = 0;
      each(kDear, [&](const float* v, int) {
        Weight w[kSome];
        weights_of(v, w);
#pragma unroll
        for (int i = 0; i < kSome; ++i) {
          h += w[i].high;
          l += w[i].low;
        }
        float x = v[0];
#pragma unroll
        for (int i = 1; i < kSome; ++i) x = fminf(x, v[i]);
        n_kept += kSome;
        if (x == -INFINITY) {  // (few vectors have a masked token)
#pragma unroll
          for (int i = 0; i < kSome; ++i) n_kept -= v[i] == -INFINITY;
        }
        if ((++held & (kHold - 1)) == 0) {
          mass += units({h, l});
          h = l = 0;
        }
      });
      mass += units({h, l});
    } else if (!saved) {
      const float cut_value = unordered((uint32_t)(cut >> 32));
      each(kLight, [&](const float* v, int a) {
        float x = v[0];  // (few vectors have one: their largest then is)
#pragma unroll
        for (int i = 1; i < N; ++i) x = fmaxf(x, v[i]);
        if (!(x >= cut_value) || (m - x) * ch > far) return;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int64_t w = kept_weight(v[i], a + i);
          if (w < 0) continue;
          mass += w;
          ++n_kept;
        }
      });
    }
    mass = warp_sum(mass);
    n_kept = warp_sum(n_kept);
    __syncthreads();
    if (lane == 0) {
      sh.warp_mass[warp] = mass;
      sh.warp_count[warp] = n_kept;
    }
    __syncthreads();
    if (warp == 0) {
      mass = warp_sum(lane < kWarps ? sh.warp_mass[lane] : (int64_t)0);
      n_kept = warp_sum(lane < kWarps ? sh.warp_count[lane] : 0);
      if (C == 1) {
        if (lane == 0) {
          sh.mass[3][0] = mass;
          sh.count[0] = n_kept;
        }
      } else if (lane < C) {
        st_cluster_u64(&sh.mass[3][rank], (uint32_t)lane, (uint64_t)mass);
        st_cluster_u32(&sh.count[rank], (uint32_t)lane, (uint32_t)n_kept);
      }
    }
    sync();
    const int64_t part = lane < C ? sh.mass[3][lane] : 0;
    const int64_t W = warp_sum(part);
    int64_t t = min((int64_t)((double)u * (double)W), W - 1);
    const int owner = locate(part, C, &t);
    n_kept = warp_sum(lane < C ? sh.count[lane] : 0) + (saved ? n_above : 0);
    if (rank == 0 && tid == 0 && p.kept) p.kept[b] = n_kept;
    // the owner's threads look through the slice of the warp that holds the place, a vector each
    if (owner == rank) {
      const int at_w = locate(lane < kWarps ? sh.warp_mass[lane] : (int64_t)0, kWarps, &t);
      const int y0 = min(c1, c0 + at_w * per_w), y1 = min(c1, y0 + per_w);
      for (int j0 = y0; j0 < y1; j0 += kThreads) {
        const int j = j0 + tid, a = (int)row.first(j);
        int64_t e[N], sum = 0, all;
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = 0;
        if (j < y1) {
          float v[N];
          Weight w[N];
          Vec<T>::unpack(vector(j), v);
#pragma unroll
          for (int i = 0; i < N; i += kSome) weights_of(v + i, w + i);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            e[i] = units(w[i]);
            if (e[i] < least || place(v[i], a + i) < cut) e[i] = 0;
          }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) sum += e[i];
        int64_t here = t - block_scan(sum, sh.warp_mass, &all);
        t -= all;
        if (here >= 0 && here < sum) {
          int at = 0;
          bool hit = false;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            if (!hit && here < e[i]) {
              hit = true;
              at = i;
            }
            if (!hit) here -= e[i];
          }
          p.tokens[b] = a + at;
        }
      }
    }
  }
  if (C > 1) cluster_sync();  // no CTA leaves while another may still read from it
}

template <typename T>
cudaError_t launch(const TokenParams& p, int B, int C, cudaStream_t st) {
  constexpr int smem = (int)sizeof(Shared);
  cudaError_t e = cudaFuncSetAttribute(token_sample_kernel<T>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && C > 8)
    e = cudaFuncSetAttribute(token_sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)B * (unsigned)C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  int log2_C = 0;
  while ((1 << log2_C) < C) ++log2_C;
  return cudaLaunchKernelEx(&cfg, token_sample_kernel<T>, p, log2_C);
}

}  // namespace

cudaError_t launch_token_sample(const tv_token_args* a, int sm_count, cudaStream_t st) {
  if (a->B == 0) return cudaSuccess;
  TokenParams p{};
  p.logits = a->logits;
  p.V = a->vocab;
  p.stride = a->logits_row_stride;
  p.temperature = a->temperature;
  p.top_k = a->top_k;
  p.top_p = a->top_p;
  p.min_p = a->min_p;
  p.uniforms = a->uniforms;
  p.tokens = a->tokens;
  p.kept = a->kept;
  p.status = a->status;
  // CTAs per row: up to the two per SM that fit at once, while a thread has 28 tokens or more (16 x
  // 50257 floats, top-k: 4 CTAs of a row 17 us, 8 CTAs 19); 16 only for a few rows: clusters of
  // that size hardly fit side by side (16 x 50257: 38 us; 1 x 163840, top-p: 34 against 40 with 8).
  int C = 1;
  const int most = a->B <= 4 ? kMaxCluster : kMaxCluster / 2;
  while (C < most && (int64_t)a->B * C <= sm_count && a->vocab >= 28ll * kThreads * C) C *= 2;
  p.B = a->B;
  p.sorted = p.top_p && a->B <= kSorted && (int64_t)a->B * C > sm_count;
  return a->logits_dt == TV_BF16 ? launch<__nv_bfloat16>(p, a->B, C, st) : launch<float>(p, a->B, C, st);
}

}  // namespace tv
