// k_token.cu -- next tokens with temperature, top-k, top-p and min-p (tv_token_sample).
//
// All filters keep a beginning of one order, falling logit and then index, so what they leave
// is a cut: every token above a logit, and the first few (by index) of those equal to it.
// top_k's cut is the k-th token's; top_p's the token at which the running sum of weights reaches
// p W, W the sum of what top_k keeps; min_p is a bound on the weight itself.  The token is then
// drawn in index order from what is kept.
//
// Finding a cut.  A row's tokens are counted (top_k) or their weights summed (top_p) in kBins
// bins of falling logit; the bin in which the running total passes the target is found, and its
// tokens are binned again, finer, until a bin is a single logit.  The first bins are linear in
// the logit (kSpan units of log2 of the weight, and one bin for all below), which spreads a
// model's logits evenly; the next ones cut the ordered bit patterns between that bin's smallest
// and largest: one level more for bf16, mostly two for float32, four at worst.  Weights are the
// exact integers of tv_tree_sample (sample_math.h), added in three parts of 15 bits, whose sums
// over a slice of 2^16 tokens stay within 32 bits: sums in any order, results that do not depend
// on it.
//
// Work.  A cluster of CTAs shares a row.  Every CTA reads its contiguous slice once into shared
// memory and works on it there.  Per level the CTAs' bins are added up by parts (each CTA the
// same share of bins, through distributed shared memory), the parts' totals exchanged, and the
// owner of the passing bin tells the others.
#include <cuda_bf16.h>

#include <algorithm>

#include "sample_math.h"
#include "sm100_ptx.h"
#include "tv_internal.h"

namespace tv {
namespace {

using namespace ptx;

constexpr int kMaxCluster = 16;
constexpr int kMaxWarps = 16;
constexpr int kBins = 1024;
constexpr float kSpan = 48.f;  // log2 units of the linear bins: below, weights are zero
constexpr int kSliceBytes = 64 * 1024;  // of a row per CTA: 2^18 floats by 16 CTAs

struct TokenParams {
  const void* logits;
  int64_t V, stride;
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
  float2 exp2_table[kTable * kCopies];
  uint32_t bins[3][kBins];        // counts, or 15-bit parts of the weights' sums
  int64_t own[kBins];             // this CTA's share of the bins, over all CTAs
  uint64_t keys[kMaxCluster];     // exchanged: the slices' maxima,
  int64_t totals[kMaxCluster];    // their sums of a share of bins,
  int64_t found[2];               // the bin that a target lies in, and what is left of it,
  int64_t mass[kMaxCluster];      // sums of the kept tokens above the cut,
  int32_t count[kMaxCluster];     // how many they are,
  int32_t ties[kMaxCluster];      // and how many tokens lie on it
  uint64_t warp_key[kMaxWarps];
  int64_t warp_mass[kMaxWarps];
  int32_t warp_count[kMaxWarps], warp_ties[kMaxWarps];
};

// Ordered keys of a type's values: 32 bits, or the upper 16 of a bf16.
template <typename T>
struct Key {
  static constexpr int kShift = sizeof(T) == 2 ? 16 : 0;
  __device__ static uint32_t of(float v) { return ordered(v) >> kShift; }
  __device__ static float value(uint32_t k) {
    const bool pos = k >> (31 - kShift);
    return unordered(sizeof(T) == 2 ? (k << 16) | (pos ? 0u : 0xFFFFu) : k);
  }
  static constexpr uint32_t kMasked = 0x007FFFFFu >> kShift;  // of -inf
  static constexpr uint32_t kTop = 0xFF800000u >> kShift;     // of +inf
};

__device__ __forceinline__ uint32_t ld_cluster_u32(const void* local, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_to_rank(smem_u32(local), rank)) : "memory");
  return v;
}

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
    token_sample_kernel(const TokenParams p, int log2_C) {
  constexpr int kWarps = kThreads / 32, N = Vec<T>::N;
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  uint4* slice = reinterpret_cast<uint4*>(smem + (sizeof(Shared) + 15) / 16 * 16);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = 1 << log2_C, b = blockIdx.x >> log2_C;
  const int rank = C > 1 ? (int)cluster_rank() : 0;
  griddep_wait();
  griddep_launch_dependents();
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
  for (int i = tid; i < kTable * kCopies; i += kThreads)
    sh.exp2_table[i] = make_float2(d_exp.hi[i / kCopies], d_exp.lo[i / kCopies]);
  constexpr float l2e = (float)(1.0 / kLn2), l2e_low = (float)(1.0 / kLn2 - (double)l2e);
  const float cq = l2e / T0;
  const float ch = fminf(fmaxf(cq, 1e-30f), 1e30f);
  const float cl = ch == cq ? (fmaf(-cq, T0, l2e) + l2e_low) / T0 : 0.f;

  // ---- the slice into shared memory, and the row's maximum with its first index ----
  const Row<T> row((const T*)p.logits + (int64_t)b * p.stride, p.V);
  const int per = (row.n_vec + C - 1) >> log2_C;
  const int c0 = min(row.n_vec, rank * per), n_vec = min(row.n_vec, c0 + per) - c0;
  {
    float best = -INFINITY;
    int best_at = 0;
    bool is_nan = false;
    constexpr int kUnroll = 8;
    for (int j0 = tid; j0 < n_vec; j0 += kUnroll * kThreads) {
      uint4 w[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int j = j0 + k * kThreads;
        if (j >= n_vec) break;
        if (row.whole(c0 + j)) {
          w[k] = row.raw(c0 + j);
        } else {  // an end of the row
          const int64_t a = row.first(c0 + j);
          alignas(16) T v[N];
#pragma unroll
          for (int i = 0; i < N; ++i)
            v[i] = a + i >= 0 && a + i < p.V ? row.x[a + i] : (T)-INFINITY;
          w[k] = *reinterpret_cast<const uint4*>(v);
        }
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int j = j0 + k * kThreads;
        if (j >= n_vec) break;
        slice[j] = w[k];
        float v[N];
        Vec<T>::unpack(w[k], v);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          is_nan |= v[i] != v[i];
          if (v[i] > best) {
            best = v[i];
            best_at = (int)row.first(c0 + j) + i;
          }
        }
      }
    }
    // order-preserving value bits, then the complemented index; a NaN beats every value
    uint64_t key = best > -INFINITY
                       ? ((uint64_t)ordered(best) << 32) | (0xFFFFFFFFu - (uint32_t)best_at)
                       : 0ull;
    key = warp_max(key);
    if (__any_sync(0xffffffffu, is_nan)) key = ~0ull;
    if (lane == 0) sh.warp_key[warp] = key;
    if (C > 1) cluster_wait();
    __syncthreads();
    if (warp == 0) {
      key = warp_max(lane < kWarps ? sh.warp_key[lane] : 0ull);
      if (C == 1) {
        if (lane == 0) sh.keys[0] = key;
      } else if (lane < C) {
        st_cluster_u64(&sh.keys[rank], (uint32_t)lane, key);
      }
    }
    if (C > 1) cluster_sync();
    else __syncthreads();
  }
  const uint64_t top = warp_max(lane < C ? sh.keys[lane] : 0ull);
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

  // ---- the cut: keys above cut_key are kept, and the first `ties` tokens at it ----
  uint32_t cut_key = Key<T>::kMasked;
  int64_t ties = 0;
  const float per_bin = ch * ((float)(kBins - 1) / kSpan);
  auto weight_of = [&](float v) { return units(weight(v, m, ch, cl, sh.exp2_table)); };
  // the linear bin of a value: falling in it, so that a bin is a range of keys
  auto linear = [&](float v) { return min((int)((m - v) * per_bin), kBins - 1); };

  // Adds up the bins of the tokens above cut_key whose keys lie in [lo, hi]: counts (mass false)
  // or weights.  Returns the total; then sh.totals holds the shares' and sh.own this one's.
  const int share = kBins >> log2_C;
  auto collect = [&](bool mass, bool first, uint32_t lo, uint32_t hi, int shift) {
    const int words = mass ? 3 : 1;
    for (int i = tid; i < words * kBins; i += kThreads) (&sh.bins[0][0])[i] = 0u;
    __syncthreads();
    for (int j = tid; j < n_vec; j += kThreads) {
      float v[N];
      Vec<T>::unpack(slice[j], v);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t key = Key<T>::of(v[i]);
        if (key <= cut_key || key < lo || key > hi) continue;
        const int bin = first ? linear(v[i]) : (int)((hi - key) >> shift);
        if (!mass) {
          atomicAdd(&sh.bins[0][bin], 1u);
          continue;
        }
        const uint64_t w = (uint64_t)weight_of(v[i]);
        if (w == 0) continue;
        atomicAdd(&sh.bins[0][bin], (uint32_t)w & 0x7FFFu);
        atomicAdd(&sh.bins[1][bin], (uint32_t)(w >> 15) & 0x7FFFu);
        atomicAdd(&sh.bins[2][bin], (uint32_t)(w >> 30));
      }
    }
    if (C > 1) cluster_sync();
    else __syncthreads();
    // this CTA's share of the bins: P threads a bin, each adding C / P of the CTAs'
    const int P = min(C, max(1, kThreads / share));
    int64_t total = 0;
    for (int i = tid / P; i < share; i += kThreads / P) {
      const int at = rank * share + i;
      int64_t s = 0;
      for (int r = tid % P; r < C; r += P) {
        if (C == 1) {
          s += sh.bins[0][at];
          if (mass) s += ((int64_t)sh.bins[1][at] << 15) + ((int64_t)sh.bins[2][at] << 30);
        } else {
          s += ld_cluster_u32(&sh.bins[0][at], (uint32_t)r);
          if (mass)
            s += ((int64_t)ld_cluster_u32(&sh.bins[1][at], (uint32_t)r) << 15) +
                 ((int64_t)ld_cluster_u32(&sh.bins[2][at], (uint32_t)r) << 30);
        }
      }
      for (int o = P / 2; o > 0; o >>= 1) s += __shfl_xor_sync(__activemask(), s, o);
      if (tid % P == 0) {
        sh.own[i] = s;
        total += s;
      }
    }
    total = warp_sum(total);
    if (lane == 0) sh.warp_mass[warp] = total;
    __syncthreads();
    if (warp == 0) {
      total = warp_sum(lane < kWarps ? sh.warp_mass[lane] : (int64_t)0);
      if (C == 1) {
        if (lane == 0) sh.totals[0] = total;
      } else if (lane < C) {
        st_cluster_u64(&sh.totals[rank], (uint32_t)lane, (uint64_t)total);
      }
    }
    if (C > 1) cluster_sync();
    else __syncthreads();
    return warp_sum(lane < C ? sh.totals[lane] : (int64_t)0);
  };
  // The bin in which the running total passes `target`, which becomes what is left of it there.
  auto find = [&](int64_t* target) {
    int64_t t = *target;
    const int owner = locate(lane < C ? sh.totals[lane] : (int64_t)0, C, &t);
    if (owner == rank && warp == 0) {
      int bin = 0;
      for (int i0 = 0; i0 < share; i0 += 32) {
        const int n = min(32, share - i0);
        const int64_t part = lane < n ? sh.own[i0 + lane] : 0;
        const int64_t all = warp_sum(part);
        if (t >= all && i0 + 32 < share) {
          t -= all;
          continue;
        }
        bin = i0 + locate(part, n, &t);
        break;
      }
      if (C == 1) {
        if (lane == 0) {
          sh.found[0] = bin;
          sh.found[1] = t;
        }
      } else if (lane < C) {
        st_cluster_u64(&sh.found[0], (uint32_t)lane, (uint64_t)(rank * share + bin));
        st_cluster_u64(&sh.found[1], (uint32_t)lane, (uint64_t)t);
      }
    }
    if (C > 1) cluster_sync();
    else __syncthreads();
    *target = sh.found[1];
    return (int)sh.found[0];
  };
  // The smallest key whose linear bin is at most `bin`, by one probe a lane.
  auto first_key = [&](int bin) {
    uint32_t lo = Key<T>::kMasked + 1, hi = Key<T>::of(m);  // linear(hi) = 0
    while (lo < hi) {
      const uint32_t step = (hi - lo + 31) / 32, probe = min(hi, lo + (uint32_t)lane * step);
      const uint32_t in = __ballot_sync(0xffffffffu, linear(Key<T>::value(probe)) <= bin);
      const int at = __ffs(in) - 1;  // (none: the answer lies above the last probe)
      if (at == 0) return lo;
      const uint32_t below = lo + (uint32_t)(at < 0 ? 31 : at - 1) * step;
      hi = at < 0 ? hi : min(hi, lo + (uint32_t)at * step);
      lo = min(hi, below + 1);
    }
    return lo;
  };
  // Moves the cut to where the running total passes `target`, given the linear bins' totals.
  auto narrow = [&](bool mass, int64_t target) {
    const int bin = find(&target);
    uint32_t lo = first_key(bin), hi = bin > 0 ? first_key(bin - 1) - 1 : Key<T>::of(m);
    for (;;) {
      int shift = 0;
      while (((hi - lo) >> shift) >= (uint32_t)kBins) ++shift;
      collect(mass, false, lo, hi, shift);
      const uint32_t at = (uint32_t)find(&target);
      hi -= at << shift;
      if (shift == 0) break;
      const uint32_t width = (1u << shift) - 1;
      lo = hi - lo > width ? hi - width : lo;
    }
    cut_key = hi;
    // target: what the tokens at the cut may sum to before the last kept one
    ties = mass ? target / weight_of(Key<T>::value(hi)) + 1 : target + 1;
  };

  if (top_k > 0 && top_k < p.V) {
    const int64_t n = collect(false, true, 0u, Key<T>::kTop, 0);
    if (top_k < n) narrow(false, (int64_t)top_k - 1);
  }
  if (top_p < 1.f) {
    const int64_t above = collect(true, true, 0u, Key<T>::kTop, 0);
    const int64_t tie = ties > 0 ? weight_of(Key<T>::value(cut_key)) : 0;
    const int64_t W = above + ties * tie;
    const int64_t share_of = (int64_t)ceil((double)fmaxf(top_p, 0.f) * (double)W);
    const int64_t target = min(max(share_of, (int64_t)1), W) - 1;
    if (target < above) narrow(true, target);
    else ties = min(ties, (target - above) / tie + 1);
  }
  const float mp = fminf(fmaxf(min_p, 0.f), 1.f);
  const int64_t least = (int64_t)ceil((double)mp * (double)kUnit);
  // (a token this far below the maximum is lighter than min_p without more ado)
  const float far = mp > 0.f ? fminf(-__log2f(mp) * 1.0001f + 0.01f, 64.f) : INFINITY;
  const int64_t tie = ties > 0 ? weight_of(Key<T>::value(cut_key)) : 0;
  if (tie < least) ties = 0;

  // ---- the kept tokens' sums by warps' slices, then the draw in index order ----
  const int per_w = (per + kWarps - 1) / kWarps;
  const int w0 = min(n_vec, warp * per_w), w1 = min(n_vec, w0 + per_w);
  auto above = [&](float v, uint32_t key) {  // weight of a token above the cut, -1: not kept
    if (key <= cut_key || (m - v) * ch > far) return (int64_t)-1;
    const int64_t w = weight_of(v);
    return w >= least ? w : (int64_t)-1;
  };
  {
    int64_t mass = 0;
    int count = 0, on_cut = 0;
    for (int j = w0 + lane; j < w1; j += 32) {
      float v[N];
      Vec<T>::unpack(slice[j], v);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t key = Key<T>::of(v[i]);
        on_cut += key == cut_key && ties > 0;
        const int64_t w = above(v[i], key);
        if (w < 0) continue;
        mass += w;
        ++count;
      }
    }
    mass = warp_sum(mass);
    count = warp_sum(count);
    on_cut = warp_sum(on_cut);
    if (lane == 0) {
      sh.warp_mass[warp] = mass;
      sh.warp_count[warp] = count;
      sh.warp_ties[warp] = on_cut;
    }
    __syncthreads();
    if (warp == 0) {
      mass = warp_sum(lane < kWarps ? sh.warp_mass[lane] : (int64_t)0);
      count = warp_sum(lane < kWarps ? sh.warp_count[lane] : 0);
      on_cut = warp_sum(lane < kWarps ? sh.warp_ties[lane] : 0);
      if (C == 1) {
        if (lane == 0) {
          sh.mass[0] = mass;
          sh.count[0] = count;
          sh.ties[0] = on_cut;
        }
      } else if (lane < C) {
        st_cluster_u64(&sh.mass[rank], (uint32_t)lane, (uint64_t)mass);
        st_cluster_u32(&sh.count[rank], (uint32_t)lane, (uint32_t)count);
        st_cluster_u32(&sh.ties[rank], (uint32_t)lane, (uint32_t)on_cut);
      }
    }
    if (C > 1) cluster_sync();
    else __syncthreads();
  }
  if (warp == 0) {
    // of parts in index order, lane i holding part i's tokens on the cut: how many are kept,
    // with `before` of them taken already
    auto kept_ties = [&](int on_cut, int64_t before) {
      int64_t up_to = on_cut;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t below = __shfl_up_sync(0xffffffffu, up_to, o);
        if (lane >= o) up_to += below;
      }
      return min(max(ties - before - (up_to - on_cut), (int64_t)0), (int64_t)on_cut);
    };
    const int q = lane < C ? sh.ties[lane] : 0;
    int64_t k = kept_ties(q, 0);
    int64_t part = lane < C ? sh.mass[lane] + k * tie : 0;
    const int64_t W = warp_sum(part);
    const int64_t n = warp_sum((lane < C ? (int64_t)sh.count[lane] : 0) + k);
    int64_t t = min((int64_t)((double)u * (double)W), W - 1);
    const int owner = locate(part, C, &t);
    if (rank == 0 && lane == 0 && p.kept) p.kept[b] = (int)n;
    if (owner == rank) {
      int64_t before = warp_sum(lane < rank ? (int64_t)q : (int64_t)0);
      const int qw = lane < kWarps ? sh.warp_ties[lane] : 0;
      k = kept_ties(qw, before);
      part = lane < kWarps ? sh.warp_mass[lane] + k * tie : 0;
      const int w = locate(part, kWarps, &t);
      before += warp_sum(lane < w ? (int64_t)qw : (int64_t)0);
      const int y0 = min(n_vec, w * per_w), y1 = min(n_vec, y0 + per_w);
      for (int j0 = y0; j0 < y1; j0 += 32) {  // a vector per lane
        const int j = j0 + lane;
        float v[N];
        int64_t e[N], sum = 0;
        int on_cut = 0;
        if (j < y1) {
          Vec<T>::unpack(slice[j], v);
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) v[i] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) on_cut += Key<T>::of(v[i]) == cut_key && ties > 0;
        k = kept_ties(on_cut, before);
        int64_t left = k;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const uint32_t key = Key<T>::of(v[i]);
          e[i] = max(above(v[i], key), (int64_t)0);
          if (key == cut_key && left > 0) {
            e[i] = tie;
            --left;
          }
          sum += e[i];
        }
        const int64_t all = warp_sum(sum);
        if (t >= all && j0 + 32 < y1) {
          t -= all;
          before += warp_sum((int64_t)on_cut);
          continue;
        }
        const int at = locate(sum, 32, &t);
        if (lane == at) {
          int i = 0;
          bool hit = false;
#pragma unroll
          for (int x = 0; x < N; ++x) {
            if (!hit && t < e[x]) {
              hit = true;
              i = x;
            }
            if (!hit) t -= e[x];
          }
          p.tokens[b] = (int)row.first(c0 + j) + i;
        }
        break;
      }
    }
  }
  if (C > 1) cluster_sync();  // no CTA leaves while another may still read from it
}

template <typename T, int kThreads>
cudaError_t launch(const TokenParams& p, int B, int C, size_t smem, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(token_sample_kernel<T, kThreads>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess && C > 8)
    e = cudaFuncSetAttribute(token_sample_kernel<T, kThreads>,
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
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
  return cudaLaunchKernelEx(&cfg, token_sample_kernel<T, kThreads>, p, log2_C);
}

template <typename T>
cudaError_t launch(const TokenParams& p, int B, int sm_count, cudaStream_t st) {
  constexpr int N = Vec<T>::N;
  // CTAs per row: enough that a slice fits, then more while the GPU is not full and a thread has
  // several vectors to read
  auto per = [&](int C) { return ((p.V + N - 1) / N + 1 + C - 1) / C; };  // vectors of a slice
  int C = 1;
  while (C < kMaxCluster && per(C) * 16 > kSliceBytes) C *= 2;
  while (C < kMaxCluster && (int64_t)B * C * 2 <= 2ll * sm_count && per(C) >= 512) C *= 2;
  const size_t smem = (sizeof(Shared) + 15) / 16 * 16 + (size_t)per(C) * 16;
  return launch<T, 512>(p, B, C, smem, st);
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
  return a->logits_dt == TV_BF16 ? launch<__nv_bfloat16>(p, a->B, sm_count, st)
                                 : launch<float>(p, a->B, sm_count, st);
}

}  // namespace tv
