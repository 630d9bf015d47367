// k_sample.cu -- sampled acceptance of a verified draft tree (tv_tree_sample).
//
// The walk starts at the root.  At node n the target's distribution is
// p = softmax(logits[n] / T).  The children of n are tested in index order with their own
// uniform numbers; with weights w (w = p at first, W their sum)
//   no draft probabilities:  accept child c iff  u_c W < w[x_c]; else w[x_c] = 0
//   draft probabilities g (G = 1 at first):
//                            accept child c iff  u_c g[x_c] W < w[x_c] G;
//                            else w = max(w - g W/G, 0), G -= g[x_c], g[x_c] = 0
// and when no child is accepted the bonus token is the first v with
// sum_{i<=v} w_i > u_0 W.  Both rules leave every emitted token distributed as p: the first
// because "accept c with the probability that p has left for x_c" is a draw from p in
// disguise, the second because w + (accepted part of g) = p term by term.
//
// Subtractions of positive amounts compose, max(max(w - a, 0) - b, 0) = max(w - a - b, 0),
// so the residual after any number of rejections is max(w - g S, 0) with one scalar S, the
// sum of the W/G so far; it is recomputed from the logits when it is needed and never
// stored.  A rejected token's own weight is zero from then on (u < 1).
//
// Passes.  A visited row is streamed once for its maximum and a float sum of exponentials
// relative to a running one; what else it takes (a residual's sum, the draw) reads it from L2.
// Floats decide first: every sum carries a bound on its error (about 5e-6 of the row's sum), a
// test whose two sides differ by more than the bounds is decided, and so is a draw that lands
// that far inside a token.  Whatever is closer sends the node back to be done with the exact
// sums below: a few tests in 10^4, and as many draws as the distribution has mass near
// boundaries (with weights that fall off as rank^-2.2: 9 in 1000 of 163840 tokens, 24 in 1000
// after a rejection of 50257; all of them for a flat one).  An exact weight costs about eight
// times a float one, and a node with k drafted children refused pays k + 1 passes of them.
//   The bound, with e = 2^-24, a rounding.  The exponent y = (x - m) log2(e) / T carries four
// (the difference, log2(e) to a float, the quotient, the product), 3.3 e |y| in all, also where
// it is reached in steps, as a thread's, a warp's, a CTA's and the row's maximum take over one
// from another: the steps' |y| add up.  The weights' mean |y| is at most 13.4 (2^18 tokens, the
// worst being one at 1 and all others at 2^-14.8), which makes 3.3 e ln 2 13.4 = 1.83e-6 of the
// sum; the exponential adds 4 e, the exact sums' own units 2^18 2^-45 (twice in a residual):
// 2.1e-6 in all.  Each step to another maximum adds 5 e (an exponential and a product), each
// addition on the way from a value to the row's sum e.  What is then computed from the sums
// counts its roundings where it is done.
//
// Exactness.  The drawn token turns on a running sum over the vocabulary: an error of d in
// that sum moves a boundary past u_0 W with probability 2 d for each boundary, and there
// are as many boundaries as tokens.  Weights are therefore held as integers in units of
// 2^-44 of the row's largest (rounded from an exponential good to about 2^-37, built from
// pairs of floats: this part's double-precision units are slow).  Their sums are exact,
// whatever order they are taken in, so splits, tests and the final search agree with one
// another to the last unit.  A vocabulary of 2^18 tokens sums to below 2^63.
//
// Work.  Only the visited rows are read: accepted length + 1 of Q.  One cluster of CTAs
// per sequence shares a row; every CTA takes a contiguous slice, sums are exchanged through
// distributed shared memory, and every CTA takes the same decisions from the same numbers.
//
// Measured (calls in a loop, inputs beyond L2).  One sequence of 9 nodes, 32000 bf16 logits:
// 9-14 us, 7.9 in a graph; 32 x 33 nodes, 163840 floats: 33-41 us; with the drafter's rows, 8 x 9
// nodes, 163840 bf16: 27-43 us, and 64 x 17 nodes, 50257 floats: 48-65 us.  The bytes alone
// would take below 0.1, 6.2, 1.5 and 5.7 us: what bounds it is the walk, one visited row after
// another, the sequences with a draw or test that needs the exact sums (about 25000 clocks),
// and, from 456 CTAs on, a second round of them.  The dear ends, from a cold cache: 32 x 33
// nodes of 163840 equal floats, every draw done twice, 56 us; wide normal logits, most of them,
// 103; 16 drafted children refused one after another, 8 sequences of 163840 bf16, 314.
#include <cuda_bf16.h>

#include <algorithm>

#include "sample_math.h"
#include "sm100_ptx.h"
#include "tv_internal.h"

namespace tv {
namespace {

using namespace ptx;

constexpr int kMaxWarps = 32;
constexpr int kMaxCluster = 16;
constexpr float kEps = 6e-8f;   // a rounding, 2^-24
constexpr float kWeightError = 2.1e-6f;  // of a row's sum (see above)

struct SampleParams {
  const void* logits;
  int64_t V, stride;
  const float* temperature;
  const int32_t* parent;
  const int32_t* tokens;
  const float* uniforms;
  const float* draft;
  int64_t draft_stride;
  int32_t draft_rows, by_node;
  int B, Q;
  int32_t* accept_len;
  int32_t* path;
  int32_t* new_tokens;
  int32_t* status;
};

// What the walk does next, decided by warp 0 of every CTA alike.
enum : int { kAccept = 0, kExact = 1, kResidual = 2, kDraw = 3, kStop = 4 };

struct Shared {
  float2 exp2_table[kTable * kCopies];
  uint64_t keys[2][kMaxCluster];  // exchanged slice maxima, two phases
  float approx[2][kMaxCluster];   // and float sums, relative to the slice's maximum
  int64_t sums[2][kMaxCluster];   // exchanged slice sums
  uint64_t warp_key[kMaxWarps];   // of this CTA's slice, by warp
  float warp_approx[kMaxWarps];
  int64_t warp_sum[kMaxWarps];
  float parts[2][kMaxCluster];    // exchanged slice sums, in floats
  float warp_part[kMaxWarps];
  int32_t rejected[64];           // tokens refused at this node whose weights are in the sums
  int n_rejected, cmd, next;
  int redo;                       // 1 + the node whose draw has to be done again
  float m, s_hi, s_lo;            // the row's maximum; S as a pair of floats
  int64_t target;                 // the draw's place in the sums, and the vectors it is in
  float target_f, margin;
  int range0, range1;
};

// max(e - q S, 0) in the same units.
__device__ __forceinline__ int64_t residual(int64_t e, float q, float sh, float sl) {
  constexpr float magic = 12582912.f;
  const float p = q * sh;
  if (!(p > 0.f)) return e;
  if (p > 1.f) return 0;  // a weight is at most 1
  const float pe = fmaf(q, sh, -p) + q * sl;
  const float a = p * 4194304.f, ra = a + magic;
  const float rb = fmaf(a - (ra - magic), 4194304.f, pe * kUnit) + magic;
  const int64_t r = e - units({__float_as_int(ra) - __float_as_int(magic),
                               __float_as_int(rb) - __float_as_int(magic)});
  return r > 0 ? r : 0;
}

// What turns a row's logits into weights: the row's maximum, the scale 1/T (of log2) and,
// after rejections under draft probabilities, the drafter's row and S.
struct Scale {
  float m, ch, cl;
  const float* q;
  float s_hi, s_lo;
  const float2* table;
};

// The weights of vector j: exact, in units, or as floats relative to the largest.
template <typename T>
__device__ __forceinline__ void weights(const Row<T>& row, const Scale& c, int j, int64_t* e) {
  float v[Vec<T>::N];
  row.load(j, v);
#pragma unroll
  for (int i = 0; i < Vec<T>::N; ++i) {
    e[i] = units(weight(v[i], c.m, c.ch, c.cl, c.table));
    if (c.s_hi > 0.f && e[i] > 0)
      e[i] = residual(e[i], __ldg(c.q + row.first(j) + i), c.s_hi, c.s_lo);
  }
}
template <typename T>
__device__ __forceinline__ void weights(const Row<T>& row, const Scale& c, int j, float* e) {
  float v[Vec<T>::N];
  row.load(j, v);
  if (c.s_hi > 0.f) {
    float g[Vec<T>::N];
    const int64_t a = row.first(j);
    if (row.whole(j) && ((uintptr_t)(c.q + a) & 15u) == 0) {
#pragma unroll
      for (int i = 0; i < Vec<T>::N; i += 4) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(c.q + a + i));
        g[i] = f.x;
        g[i + 1] = f.y;
        g[i + 2] = f.z;
        g[i + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < Vec<T>::N; ++i)
        g[i] = a + i >= 0 && a + i < row.V ? __ldg(c.q + a + i) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i)
      e[i] = fmaxf(fmaf(-g[i], c.s_hi, ex2((v[i] - c.m) * c.ch)), 0.f);
  } else {
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) e[i] = ex2((v[i] - c.m) * c.ch);
  }
}

// Sum of the weights of vectors [j0, j1), by one warp.
template <typename S, typename T>
__device__ __forceinline__ S sum_range(const Row<T>& row, const Scale& c, int j0, int j1) {
  S s = 0;
#pragma unroll 2
  for (int j = j0 + (int)(threadIdx.x & 31); j < j1; j += 32) {
    S e[Vec<T>::N], part = 0;
    weights(row, c, j, e);
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) part += e[i];
    s += part;
  }
  return warp_sum(s);
}

template <typename U>
__device__ __forceinline__ U pick(const U* two, int i) {  // slot i / 32 of lane i % 32
  return __shfl_sync(0xffffffffu, (i >> 5) ? two[1] : two[0], i & 31);
}
__device__ __forceinline__ int64_t& target_of(Shared& sh, int64_t) { return sh.target; }
__device__ __forceinline__ float& target_of(Shared& sh, float) { return sh.target_f; }
__device__ __forceinline__ int64_t* warp_sums(Shared& sh, int64_t) { return sh.warp_sum; }
__device__ __forceinline__ float* warp_sums(Shared& sh, float) { return sh.warp_part; }

// The owner's part of a draw, by the whole CTA: the token at place target_of(sh) of vectors
// range0 .. range1-1, a vector per thread at a time.  Returns it in the thread that has it
// (others -1), or -2 there where a float draw lands within `margin` of a token's edge.
template <typename S, int kWarps, typename T>
__device__ __forceinline__ int draw(Shared& sh, const Row<T>& row, const Scale& sc) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n_out = sh.n_rejected;
  const int y0 = sh.range0, y1 = sh.range1;
  S t = target_of(sh, (S)0);
  // the weights of one vector, without the tokens refused
  auto load = [&](int j, S* e) {
    S s = 0;
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) e[i] = 0;
    if (j < y1) weights(row, sc, j, e);
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) {
      for (int r = 0; r < n_out; ++r)
        if (row.first(j) + i == sh.rejected[r]) e[i] = 0;
      s += e[i];
    }
    return s;
  };
  S* sums = warp_sums(sh, (S)0);
  for (int base = y0; base < y1; base += 32 * kWarps) {  // a vector per thread
    const int j = base + 32 * warp + lane;
    S e[Vec<T>::N];
    const S s = load(j, e);
    const S part = warp_sum(s);
    __syncthreads();
    if (lane == 0) sums[warp] = part;
    __syncthreads();
    const S mine = lane < kWarps ? sums[lane] : (S)0;
    const S all = warp_sum(mine);
    if (t >= all && base + 32 * kWarps < y1) {
      t -= all;
      continue;
    }
    if (warp != locate(mine, kWarps, &t)) return -1;
    if (lane != locate(s, 32, &t)) return -1;
    int k = 0;
    S width = 0;
    bool found = false;
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) {
      if (!found && t < e[i]) {
        found = true;
        width = e[i];
        k = i;
      }
      if (!found) t -= e[i];
    }
    const float edge = fminf((float)t, (float)(width - t));
    if (sizeof(S) == 4 && !(found && edge > sh.margin)) return -2;
    return (int)row.first(j) + k;
  }
  return sizeof(S) == 4 && threadIdx.x == 0 ? -2 : -1;
}

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 3 : 1)
    tree_sample_kernel(SampleParams p, int log2_C) {
  constexpr int kWarps = kThreads / 32;
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = 1 << log2_C, b = blockIdx.x >> log2_C, Q = p.Q;
  const int rank = C > 1 ? (int)cluster_rank() : 0;
  int32_t* path = p.path + (int64_t)b * Q;
  int32_t* emit = p.new_tokens + (int64_t)b * Q;
  // (launched as a programmatic dependent of the kernel before it; the next one may start once
  // that has ended, so that it overlaps this kernel alone)
  griddep_wait();
  griddep_launch_dependents();
  // warp 0 holds the tree: node lane and node lane + 32
  int par[2] = {-2, -2}, tok[2] = {-1, -1};
  float uni[2] = {0.f, 0.f};
  bool ok_tree = true;
  if (warp == 0) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int i = lane + 32 * s;
      if (i >= Q) continue;
      par[s] = p.parent[(int64_t)b * Q + i];
      tok[s] = p.tokens[(int64_t)b * Q + i];
      // outside [0, 1): the nearest number inside (NaN: 0)
      uni[s] = fminf(fmaxf(p.uniforms[(int64_t)b * Q + i], 0.f), 0x1.fffffep-1f);
      ok_tree = ok_tree && (i == 0 ? par[s] == -1 : par[s] >= 0 && par[s] < i);
      if (rank == 0) {
        path[i] = i == 0 ? 0 : -1;
        emit[i] = -1;
      }
    }
  }
  const float T0 = p.temperature ? p.temperature[b] : 1.f;
  for (int i = tid; i < kTable * kCopies; i += kThreads)
    sh.exp2_table[i] = make_float2(d_exp.hi[i / kCopies], d_exp.lo[i / kCopies]);
  if (tid == 0) sh.redo = 0;  // (before the first cluster barrier: other CTAs set it)
  const bool ok_temp = T0 >= 0.f;  // a NaN is not
  if (__syncthreads_or(!ok_tree) || !ok_temp) {  // the whole cluster alike
    if (rank == 0 && tid == 0) {
      p.accept_len[b] = 0;
      report(p.status, ok_temp ? TV_ERR_INVALID_TREE : TV_ERR_INVALID_ARG);
    }
    return;
  }
  // (a CTA's shared memory may be written once it is known to have started)
  if (C > 1) cluster_arrive();
  const bool greedy = T0 == 0.f;
  // 1/T in units of log2 as a pair of floats; the clamp keeps 0 * inf out of the weights
  constexpr float l2e = (float)(1.0 / kLn2), l2e_low = (float)(1.0 / kLn2 - (double)l2e);
  const float cq = l2e / T0;
  const float ch = fminf(fmaxf(cq, 1e-30f), 1e30f);
  const float cl =
      ch == cq ? (fmaf(-cq, T0, l2e) + l2e_low) / T0 : 0.f;

  int node = 0, count = 0, phase = 0;
  for (;;) {
    const Row<T> row((const T*)p.logits + ((int64_t)b * Q + node) * p.stride, p.V);
    const int per = (row.n_vec + C - 1) >> log2_C;
    const int c0 = min(row.n_vec, rank * per), c1 = min(row.n_vec, c0 + per);
    const int per_w = (per + kWarps - 1) / kWarps;
    const int w0 = min(c1, c0 + warp * per_w), w1 = min(c1, w0 + per_w);
    const float* q = nullptr;
    bool has_q = false;
    if (p.draft) {
      const int r = p.by_node ? node : count;
      has_q = r < p.draft_rows;
      q = p.draft + ((int64_t)b * p.draft_rows + min(r, p.draft_rows - 1)) * p.draft_stride;
    }
    // ---- the row's maximum, and the float sum or (greedy) the maximum's first index ----
    // (a NaN ends up in the sum)
    constexpr int N = Vec<T>::N, kUnroll = Vec<T>::kUnroll;
    float best = -INFINITY, sum = 0.f;
    int best_at = 0;
    // the row's ends, where they are no whole vector: one value a lane
    auto end_value = [&](int j) {
      if (j < w0 || j >= w1) return;
      const int64_t a = row.first(j) + lane;
      const float v = lane < N && a >= 0 && a < p.V ? Vec<T>::one(row.x + a) : -INFINITY;
      if (v != v) sum = v;
      if (v > best) {
        sum = (greedy ? sum : sum * ex2((best - v) * ch)) + 1.f;
        best = v;
        best_at = (int)a;
      } else if (best > -INFINITY) {
        sum += ex2((v - best) * ch);
      }
    };
    const int e0 = row.first_whole(), e1 = row.end_whole();
    if (e0 > 0) end_value(0);
    const int v0 = max(w0, e0), v1 = min(w1, e1);
    for (int j0 = v0; j0 < v1; j0 += 32 * kUnroll) {
      const int j = j0 + lane;
      uint4 w[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        w[k] = make_uint4(Vec<T>::kMasked, Vec<T>::kMasked, Vec<T>::kMasked, Vec<T>::kMasked);
        if (j + 32 * k < v1) w[k] = row.raw(j + 32 * k);
      }
      float m = best;
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        if (j0 + 32 * k >= v1) break;  // no lane of the warp has one
        float v[N];
        Vec<T>::unpack(w[k], v);
        if (!greedy) {
#pragma unroll
          for (int i = 0; i < N; i += 2) m = fmax3(m, v[i], v[i + 1]);
          continue;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (v[i] != v[i]) sum = v[i];
          if (v[i] > best) {
            best = v[i];
            best_at = (int)row.first(j + 32 * k) + i;
          }
        }
      }
      if (greedy) continue;
      if (m > best) {
        sum *= ex2((best - m) * ch);  // (from -inf: 0)
        best = m;
      }
      const float at = best > -INFINITY ? best : 0.f;
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        if (j0 + 32 * k >= v1) break;
        float v[N], part = 0.f;
        Vec<T>::unpack(w[k], v);
#pragma unroll
        for (int i = 0; i < N; ++i) part += ex2((v[i] - at) * ch);
        sum += part;
      }
    }
    if (e1 < row.n_vec && e1 >= e0) end_value(e1);
    // warp 0: the children and their logits, which the row has brought to L2
    uint64_t children = 0;
    float child[2] = {-INFINITY, -INFINITY}, child_q[2] = {0.f, 0.f};
    if (warp == 0) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const bool is = par[s] == node && tok[s] >= 0 && tok[s] < p.V;
        children |= (uint64_t)__ballot_sync(0xffffffffu, is) << (32 * s);
        if (is) {
          child[s] = Vec<T>::one(row.x + tok[s]);
          if (has_q) child_q[s] = __ldg(q + tok[s]);
        }
      }
    }
    // order-preserving value bits, then the complemented index: the largest key is the
    // largest value's first place; a NaN anywhere beats every value
    uint64_t key = best > -INFINITY ? ((uint64_t)ordered(best) << 32) |
                                          (uint32_t)(0xFFFFFFFFu - (uint32_t)best_at)
                                    : 0ull;
    const bool is_nan = sum != sum && best < INFINITY;
    key = warp_max(key);
    sum = key ? sum * ex2((best - unordered((uint32_t)(key >> 32))) * ch) : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (__any_sync(0xffffffffu, is_nan)) key = ~0ull;
    if (lane == 0) {
      sh.warp_key[warp] = key;
      sh.warp_approx[warp] = sum;
    }
    if (C > 1 && count == 0) cluster_wait();
    __syncthreads();
    if (warp == 0) {
      const uint64_t mine = lane < kWarps ? sh.warp_key[lane] : 0ull;
      key = warp_max(mine);
      float t = mine ? sh.warp_approx[lane] * ex2((unordered((uint32_t)(mine >> 32)) -
                                                   unordered((uint32_t)(key >> 32))) * ch)
                     : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      if (C == 1) {
        if (lane == 0) {
          sh.keys[phase][0] = key;
          sh.approx[phase][0] = t;
        }
      } else if (lane < C) {
        st_cluster_u64(&sh.keys[phase][rank], (uint32_t)lane, key);
        st_cluster_f32(&sh.approx[phase][rank], (uint32_t)lane, t);
      }
    }
    if (C > 1) cluster_sync();
    else __syncthreads();
    const uint64_t slice_key = lane < C ? sh.keys[phase][lane] : 0ull;
    key = warp_max(slice_key);
    const float m = unordered((uint32_t)(key >> 32));
    Scale sc{m, ch, cl, q, 0.f, 0.f, sh.exp2_table};
    int64_t child_e[2] = {0, 0};
    if (key == 0 || key == ~0ull || m == INFINITY || greedy) {
      if (warp == 0) {
        const int top = (int)(0xFFFFFFFFu - (uint32_t)key);
        const bool none = key == 0 || key == ~0ull || m == INFINITY;  // nothing to draw from
        const uint32_t h0 =
            __ballot_sync(0xffffffffu, ((uint32_t)children >> lane & 1) && tok[0] == top);
        const uint32_t h1 =
            __ballot_sync(0xffffffffu, ((uint32_t)(children >> 32) >> lane & 1) && tok[1] == top);
        const int next = none ? -1 : h0 ? __ffs(h0) - 1 : h1 ? 31 + __ffs(h1) : -1;
        if (lane == 0) {
          if (rank == 0 && none) report(p.status, TV_ERR_INVALID_ARG);
          else if (rank == 0 && next < 0) emit[count] = top;
          sh.next = next;
          sh.cmd = next < 0 ? kStop : kAccept;
        }
      }
      __syncthreads();
      phase ^= 1;
    } else {
      // ---- by floats, with bounds on their errors ----
      float part = slice_key ? sh.approx[phase][lane] *
                                   ex2((unordered((uint32_t)(slice_key >> 32)) - m) * ch)
                             : 0.f;  // lane r: slice r's sum
      phase ^= 1;
      const float Z = warp_sum(part);
      // additions from a value to the row's sum (in a vector, a thread, a warp, a CTA, a
      // cluster), and changes of maximum, of which a thread's first costs nothing
      const int ends = (e0 > 0) + (e1 < row.n_vec);
      const int moves = (per_w + 32 * kUnroll - 1) / (32 * kUnroll) + ends + 2;
      const float adds = kEps * (float)(N + (per_w + 31) / 32 + ends + 15 + 5 * moves);
      float W = Z, dW = (kWeightError + adds) * Z, S = 0.f, dS = 0.f, G = 1.f, dG = 0.f;
      uint64_t left = p.draft && !has_q ? 0ull : children, refused = 0;
      float ew[2] = {0.f, 0.f};
      if (warp == 0) {
        if (p.draft && !has_q && children && rank == 0 && lane == 0)
          report(p.status, TV_ERR_BOUNDS);  // no drafter's row for this depth: no test
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          child_e[s] = units(weight(child[s], m, ch, cl, sh.exp2_table));
          ew[s] = (float)child_e[s] * (1.f / kUnit);
        }
      }
      for (;;) {
        if (warp == 0) {
          int cmd = kDraw, next = -1, n = 0;
          if (!(W > 16.f * dW)) cmd = kExact;
          while (cmd == kDraw && left) {
            const int i = __ffsll((long long)left) - 1;
            left &= left - 1;
            const int x = pick(tok, i);
            const uint64_t same =
                (uint64_t)__ballot_sync(0xffffffffu, tok[0] == x) |
                (uint64_t)__ballot_sync(0xffffffffu, tok[1] == x) << 32;
            const bool again = same & refused;  // a token refused before has no weight left
            const float u = pick(uni, i), e = pick(ew, i);
            const float g = !p.draft ? 1.f : again ? 0.f : pick(child_q, i);
            const float w = again ? 0.f : p.draft ? fmaxf(fmaf(-g, S, e), 0.f) : e;
            const float over = u * g * W - w * G;
            // (6e-14: the exact residual's units)
            const float error = u * g * (dW + 3.f * kEps * W) + w * (dG + 2.f * kEps * G) +
                                G * (1e-6f * e + g * (dS + 1e-6f * S) + 6e-14f);
            if (over < -error) {
              cmd = kAccept;
              next = i;
              break;
            }
            if (over < error && !again && e > 0.f) {
              cmd = kExact;
              break;
            }
            if (!p.draft) {
              refused |= 1ull << i;
              dW += 2.f * kEps * W;
              W -= w;
              if (!again) {
                if (row.in_part(x, per, lane)) part -= w;
                if (lane == 0) sh.rejected[n] = x;
                ++n;
              }
              continue;
            }
            refused |= 1ull << i;
            S += W / G;
            dS += (dW + W * (1.01f * dG / G + 2.f * kEps)) / G + 2.f * kEps * S;
            G -= g;
            dG += kEps * G;
            cmd = G > 1e-3f ? kResidual : kExact;
          }
          if (cmd == kDraw) {
            // which slice, and where in it; then (of use to that slice's CTA) which warp
            if (!(W > 16.f * dW)) cmd = kExact;
            float t = uni[0] * W;
            t = __shfl_sync(0xffffffffu, t, 0);
            const int owner = locate(part, C, &t);
            float mine = 0.f;
            if (lane < kWarps) {
              mine = sh.warp_part[lane];
              if (S == 0.f) {
                const uint64_t k = sh.warp_key[lane];
                mine = k ? sh.warp_approx[lane] * ex2((unordered((uint32_t)(k >> 32)) - m) * ch)
                         : 0.f;
              }
            }
            __syncwarp();
            for (int r = 0; r < n; ++r) {
              const int x = sh.rejected[r];
              const uint64_t same =
                  (uint64_t)__ballot_sync(0xffffffffu, tok[0] == x) |
                  (uint64_t)__ballot_sync(0xffffffffu, tok[1] == x) << 32;
              const float w = pick(ew, __ffsll((long long)(same & refused)) - 1);
              if (row.in_part(x, per, rank) && row.in_part(x, per_w, lane, c0)) mine -= w;
            }
            const int w = locate(mine, kWarps, &t);
            next = owner;
            if (lane == 0) {
              sh.target_f = t;
              // the target's error, the sums' (every weight is in those of one pass), and the
              // roundings of the target on its way: a product, subtractions and scans
              const int steps = (per_w + 32 * kWarps - 1) / (32 * kWarps);
              sh.margin = 2.f * dW + kEps * (float)(32 + N + 2 * n + steps) * W;
              sh.range0 = min(c1, c0 + w * per_w);
              sh.range1 = min(c1, sh.range0 + per_w);
            }
          }
          if (lane == 0) {
            sh.s_hi = S;
            sh.n_rejected = n;
            sh.cmd = cmd;
            sh.next = next;
          }
        }
        __syncthreads();
        if (sh.cmd != kResidual) break;
        sc.s_hi = sh.s_hi;
        const float ws = sum_range<float>(row, sc, w0, w1);
        if (lane == 0) sh.warp_part[warp] = ws;
        __syncthreads();
        if (warp == 0) {
          const float t = warp_sum(lane < kWarps ? sh.warp_part[lane] : 0.f);
          if (C == 1) {
            if (lane == 0) sh.parts[phase][0] = t;
          } else if (lane < C) {
            st_cluster_f32(&sh.parts[phase][rank], (uint32_t)lane, t);
          }
        }
        if (C > 1) cluster_sync();
        else __syncthreads();
        if (warp == 0) {
          part = lane < C ? sh.parts[phase][lane] : 0.f;
          W = warp_sum(part);
          dW = kWeightError * Z + (adds + kEps) * W + 1.01f * dS;  // (the g sum to 1)
        }
        phase ^= 1;
      }
      if (sh.cmd == kDraw) {
        if (sh.next == rank) {
          const int token = draw<float, kWarps>(sh, row, sc);
          if (token >= 0) emit[count] = token;
          if (token == -2)  // tell every CTA of the cluster
            for (int r = 0; r < C; ++r) {
              if (C > 1) st_cluster_u32(&sh.redo, (uint32_t)r, (uint32_t)node + 1);
              else sh.redo = node + 1;
            }
        }
        if (C > 1) cluster_sync();
        else __syncthreads();
        if (tid == 0) sh.cmd = sh.redo == node + 1 ? kExact : kStop;
        __syncthreads();
      }
    }
    if (sh.cmd == kExact) {
      // ---- exact sums of the weights, the tests by them, and residuals after rejections ----
      sc.s_hi = 0.f;
      // warp 0's: S and G, the children left, the tokens refused, the child whose rejection
      // the residual that is being summed belongs to, and S before that
      double S = 0.0, G = 1.0, S_before = 0.0;
      uint64_t left = p.draft && !has_q ? 0ull : children, refused = 0;
      int refusing = -1;
      for (;;) {
        const int64_t ws = sum_range<int64_t>(row, sc, w0, w1);
        if (lane == 0) sh.warp_sum[warp] = ws;
        __syncthreads();
        if (warp == 0) {
          const int64_t t = warp_sum(lane < kWarps ? sh.warp_sum[lane] : 0);
          if (C == 1) {
            if (lane == 0) sh.sums[phase][0] = t;
          } else if (lane < C) {
            st_cluster_u64(&sh.sums[phase][rank], (uint32_t)lane, (uint64_t)t);
          }
        }
        if (C > 1) cluster_sync();
        else __syncthreads();
        if (warp == 0) {
          int64_t part = lane < C ? sh.sums[phase][lane] : 0;
          int64_t W = warp_sum(part);
          int cmd = kDraw, next = -1, n = 0;
          if (refusing >= 0 && W == 0) {
            if (pick(child_e, refusing) > 0) {
              // the drafter covers all that p has left: the two are equal but for rounding
              cmd = kAccept;
              next = refusing;
            } else {  // a token that p excludes: the draw is from what was left before it
              cmd = kResidual;
              S = S_before;
              left = 0;
              refusing = -1;
            }
          }
          while (cmd == kDraw && left && (!p.draft || G > 0.0)) {
            const int i = __ffsll((long long)left) - 1;
            left &= left - 1;
            const int x = pick(tok, i);
            const uint64_t same =
                (uint64_t)__ballot_sync(0xffffffffu, tok[0] == x) |
                (uint64_t)__ballot_sync(0xffffffffu, tok[1] == x) << 32;
            const bool again = same & refused;  // a token refused before has no weight left
            const float qx = pick(child_q, i);
            const double u = pick(uni, i), g = !p.draft ? 1.0 : again ? 0.0 : (double)qx;
            int64_t w = pick(child_e, i);
            if (again) w = 0;
            else if (p.draft) w = residual(w, qx, sc.s_hi, sc.s_lo);
            if (u * g * (double)W < (double)w * G) {
              cmd = kAccept;
              next = i;
              break;
            }
            refused |= 1ull << i;
            if (!p.draft) {
              W -= w;
              if (!again) {
                if (row.in_part(x, per, lane)) part -= w;
                if (lane == 0) sh.rejected[n] = x;
                ++n;
              }
              continue;
            }
            cmd = kResidual;
            refusing = i;
            S_before = S;
            S += (double)W * (1.0 / (double)kUnit) / G;
            G -= g;
          }
          if (cmd == kDraw) {
            int64_t t = min((int64_t)((double)uni[0] * (double)W), W - 1);
            t = __shfl_sync(0xffffffffu, t, 0);
            next = locate(part, C, &t);
            int64_t mine = lane < kWarps ? sh.warp_sum[lane] : 0;
            __syncwarp();
            for (int r = 0; r < n; ++r) {
              const int x = sh.rejected[r];
              const uint64_t same =
                  (uint64_t)__ballot_sync(0xffffffffu, tok[0] == x) |
                  (uint64_t)__ballot_sync(0xffffffffu, tok[1] == x) << 32;
              const int64_t w = pick(child_e, __ffsll((long long)(same & refused)) - 1);
              if (row.in_part(x, per, rank) && row.in_part(x, per_w, lane, c0)) mine -= w;
            }
            const int w = locate(mine, kWarps, &t);
            if (lane == 0) {
              sh.target = t;
              sh.range0 = min(c1, c0 + w * per_w);
              sh.range1 = min(c1, sh.range0 + per_w);
            }
          }
          if (lane == 0) {
            sh.s_hi = (float)S;
            sh.s_lo = (float)(S - (double)(float)S);
            sh.n_rejected = n;
            sh.cmd = cmd;
            sh.next = next;
          }
        }
        __syncthreads();
        if (sh.cmd != kResidual) break;
        sc.s_hi = sh.s_hi;
        sc.s_lo = sh.s_lo;
        phase ^= 1;
      }
      if (sh.cmd == kDraw) {
        if (sh.next == rank) {
          const int token = draw<int64_t, kWarps>(sh, row, sc);
          if (token >= 0) emit[count] = token;
        }
        break;
      }
      phase ^= 1;
    }
    if (sh.cmd == kStop) break;
    node = sh.next;
    ++count;
    if (warp == 0 && rank == 0) {
      const int x = pick(tok, node);
      if (lane == 0) {
        emit[count - 1] = x;
        path[count] = node;
      }
    }
  }
  if (rank == 0 && tid == 0) p.accept_len[b] = count;
  if (C > 1) cluster_sync();  // no CTA leaves while another may still write to it
}

template <typename T, int kThreads>
cudaError_t launch(const SampleParams& p, int C, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.B * C));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  if (C > 8) {
    cudaError_t e = cudaFuncSetAttribute(tree_sample_kernel<T, kThreads>,
                                         cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  int log2_C = 0;
  while ((1 << log2_C) < C) ++log2_C;
  return cudaLaunchKernelEx(&cfg, tree_sample_kernel<T, kThreads>, p, log2_C);
}

// Threads per CTA: 1024 or 512 where the CTAs are few and a thread still has eight values to
// read.  An SM's registers hold one CTA of 1024 threads, one of 512 (119-124 registers each) or
// three of 256 (80): between one and two CTAs of 512 per SM, the last ones start when the first
// have ended, and so do those of 256 past three.
template <typename T>
cudaError_t launch(const SampleParams& p, int C, int sm_count, cudaStream_t st) {
  const int64_t ctas = (int64_t)p.B * C, slice = p.V / C;
  if (ctas <= sm_count && slice >= 8192) return launch<T, 1024>(p, C, st);
  if (ctas <= 2ll * sm_count && slice >= 4096) return launch<T, 512>(p, C, st);
  return launch<T, 256>(p, C, st);
}

}  // namespace

// CTAs per sequence: at most 16, about 2048 vocabulary entries each at least, and no more than
// four per SM in all, of which three are resident.  (32 x 33 nodes of 163840 floats, and 64 x 17
// of 50257 with the drafter's rows, 512 CTAs: 36-40 and 52-54 us.  A limit of three or of two
// both comes to 256 CTAs of 512 threads: 39-47 and 57-85 over seeds.)
int sample_cluster(int B, int64_t V, int sm_count) {
  int C = kMaxCluster;
  while (C > 1 && ((int64_t)B * C > 4 * (int64_t)sm_count || V < 2048ll * C)) C /= 2;
  return C;
}

cudaError_t launch_tree_sample(const tv_sample_args* a, int sm_count, cudaStream_t st) {
  if (a->B == 0) return cudaSuccess;
  SampleParams p{};
  p.logits = a->logits;
  p.V = a->vocab;
  p.stride = a->logits_row_stride;
  p.temperature = a->temperature;
  p.parent = a->parent;
  p.tokens = a->tokens;
  p.uniforms = a->uniforms;
  p.draft = a->draft_probs;
  p.draft_stride = a->draft_row_stride;
  p.draft_rows = a->draft_rows;
  p.by_node = a->draft_mode == TV_DRAFT_BY_NODE;
  p.B = a->B;
  p.Q = a->Q;
  p.accept_len = a->accept_len;
  p.path = a->path;
  p.new_tokens = a->new_tokens;
  p.status = a->status;
  const int C = sample_cluster(a->B, a->vocab, sm_count);
  return a->logits_dt == TV_BF16 ? launch<__nv_bfloat16>(p, C, sm_count, st)
                                 : launch<float>(p, C, sm_count, st);
}

}  // namespace tv
