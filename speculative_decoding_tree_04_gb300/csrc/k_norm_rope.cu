// k_norm_rope.cu -- rotary positions in every layout (tv_rope), and the norms of queries and
// keys with the rotation in the same pass, keys written into the cache (tv_norm_rope).
//
// A vector x of n elements (a head of one token) becomes, with r = 1 / sqrt(mean x^2 + eps)
// where it has a norm,
//   y_e = x_e r w_e,   and in its rotated part, for pair k = (a, b) at angle t = pos * f_k,
//   out_a = y_a cos t - y_b sin t,   out_b = y_b cos t + y_a sin t
// (cos and sin times the scaling's magnitude).  A pair is (k, k + rot/2) in the half layout,
// (2k, 2k+1) in the interleaved one.  The norm's sum, the product and the rotation are taken in
// 32 bits and rounded once.
//
// What bounds it: bytes for prompts, latency for single tokens.  A warp holds one vector (up to
// four short ones) in registers, 16 bytes a lane, so that the norm costs a shuffle reduction
// and no second read; in the half layout a lane loads its partners too, from lines that the
// warp's own loads have brought.  A block serves one token, or a part of its heads where the
// tokens are few (about two blocks per SM), and takes the angles' cosines and sines once, while
// the first vectors are on their way.
//
// Angles.  The product pos * f_k and its reduction by multiples of pi/2 (Cody and Waite's
// two-part subtraction) run in double; float32 tensors take cos and sin in double, too, as
// tv_rope_neox does, with its error-free rotation (rope_math.h).  For bf16 the remainder
// |r| <= pi/4 goes on as a float, through the Taylor series up to r^9 and r^10 (truncation
// below 2^-28): cos and sin within 2^-23, which moves a bf16 result by 2^-13 of its rounding
// step, at about nine double operations a pair instead of about a hundred.  This part's
// double-precision units do two a clock and SM: with full double trigonometry they, not the
// memory, would bound a prompt of few heads.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "rope_math.h"
#include "sm100_ptx.h"
#include "tv_internal.h"

namespace tv {
namespace {

using namespace rope;

constexpr int kMaxThreads = 256;
constexpr int kMaxVecs = 4;  // 16-byte vectors of one head that a lane holds

// cos and sin of one pair's angle as the rotation takes them.
template <typename T>
struct Turn;
template <>
struct Turn<float> {
  CosSin t;
  __device__ static Turn make(double angle, double mag) {
    double s, c;
    sincos(angle, &s, &c);
    Turn r;
    r.t.c = __dmul_rn(c, mag);
    r.t.s = __dmul_rn(s, mag);
    r.t.ch = __double2float_rn(r.t.c);
    r.t.cl = __double2float_rn(__dsub_rn(r.t.c, (double)r.t.ch));
    r.t.sh = __double2float_rn(r.t.s);
    r.t.sl = __double2float_rn(__dsub_rn(r.t.s, (double)r.t.sh));
    return r;
  }
  // a cos - b sin
  __device__ float out(float a, float b) const { return RotOut<float>::f(a, b, t.ch, t.cl, t.sh, t.sl, &t.c); }
};
template <>
struct Turn<__nv_bfloat16> {
  float c, s;
  __device__ static Turn make(double angle, double mag) {
    constexpr double kMagic = 6755399441055744.0;  // 1.5 * 2^52: adding it rounds to an integer
    constexpr double kTwoOverPi = 0.63661977236758134308;
    constexpr double kHalfPiHigh = 1.5707963267948965580, kHalfPiLow = 6.1232339957367658e-17;
    const double q0 = __fma_rn(angle, kTwoOverPi, kMagic);
    const double q = q0 - kMagic;
    const int quarter = (int)__double2loint(q0);
    const float r = (float)__fma_rn(-q, kHalfPiLow, __fma_rn(-q, kHalfPiHigh, angle));
    const float z = r * r;
    const float ps = fmaf(z, fmaf(z, fmaf(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f);
    const float sn = fmaf(r * z, ps, r);
    const float pc = fmaf(
        z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f), -0.5f);
    const float cs = fmaf(z, pc, 1.f);
    const float m = (float)mag;
    const float c0 = (quarter & 1) ? sn : cs, s0 = (quarter & 1) ? cs : sn;
    Turn t;
    t.c = ((quarter + 1) & 2) ? -c0 * m : c0 * m;
    t.s = (quarter & 2) ? -s0 * m : s0 * m;
    return t;
  }
  __device__ float out(float a, float b) const { return fmaf(a, c, -(b * s)); }
};

template <typename T>
struct Vec16;
template <>
struct Vec16<float> {
  static constexpr int N = 4;
  __device__ static void unpack(const uint4& u, float* x) {
    x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
  }
  __device__ static uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};
template <>
struct Vec16<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static void unpack(const uint4& u, float* x) {
    const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(v[i] << 16);
      x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  }
  __device__ static uint4 pack(const float* x) {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      v[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
  }
};

// A kind of vector: n elements, of which [at, at + rot) are rotated; elements below `split` go
// to the first output, the others to the second.
struct Kind {
  int n, at, rot, split;
  float eps;  // with a weight: the norm's
};

// A vector's addresses.
template <typename T>
struct Place {
  const T* src;
  T* low;        // element e < split at low + e
  T* high;       // element e >= split at high + e - split
  const T* w;    // norm weights, or null for no norm
};

// Where pair k's turn lies: the turns that a lane reads in step i (of one vector's eight or
// four elements) are consecutive over the lanes, so that no two of them meet in a bank.
template <typename T>
__device__ __forceinline__ int turn_slot(int k, int half, bool pairs) {
  constexpr int N = Vec16<T>::N;
  const int per = pairs ? N / 2 : N;  // pairs of one vector
  return half % per ? k : (k % per) * (half / per) + k / per;
}

// One vector in 16-byte pieces by the `width` lanes of a group (lane `l` of it).  Loads first,
// then, by `finish`, the norm, the rotation and the stores.
template <typename T, int NV>
struct Held {
  uint4 own[NV], other[NV];
  __device__ __forceinline__ void load(const T* src, const Kind& k, bool pairs, bool on, int l, int width) {
    constexpr int N = Vec16<T>::N;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = l + i * width, e = v * N;
      if (!on || e >= k.n) continue;
      own[i] = *reinterpret_cast<const uint4*>(src + e);
      if (!pairs && e >= k.at && e < k.at + k.rot) {
        const int half = k.rot / 2;
        other[i] = *reinterpret_cast<const uint4*>(src + (e < k.at + half ? e + half : e - half));
      }
    }
  }
  __device__ __forceinline__ void finish(const Place<T>& p, const Kind& k, bool pairs, bool on, int l,
                                         int width, const Turn<T>* turns) {
    constexpr int N = Vec16<T>::N;
    const int half = k.rot / 2;
    float r = 1.f;
    if (p.w) {  // the same for the whole warp
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!on || (l + i * width) * N >= k.n) continue;
        float x[N];
        Vec16<T>::unpack(own[i], x);
#pragma unroll
        for (int j = 0; j < N; ++j) sum = fmaf(x[j], x[j], sum);
      }
      for (int o = width / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      r = 1.f / sqrtf(sum / (float)k.n + k.eps);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (l + i * width) * N;
      if (!on || e >= k.n) continue;
      float x[N];
      Vec16<T>::unpack(own[i], x);
      if (p.w) {
        float w[N];
        Vec16<T>::unpack(__ldg(reinterpret_cast<const uint4*>(p.w + e)), w);
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = x[j] * r * w[j];
      }
      if (e >= k.at && e < k.at + k.rot) {
        const int q = e - k.at;
        if (pairs) {
          const int per = N / 2, step = half / per;
#pragma unroll
          for (int j = 0; j < N / 2; ++j) {
            const Turn<T> t = turns[j * step + q / N];
            const float a = x[2 * j], b = x[2 * j + 1];
            x[2 * j] = t.out(a, b);
            x[2 * j + 1] = t.out(b, -a);
          }
        } else {
          const bool first = q < half;
          const int step = half / N, k0 = (first ? q : q - half) / N;
          float y[N];
          Vec16<T>::unpack(other[i], y);
          if (p.w) {
            float w[N];
            Vec16<T>::unpack(
                __ldg(reinterpret_cast<const uint4*>(p.w + (first ? e + half : e - half))), w);
#pragma unroll
            for (int j = 0; j < N; ++j) y[j] = y[j] * r * w[j];
          }
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const Turn<T> t = turns[j * step + k0];
            x[j] = first ? t.out(x[j], y[j]) : t.out(x[j], -y[j]);
          }
        }
      }
      T* dst = e < k.split ? p.low + e : p.high + (e - k.split);
      *reinterpret_cast<uint4*>(dst) = Vec16<T>::pack(x);
    }
  }
};

// The same for one vector of any size and alignment, an element (or a pair) at a time; a lane
// reads both elements of a pair before it writes either, so the vector may be turned in place.
template <typename T>
__device__ void one_by_one(const Place<T>& p, const Kind& k, bool pairs, const Turn<T>* turns, int lane) {
  float r = 1.f;
  if (p.w) {
    float sum = 0.f;
    for (int e = lane; e < k.n; e += 32) {
      const float x = to_float(p.src[e]);
      sum = fmaf(x, x, sum);
    }
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    r = 1.f / sqrtf(sum / (float)k.n + k.eps);
  }
  auto get = [&](int e) {
    const float x = to_float(p.src[e]);
    return p.w ? x * r * to_float(p.w[e]) : x;
  };
  auto put = [&](int e, float y) { store_float(e < k.split ? p.low + e : p.high + (e - k.split), y); };
  for (int e = lane; e < k.n; e += 32)
    if (e < k.at || e >= k.at + k.rot) put(e, get(e));
  const int half = k.rot / 2;
  for (int i = lane; i < half; i += 32) {
    const int ea = k.at + (pairs ? 2 * i : i), eb = pairs ? ea + 1 : ea + half;
    const float a = get(ea), b = get(eb);
    const Turn<T> t = turns[turn_slot<T>(i, half, pairs)];
    put(ea, t.out(a, b));
    put(eb, t.out(b, -a));
  }
}

// The heads a block turns for its token: heads h0 .. h0+nh-1 of `kind`, from src + h*stride,
// to low + h*low_stride and high + h*high_stride.
template <typename T>
struct Heads {
  const T* src;
  T* low;
  T* high;
  const T* w;
  int64_t stride, low_stride, high_stride;
  __device__ Place<T> place(int h) const {
    return {src + h * stride, low + h * low_stride, high + h * high_stride, w};
  }
};

constexpr int kAhead = 4;  // vectors of a warp's that are on their way at once

// Turns the block's heads with warps [w0, w0 + nw); `ready` is called once, between the first
// loads and their use, and returns whether to go on (all threads alike).
template <typename T, int NV, typename Ready>
__device__ __forceinline__ bool turn_heads(const Heads<T>& hd, const Kind& k, bool pairs, bool vec, int nh,
                                           int width, const Turn<T>* turns, Ready ready) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (!vec) {
    if (!ready()) return false;
    for (int h = warp; h < nh; h += nw) one_by_one<T>(hd.place(h), k, pairs, turns, lane);
    return true;
  }
  const int groups = 32 / width, l = lane & (width - 1), g = lane / width;
  constexpr int kHold = NV == 1 ? kAhead : 1;
  Held<T, NV> held[kHold];
  bool first = true;
  const int step = nw * groups;
  // (the bound is the same for a whole warp: its lanes meet in the norm's shuffles)
  for (int h0 = warp * groups; first || h0 < nh; h0 += kHold * step) {
#pragma unroll
    for (int u = 0; u < kHold; ++u) {
      const int h = h0 + u * step + g;
      held[u].load(hd.src + h * hd.stride, k, pairs, h < nh, l, width);
    }
    if (first && !ready()) return false;
    first = false;
    __syncwarp();  // in place: every lane's loads come before any lane's stores
#pragma unroll
    for (int u = 0; u < kHold; ++u) {
      const int h = h0 + u * step + g;
      if (h0 + u * step < nh) held[u].finish(hd.place(h), k, pairs, h < nh, l, width, turns);
    }
  }
  return true;
}

struct RopeParams {
  const void* in;
  void* out;
  int64_t in_token, in_head, out_token, out_head;
  int heads, per_block;
  Kind kind;
  int pairs, vec, width;
  const int32_t* positions;
  double sign, mag;
};

template <typename T>
__global__ void __launch_bounds__(kMaxThreads)
    rope_kernel(const RopeParams p, const __grid_constant__ InvFreq inv) {
  extern __shared__ __align__(16) unsigned char smem[];
  Turn<T>* turns = reinterpret_cast<Turn<T>*>(smem);
  const int64_t t = blockIdx.x;
  const int h0 = (int)blockIdx.y * p.per_block, nh = min(p.per_block, p.heads - h0);
  const T* src = (const T*)p.in + t * p.in_token + h0 * p.in_head;
  T* dst = (T*)p.out + t * p.out_token + h0 * p.out_head;
  const Heads<T> hd{src, dst, dst, nullptr, p.in_head, p.out_head, p.out_head};
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const double pos = (double)p.positions[t] * p.sign;
  turn_heads<T, 1>(hd, p.kind, p.pairs, p.vec, nh, p.width, turns, [&]() {
    const int half = p.kind.rot / 2;
    for (int k = threadIdx.x; k < half; k += blockDim.x)
      turns[turn_slot<T>(k, half, p.pairs)] = Turn<T>::make(__dmul_rn(pos, inv.v[k]), p.mag);
    __syncthreads();
    return true;
  });
}

struct NormRopeParams {
  const void *q, *kv, *q_w, *kv_w, *k_w;
  void *q_nope, *q_pe, *c_kv, *k_pe;
  int64_t q_token, q_head, kv_token, ckv_row, kpe_row;
  int64_t nope_token, nope_head, pe_token, pe_head;
  int T, B, H, per_block, groups;
  Kind q_kind, c_kind, k_kind;
  int pairs, q_vec, q_width, c_vec, k_vec, k_width;
  CacheGeom cache;
  int64_t num_rows;
  const int32_t* q_start;
  const int32_t* prefix_len;
  const int32_t* depth;
  int32_t* status;
  double mag;
};

// The sequence of packed token t: the last b with q_start[b] <= t (-1 if there is none, B past
// the last), by one warp in rounds of 32 probes.
__device__ __forceinline__ int sequence_of(const int32_t* __restrict__ q_start, int B, int t, int lane) {
  int lo = 0, n = B + 1;  // the answer is lo - 1 .. lo + n - 1
  while (n > 0) {
    const int step = (n + 31) / 32, i = lo + lane * step;
    const bool le = lane * step < n && __ldg(q_start + i) <= t;
    const uint32_t m = __ballot_sync(0xffffffffu, le);
    const int c = __popc(m);  // probes at or below t (entries ascend)
    if (c == 0) return lo - 1;
    const int last = lo + (c - 1) * step;
    const int end = min(lo + n, last + step);
    lo = last + 1;
    n = end - lo;
  }
  return lo - 1;
}

template <typename T>
__global__ void __launch_bounds__(kMaxThreads)
    norm_rope_kernel(const NormRopeParams p, const __grid_constant__ InvFreq inv) {
  extern __shared__ __align__(16) unsigned char smem[];
  Turn<T>* turns = reinterpret_cast<Turn<T>*>(smem);
  __shared__ int64_t s_row;     // the token's cache row, -1: none
  __shared__ double s_pos;
  __shared__ int s_on;
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h0 = (int)blockIdx.y * p.per_block, nh = max(0, min(p.per_block, p.H - h0));
  const bool keys = p.kv && blockIdx.y == gridDim.y - 1;
  const Heads<T> hd{(const T*)p.q + t * p.q_token + h0 * p.q_head,
                    (T*)p.q_nope + t * p.nope_token + h0 * p.nope_head,
                    (T*)p.q_pe + t * p.pe_token + h0 * p.pe_head,
                    (const T*)p.q_w,
                    p.q_head,
                    p.nope_head,
                    p.pe_head};
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  auto ready = [&]() {
    if (warp == 0) {
      const int b = sequence_of(p.q_start, p.B, (int)t, lane);
      if (lane == 0) {
        bool on = b >= 0 && b < p.B;
        int64_t row = -1;
        if (on) {
          const int64_t i = t - p.q_start[b];
          const int64_t dep = p.depth ? p.depth[t] : i;
          const int P = p.prefix_len[b];
          if (dep < 0) on = false;  // a node of an invalid tree: the row is left alone
          if (on && P < 0) {
            on = false;
            report(p.status, TV_ERR_BOUNDS);
          }
          if (on) {
            s_pos = (double)P + (double)dep;
            const int64_t j = (int64_t)P + i;
            if (keys) {
              if (p.cache.page_table) {
                const int64_t pg = j / p.cache.page_size < p.cache.max_pages
                                       ? p.cache.page_table[(int64_t)b * p.cache.max_pages +
                                                            j / p.cache.page_size]
                                       : -1;
                if (pg >= 0) row = pg * p.cache.page_size + j % p.cache.page_size;
              } else if (j < p.cache.kv_stride_b) {
                row = (int64_t)b * p.cache.kv_stride_b + j;
              }
              if (row >= p.num_rows) row = -1;
              if (row < 0) report(p.status, TV_ERR_BOUNDS);
            }
          }
        }
        s_on = on;
        s_row = row;
      }
    }
    __syncthreads();
    if (!s_on) return false;
    const int half = p.k_kind.rot / 2;
    const double pos = s_pos;
    for (int k = threadIdx.x; k < half; k += blockDim.x)
      turns[turn_slot<T>(k, half, p.pairs)] = Turn<T>::make(__dmul_rn(pos, inv.v[k]), p.mag);
    __syncthreads();
    return true;
  };
  if (!turn_heads<T, 1>(hd, p.q_kind, p.pairs, p.q_vec, nh, p.q_width, turns, ready)) return;
  const int64_t row = s_row;
  if (!keys || row < 0) return;
  const int nw = blockDim.x >> 5;
  const T* src = (const T*)p.kv + t * p.kv_token;
  // the last warp takes the latent row, the one before it (if there is one) the rope part
  if (warp == nw - 1) {
    T* dst = (T*)p.c_kv + row * p.ckv_row;
    const Place<T> pl{src, dst, dst, (const T*)p.kv_w};
    if (p.c_vec) {
      Held<T, kMaxVecs> held;
      held.load(src, p.c_kind, true, true, lane, 32);
      held.finish(pl, p.c_kind, true, true, lane, 32, turns);
    } else {
      one_by_one<T>(pl, p.c_kind, true, turns, lane);
    }
  }
  if (warp == max(0, nw - 2)) {
    T* dst = (T*)p.k_pe + row * p.kpe_row;
    const T* s = src + p.c_kind.n;
    const Place<T> pl{s, dst, dst, (const T*)p.k_w};
    if (p.k_vec) {
      Held<T, 1> held;
      const bool on = lane < p.k_width;
      held.load(s, p.k_kind, p.pairs, on, lane, 32);
      held.finish(pl, p.k_kind, p.pairs, on, lane, 32, turns);
    } else {
      one_by_one<T>(pl, p.k_kind, p.pairs, turns, lane);
    }
  }
}

template <typename T>
bool fits(const void* p) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0;
}

// Whether a kind of vector can be handled 16 bytes at a time by at most `vecs` per lane, and by
// how many lanes (a power of two).
template <typename T>
bool whole_vectors(const Kind& k, bool pairs, int vecs, int* width) {
  constexpr int N = Vec16<T>::N;
  const int part = pairs ? k.rot : k.rot / 2;
  *width = 32;
  if (k.n % N || k.split % N || k.at % N || part % N || k.n > 32 * N * vecs) return false;
  while (*width > 1 && (*width / 2) * N >= k.n) *width /= 2;
  return true;
}

// Heads per block and threads: where the tokens are few their heads go to several blocks, about
// two per SM in all; a warp has `vectors` heads at a time.
struct Shape {
  int per_block, groups, threads;
};
Shape shape(int64_t tokens, int heads, int per_warp) {
  const int64_t want = 2ll * current_sm_count();
  const int groups = tokens >= want ? 1 : (int)std::min<int64_t>(std::max(heads, 1), (want + tokens - 1) / tokens);
  Shape s;
  s.per_block = std::max(1, (heads + groups - 1) / groups);
  s.groups = std::max(1, (heads + s.per_block - 1) / s.per_block);
  const int warps = (s.per_block + 2 * per_warp - 1) / (2 * per_warp);
  s.threads = 32 * std::min(kMaxThreads / 32, std::max(2, warps));
  return s;
}

bool same(const tv_rope_scaling& a, const tv_rope_scaling& b) {
  return a.base == b.base && a.kind == b.kind && a.factor == b.factor &&
         a.original_context == b.original_context && a.low == b.low && a.high == b.high &&
         a.magnitude == b.magnitude;
}
// (the table of the last scaling that a thread used is kept)
const InvFreq& table_of(const tv_rope_scaling& sc, int rot, double* mag) {
  thread_local InvFreq inv{};
  thread_local tv_rope_scaling of{};
  thread_local double of_mag = 1.0;
  thread_local int of_rot = -1;
  if (of_rot != rot || !same(of, sc)) {
    rope_frequencies(sc, rot, inv.v, &of_mag);
    of = sc;
    of_rot = rot;
  }
  *mag = of_mag;
  return inv;
}

template <typename... Args, typename... Given>
cudaError_t start(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                  Given&&... given) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Given>(given)...);
}

template <typename T>
cudaError_t launch_rope_t(const tv_rope_args* a, cudaStream_t st) {
  constexpr int N = Vec16<T>::N;
  RopeParams p{};
  p.in = a->in;
  p.out = a->out;
  p.in_token = a->in_stride_token;
  p.in_head = a->in_stride_head;
  p.out_token = a->out_stride_token;
  p.out_head = a->out_stride_head;
  p.heads = a->n_heads;
  p.kind = {a->d_head, a->rot_offset, a->rot_dim, a->d_head, 0.f};
  const bool in_place = a->in == a->out;
  if (in_place) {  // the elements outside the rotated part are there already
    p.in = (const T*)a->in + a->rot_offset;
    p.out = (T*)a->out + a->rot_offset;
    p.kind = {a->rot_dim, 0, a->rot_dim, a->rot_dim, 0.f};
  }
  p.pairs = a->layout == TV_ROPE_INTERLEAVED;
  p.vec = whole_vectors<T>(p.kind, p.pairs, 1, &p.width) && fits<T>(p.in) && fits<T>(p.out) &&
          p.in_token % N == 0 && p.in_head % N == 0 && p.out_token % N == 0 && p.out_head % N == 0;
  p.positions = a->positions;
  p.sign = a->inverse ? -1.0 : 1.0;
  const InvFreq& inv = table_of(a->scaling, a->rot_dim, &p.mag);
  const Shape s = shape(a->T, a->n_heads, p.vec ? 32 / p.width * kAhead / 2 : 1);
  p.per_block = s.per_block;
  return start(rope_kernel<T>, dim3((unsigned)a->T, (unsigned)s.groups), s.threads,
               sizeof(Turn<T>) * (a->rot_dim / 2), st, p, inv);
}

template <typename T>
cudaError_t launch_norm_rope_t(const tv_norm_rope_args* a, cudaStream_t st) {
  constexpr int N = Vec16<T>::N;
  NormRopeParams p{};
  p.q = a->q;
  p.kv = a->kv;
  p.q_w = a->q_weight;
  p.kv_w = a->kv_weight;
  p.k_w = a->k_weight;
  p.q_nope = a->q_nope;
  p.q_pe = a->q_pe;
  p.c_kv = a->c_kv;
  p.k_pe = a->k_pe;
  p.q_token = a->q_stride_token;
  p.q_head = a->q_stride_head;
  p.kv_token = a->kv_stride_token;
  p.ckv_row = a->ckv_row_stride;
  p.kpe_row = a->kpe_row_stride;
  p.nope_head = a->d_nope;
  p.nope_token = (int64_t)a->H * a->d_nope;
  p.pe_head = a->d_rope;
  p.pe_token = (int64_t)a->H * a->d_rope;
  p.T = a->T;
  p.B = a->B;
  p.H = a->q ? a->H : 0;
  p.q_kind = {a->d_nope + a->d_rope, a->d_nope, a->rot_dim, a->d_nope, a->eps};
  p.c_kind = {a->d_latent, 0, 0, a->d_latent, a->eps};
  p.k_kind = {a->d_rope, 0, a->rot_dim, a->d_rope, a->eps};
  p.pairs = a->layout == TV_ROPE_INTERLEAVED;
  int w;
  p.q_vec = whole_vectors<T>(p.q_kind, p.pairs, 1, &p.q_width) && fits<T>(a->q) && fits<T>(a->q_nope) &&
            fits<T>(a->q_pe) && fits<T>(a->q_weight) && p.q_token % N == 0 && p.q_head % N == 0;
  const bool kv_ok = fits<T>(a->kv) && p.kv_token % N == 0 && a->d_latent % N == 0;
  p.c_vec = whole_vectors<T>(p.c_kind, true, kMaxVecs, &w) && kv_ok && fits<T>(a->c_kv) &&
            p.ckv_row % N == 0 && fits<T>(a->kv_weight);
  p.k_vec = whole_vectors<T>(p.k_kind, p.pairs, 1, &p.k_width) && kv_ok && fits<T>(a->k_pe) &&
            p.kpe_row % N == 0 && fits<T>(a->k_weight);
  p.cache = {a->cache.page_table, a->cache.page_size, a->cache.max_pages, a->cache.kv_stride_b};
  p.num_rows = a->cache.num_rows;
  p.q_start = a->q_start;
  p.prefix_len = a->prefix_len;
  p.depth = a->depth;
  p.status = a->status;
  const InvFreq& inv = table_of(a->scaling, a->rot_dim, &p.mag);
  const Shape s = shape(a->T, p.H, p.q_vec ? 32 / p.q_width * kAhead / 2 : 1);
  p.per_block = s.per_block;
  return start(norm_rope_kernel<T>, dim3((unsigned)a->T, (unsigned)s.groups), s.threads,
               sizeof(Turn<T>) * (a->rot_dim / 2), st, p, inv);
}

}  // namespace

// Frequencies of the rot / 2 pairs and the factor on cos and sin (host).
void rope_frequencies(const tv_rope_scaling& sc, int rot, double* inv, double* mag) {
  constexpr double kTwoPi = 6.283185307179586477;
  const double base = sc.kind == TV_ROPE_NTK
                          ? sc.base * std::pow(sc.factor, (double)rot / std::max(1, rot - 2))
                          : sc.base;
  double lo = 0.0, hi = 0.0;
  if (sc.kind == TV_ROPE_YARN) {
    auto pair_of = [&](double turns) {  // the pair that turns so often over the context
      return rot * std::log(sc.original_context / (kTwoPi * turns)) / (2.0 * std::log(sc.base));
    };
    lo = std::max(std::floor(pair_of(sc.high)), 0.0);
    hi = std::min(std::ceil(pair_of(sc.low)), (double)(rot - 1));
  }
  for (int k = 0; k < rot / 2; ++k) {
    const double f = 1.0 / std::pow(base, (2.0 * (double)k) / (double)rot);
    double keep = 1.0;  // the share of the frequency that is not stretched
    if (sc.kind == TV_ROPE_LINEAR) {
      keep = 0.0;
    } else if (sc.kind == TV_ROPE_YARN) {
      keep = 1.0 - std::min(1.0, std::max(0.0, (k - lo) / std::max(hi - lo, 1e-3)));
    } else if (sc.kind == TV_ROPE_WAVELENGTH) {
      const double turns = sc.original_context * f / kTwoPi;
      keep = std::min(1.0, std::max(0.0, (turns - sc.low) / (sc.high - sc.low)));
    }
    inv[k] = keep == 1.0 || sc.factor == 1.0 ? f : f * keep + f / sc.factor * (1.0 - keep);
  }
  *mag = sc.magnitude != 0.0 ? sc.magnitude
                             : sc.kind == TV_ROPE_YARN ? 0.1 * std::log(sc.factor) + 1.0 : 1.0;
}

cudaError_t launch_rope_any(const tv_rope_args* a, cudaStream_t st) {
  return a->dt == TV_BF16 ? launch_rope_t<__nv_bfloat16>(a, st) : launch_rope_t<float>(a, st);
}

cudaError_t launch_norm_rope(const tv_norm_rope_args* a, cudaStream_t st) {
  return a->dt == TV_BF16 ? launch_norm_rope_t<__nv_bfloat16>(a, st) : launch_norm_rope_t<float>(a, st);
}

}  // namespace tv
