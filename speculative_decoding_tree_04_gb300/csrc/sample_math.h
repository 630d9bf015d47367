// sample_math.h -- arithmetic shared by the sampling kernels (tv_tree_sample, tv_token_sample):
// the integer weights of logits, rows as 16-byte vectors, and reductions over warps.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "sm100_ptx.h"

namespace tv {
namespace {

using namespace ptx;

constexpr float kUnit = 17592186044416.f;  // 2^44 units per largest weight
constexpr int kTable = 64;
constexpr double kLn2 = 0.693147180559945309417;
constexpr int kCopies = 16;     // of the table, one for each lane of a half warp: no conflicts

// 2^(j/64) as the sum of two floats, from the exponential's Taylor series in double.
struct ExpTable {
  float hi[kTable], lo[kTable];
};
constexpr ExpTable make_exp_table(bool over_linear) {
  ExpTable t{};
  for (int j = 0; j < kTable; ++j) {
    const double x = kLn2 * j / kTable;
    double term = 1.0, sum = 1.0;
    for (int k = 1; k < 24; ++k) {
      term *= x / k;
      sum += term;
    }
    if (over_linear) sum /= 1.0 + (double)j / kTable;
    t.hi[j] = (float)sum;
    t.lo[j] = (float)(sum - (double)t.hi[j]);
  }
  return t;
}
__device__ const ExpTable d_exp = make_exp_table(false);
__device__ const ExpTable d_exp_over_linear = make_exp_table(true);  // 2^(j/64) / (1 + j/64)

// 2^((x - m) c) in units of 2^-44 (tv_tree_sample), as high * 2^22 + low; c = ch + cl.
// With y = (x - m) c = k/64 + f: 2^y = 2^(k/64) e^(f ln 2), the first factor from the
// table, the second by its series (|f ln 2| < 0.0055: the z^5 term is below 2^-44).  Floats
// become integers by adding 1.5 * 2^23, whose last place is 1, which takes magnitudes up to
// 2^22: conversions run at a quarter of the rate.
struct Weight {
  int high, low;
};
__device__ __forceinline__ Weight weight(float x, float m, float ch, float cl,
                                         const float2* __restrict__ table) {
  const float dh = x - m;
  const float y0 = dh * ch;
  const bool some = y0 > -46.f;  // else below half a unit; -inf (masked) too
  const float yh = some ? y0 : 0.f;
  const float bb = dh - x;
  const float dl = (x - (dh - bb)) - (m + bb);
  const float yl = fmaf(dh, ch, -yh) + fmaf(dh, cl, dl * ch);
  constexpr float magic = 12582912.f;
  const float kr = fmaf(yh, (float)kTable, magic);
  const int ki = __float_as_int(kr) - __float_as_int(magic);
  const float f = fmaf(kr - magic, -1.f / kTable, yh);  // exact
  constexpr float ln2h = (float)kLn2, ln2l = (float)(kLn2 - (double)ln2h);
  const float zh = f * ln2h;
  const float zl = fmaf(f, ln2h, -zh) + fmaf(f, ln2l, yl * ln2h);
  const float p =
      zh * zh * fmaf(zh, fmaf(zh, fmaf(zh, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f), 0.5f);
  const float el = fmaf(zh, zl, zl) + p;
  const float2 t = table[(ki & (kTable - 1)) * kCopies + (threadIdx.x & (kCopies - 1))];
  const float ph = t.x * zh;
  const float pl = fmaf(t.x, zh, -ph) + fmaf(t.x, el, fmaf(t.y, zh, t.y));
  // (summed once more, so that the low part is a rounding of the high one, 2^20 units at most:
  // without that it holds z^2 / 2, up to 2^28 units, past what the sum below can take)
  const float h1 = t.x + ph, l1 = ((t.x - h1) + ph) + pl;
  const float hi = h1 + l1, lo = (h1 - hi) + l1;
  const int e = (ki >> 6) << 23;
  const float a = hi * __int_as_float(e + ((22 + 127) << 23));
  const float ra = a + magic;
  const float rb = fmaf(a - (ra - magic), 4194304.f,
                        lo * __int_as_float(e + ((44 + 127) << 23))) + magic;
  return {some ? __float_as_int(ra) - __float_as_int(magic) : 0,
          some ? __float_as_int(rb) - __float_as_int(magic) : 0};
}
__device__ __forceinline__ int64_t units(Weight w) { return ((int64_t)w.high << 22) + w.low; }

// e^((x - m) / T) in the same units, in 31 float operations.  With d = m - x and
// d / T = k ln 2 / 64 + q - s, k an integer, q what is left of the rounded quotient (exact: its last
// place is not below 2^-31 where k is not 0) and s the errors of all roundings,
//     e^(-d/T) = 2^(-k/64) e^(s - q),   e^(s - q) = 1 - q + s (1 - q) + q^2/2 - q^3/6 + q^4/24
// up to 2^-44.  The difference's error takes two operations where m is a multiple of every logit's
// last place (Dekker's sum); m is rounded to one, by 2^-24 of itself or of 60 T, and what that
// leaves is added to d / T, to 2^-49 of |m| / T.  The bits may differ from those of `weight`: the
// two parts are summed before the low one is rounded, which is off by 5/8 of a unit at most.  The
// logits lie between the scale's lowest and the maximum.
// The power of two: the bits of -k, moved to where an exponent's begin, are a float 2^i (1 + j/64)
// with -k = 64 i + j, so that the table holds 2^(j/64) / (1 + j/64).  Its two floats are in arrays
// of their own, a copy for each lane.
struct ScaledTable {
  float hi[kTable * 32], lo[kTable * 32];
};
struct RowScale {
  float m, rest;  // m + rest T: the maximum
  float th, tl;   // 1 / T as two floats
  float k64;      // 64 log2(e) / T
  // largest: the maximum; lowest: what smaller logits may be raised to, a logit of weight zero, 46 ..
  // 140 log2 units below it; NaN where there is none, the float before the maximum being farther
  // away: then all others weigh nothing.
  __device__ RowScale(float largest, float T, float* lowest) {
    T = fminf(fmaxf(T, 1.5e-30f), 1.4e30f);
    th = 1.f / T;
    tl = fmaf(-th, T, 1.f) / T;
    const float log2e = (float)(1.0 / kLn2);
    k64 = (float)kTable * log2e * th;
    auto below = [&](float x) { return (largest - x) * th * log2e; };
    float x = largest - 60.f / (log2e * th);
    if (below(x) < 46.f) x = nextafterf(x, -INFINITY);
    *lowest = below(x) >= 46.f && below(x) <= 140.f ? x : NAN;
    m = largest;
    if (fabsf(x) > fabsf(largest)) {  // (then x is finite or there is no lowest)
      // 1.5 * 2^23 of x's last places
      const float c = 1.5f * __uint_as_float(__float_as_uint(x) & 0x7F800000u);
      m = __fadd_rn(__fadd_rn(largest, c), -c);
    }
    rest = (largest - m) / T;
  }
};
__device__ __forceinline__ Weight scaled_weight(float x, const RowScale& c, const ScaledTable& table) {
  constexpr float magic = 12582912.f;
  constexpr float step = (float)(kLn2 / kTable), step_low = (float)(kLn2 / kTable - (double)step);
  const float d = __fsub_rn(c.m, x), dl = __fsub_rn(__fsub_rn(c.m, d), x);
  const float p = fmaf(d, c.th, c.rest);
  const float kr = fmaf(d, -c.k64, magic), k = __fsub_rn(kr, magic);  // -k
  const float q = fmaf(k, step, p);
  float s = fmaf(d, -c.tl, __fsub_rn(fmaf(d, -c.th, p), c.rest));
  s = fmaf(k, -step_low, fmaf(dl, -c.th, s));
  const float series = fmaf(q, fmaf(q, 1.f / 24.f, -1.f / 6.f), 0.5f);
  const float e = fmaf(__fmul_rn(q, q), series, fmaf(s, -q, s));
  const int i = __float_as_int(kr);
  const int t = (i & (kTable - 1)) * 32 + (threadIdx.x & 31);
  const float th = table.hi[t], tl = table.lo[t];
  const float ph = __fmul_rn(th, q);
  const float low = __fadd_rn(fmaf(th, e, fmaf(tl, -q, tl)), fmaf(-th, q, ph));
  const float hi = __fadd_rn(th, __fsub_rn(low, ph));
  const float lo = __fadd_rn(__fsub_rn(__fsub_rn(th, hi), ph), low);
  const float s22 = __int_as_float((int)((uint32_t)i << 17) + ((22 + 127) << 23));
  const float ra = fmaf(hi, s22, magic);
  const float left = fmaf(lo, s22, fmaf(hi, s22, __fsub_rn(magic, ra)));
  const float rb = fmaf(left, 4194304.f, magic);
  return {__float_as_int(ra) - __float_as_int(magic), __float_as_int(rb) - __float_as_int(magic)};
}
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4, kUnroll = 8;  // elements per 16 bytes, loads in flight
  static constexpr uint32_t kMasked = 0xFF800000u;  // a word of -inf
  __device__ static void unpack(const uint4& w, float* x) {
    x[0] = __uint_as_float(w.x);
    x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z);
    x[3] = __uint_as_float(w.w);
  }
  __device__ static float one(const float* p) { return __ldg(p); }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8, kUnroll = 4;
  static constexpr uint32_t kMasked = 0xFF80FF80u;
  __device__ static void unpack(const uint4& w, float* x) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(v[i] << 16);
      x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    }
  }
  __device__ static float one(const __nv_bfloat16* p) { return __bfloat162float(__ldg(p)); }
};

// A row as 16-byte vectors on 16-byte boundaries: vector j holds elements j*N - off ..,
// where the row starts `off` elements past a boundary.  Elements outside the row read as
// -inf, whose weight is zero.
template <typename T>
struct Row {
  const T* x;
  int64_t V;
  int off, n_vec;
  __device__ Row(const T* row, int64_t vocab) : x(row), V(vocab) {
    off = (int)(((uintptr_t)row & 15u) / sizeof(T));
    n_vec = (int)((V + off + Vec<T>::N - 1) / Vec<T>::N);
  }
  // Whether token v lies in the i-th of the parts of `per` vectors that start at `from`.
  __device__ bool in_part(int64_t v, int per, int i, int from = 0) const {
    const int j = (int)((v + off) / Vec<T>::N) - from;
    return j >= i * per && j < (i + 1) * per;
  }
  __device__ int64_t first(int j) const { return (int64_t)j * Vec<T>::N - off; }
  __device__ bool whole(int j) const { return first(j) >= 0 && first(j) + Vec<T>::N <= V; }
  // The vectors that lie in the row whole, [first_whole, end_whole).
  __device__ int first_whole() const { return off > 0 ? 1 : 0; }
  __device__ int end_whole() const { return (int)((V + off) / Vec<T>::N); }
  __device__ uint4 raw(int j) const {  // of those
    return __ldg(reinterpret_cast<const uint4*>(x + first(j)));
  }
  __device__ void load(int j, float* v) const {
    const int64_t a = first(j);
    if (whole(j)) {
      Vec<T>::unpack(__ldg(reinterpret_cast<const uint4*>(x + a)), v);
      return;
    }
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i)
      v[i] = a + i >= 0 && a + i < V ? Vec<T>::one(x + a + i) : -INFINITY;
  }
};

__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v == 0.f ? 0.f : v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

__device__ __forceinline__ void st_cluster_u32(const void* local, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_to_rank(smem_u32(local), rank)), "r"(v)
               : "memory");
}
__device__ __forceinline__ void st_cluster_f32(const void* local, uint32_t rank, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(map_to_rank(smem_u32(local), rank)), "f"(v)
               : "memory");
}
__device__ __forceinline__ void st_cluster_u64(const void* local, uint32_t rank, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(map_to_rank(smem_u32(local), rank)), "l"(v)
               : "memory");
}

template <typename S>
__device__ __forceinline__ S warp_sum(S s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// Largest of one 64-bit key per lane.
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
  const uint32_t high = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
  const uint32_t low =
      __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == high ? (uint32_t)k : 0u);
  return ((uint64_t)high << 32) | low;
}
// Where `target` lies among one part per lane: the lane, and what is left of the target there.
// The last lane below `parts` takes what rounding might leave over.
template <typename S>
__device__ __forceinline__ int locate(S part, int parts, S* target) {
  const int lane = threadIdx.x & 31;
  S up_to = lane < parts ? part : (S)0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const S below = __shfl_up_sync(0xffffffffu, up_to, o);
    if (lane >= o) up_to += below;
  }
  const uint32_t past = __ballot_sync(0xffffffffu, lane < parts && up_to > *target);
  const int at = past ? __ffs(past) - 1 : parts - 1;
  *target -= __shfl_sync(0xffffffffu, up_to - part, at);
  return at;
}

}  // namespace
}  // namespace tv
