// sample_math.h -- arithmetic shared by the sampling kernels (tv_tree_sample, tv_token_sample):
// the exact weights of logits, rows as 16-byte vectors, and reductions over warps.
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
constexpr ExpTable make_exp_table() {
  ExpTable t{};
  for (int j = 0; j < kTable; ++j) {
    const double x = kLn2 * j / kTable;
    double term = 1.0, sum = 1.0;
    for (int k = 1; k < 24; ++k) {
      term *= x / k;
      sum += term;
    }
    t.hi[j] = (float)sum;
    t.lo[j] = (float)(sum - (double)t.hi[j]);
  }
  return t;
}
__device__ const ExpTable d_exp = make_exp_table();

// 2^((x - m) c) in units of 2^-44, as high * 2^22 + low; c = ch + cl.
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

// The same for two logits at once, in packed float operations (half the instructions; the float
// pipe's work is the same, which is why they are fewer than above: 44 a logit).  The bits may differ
// from those of `weight`: the two parts are summed before the low one is rounded, which is off by
// 5/8 of a unit at most.  The logits lie between lowest() and m: below it weights are zero.
// The table: the two floats in arrays of their own, a copy for each lane.
struct PairTable {
  float hi[kTable * 32], lo[kTable * 32];
};
struct PairScale {
  float m, ch, cl;
  // What smaller logits may be raised to: a logit of weight zero, 46 .. 140 log2 units below m; NaN
  // where there is none, the float before m being farther away.
  __device__ float lowest() const {
    float x = m - 60.f / ch;
    if ((x - m) * ch > -46.f) x = nextafterf(x, -INFINITY);
    const float y = (x - m) * ch;
    return y <= -46.f && y >= -140.f ? x : NAN;
  }
};
struct WeightPair {  // the high and low parts as they leave the float pipe: kPart more each
  int high0, low0, high1, low1;
};
constexpr int kPart = 0x4B400000;  // the bits of 1.5 * 2^23
__device__ __forceinline__ WeightPair weight_pair(float x0, float x1, const PairScale& c,
                                                  const PairTable& table) {
  auto two = [](float v) { return f2_pack(v, v); };
  auto sub = [&](uint64_t a, uint64_t b) { return f2_fma(b, two(-1.f), a); };  // a - b
  constexpr float magic = 12582912.f;
  constexpr float ln2h = (float)kLn2, ln2l = (float)(kLn2 - (double)ln2h);
  const uint64_t x = f2_pack(x0, x1), dh = f2_add(x, two(-c.m)), yh = f2_mul(dh, two(c.ch));
  const uint64_t bb = sub(dh, x);
  const uint64_t dl = sub(sub(x, sub(dh, bb)), f2_add(two(c.m), bb));
  const uint64_t yl = sub(f2_fma(dh, two(c.cl), f2_mul(dl, two(c.ch))), f2_fma(dh, two(-c.ch), yh));
  const uint64_t kr = f2_fma(yh, two((float)kTable), two(magic));
  const uint64_t f = f2_fma(f2_add(kr, two(-magic)), two(-1.f / kTable), yh);
  const uint64_t zh = f2_mul(f, two(ln2h));
  const uint64_t zl = sub(f2_fma(f, two(ln2l), f2_mul(yl, two(ln2h))), f2_fma(f, two(-ln2h), zh));
  const uint64_t q = f2_fma(zh, f2_fma(zh, two(1.f / 24.f), two(1.f / 6.f)), two(0.5f));
  const uint64_t el = f2_fma(f2_mul(zh, zh), q, f2_fma(zh, zl, zl));
  float k0, k1;
  f2_unpack(kr, k0, k1);
  const int i0 = __float_as_int(k0), i1 = __float_as_int(k1), lane = threadIdx.x & 31;
  const int t0 = (i0 & (kTable - 1)) * 32 + lane, t1 = (i1 & (kTable - 1)) * 32 + lane;
  const uint64_t th = f2_pack(table.hi[t0], table.hi[t1]), tl = f2_pack(table.lo[t0], table.lo[t1]);
  const uint64_t ph = f2_mul(th, zh);
  const uint64_t pl = sub(f2_fma(th, el, f2_fma(tl, zh, tl)), f2_fma(th, f2_mul(zh, two(-1.f)), ph));
  const uint64_t h1 = f2_add(th, ph), l1 = f2_add(f2_add(sub(th, h1), ph), pl);
  const uint64_t hi = f2_add(h1, l1), lo = f2_add(sub(h1, hi), l1);
  // 2^22 times the power of two: the integer part of k0 moved to the exponent
  constexpr int e = (22 + 127) << 23;
  const uint64_t s22 = f2_pack(__int_as_float((int)((uint32_t)(i0 & ~(kTable - 1)) << 17) + e),
                               __int_as_float((int)((uint32_t)(i1 & ~(kTable - 1)) << 17) + e));
  const uint64_t a = f2_mul(hi, s22), ra = f2_add(a, two(magic));
  const uint64_t rest = f2_fma(lo, s22, sub(a, f2_add(ra, two(-magic))));
  const uint64_t rb = f2_fma(rest, two(4194304.f), two(magic));
  float a0, a1, b0, b1;
  f2_unpack(ra, a0, a1);
  f2_unpack(rb, b0, b1);
  return {__float_as_int(a0), __float_as_int(b0), __float_as_int(a1), __float_as_int(b1)};
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
