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
// What bounds it: bytes for prompts, latency for single tokens.  A head is held in registers by a
// group of 1 to 32 lanes, up to four 16-byte vectors a lane, as few lanes idle as that allows (192
// bf16: 8 lanes of three), so that the norm costs a few shuffles and no second read; in the half
// layout a lane loads its vectors' partners too, from
// lines that the warp's own loads bring.  A block serves up to eight tokens, their heads one
// list that its warps go through without meeting again once the tokens' cosines and sines are
// there (taken while the first heads are on their way), or where the tokens are few a part of
// one token's heads.
//
// Measured, in a graph of such calls: 4096 tokens of 64 bf16 heads of 192, the last 64 turned, 34.6 us
// = 5.8 TB/s, 87 % of a copy's rate; 1001 x 5 float32 heads of 80, 6.4 us (double trigonometry);
// 64 single tokens of 64 heads of 64, 3.1 us.  With norms and keys, bf16, 64 heads of 128 + 64 and
// latent rows of 512: 2619 tokens 35 us = 3.9 TB/s, where issue slots (0.57 a cycle) and the
// latency between a head's loads, its norm's shuffles and its stores share the time; 64 single
// tokens 5.2 us.  The same in float32: 2619 tokens of one prompt 77 us = 3.5 TB/s; 64 of one, 7.3 us.  A software pipeline over heads took the norms to 34.1 us and the rotations to
// 39.3, and was not kept; nor two or four blocks per SM for the norms in the place of three.
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
using namespace ptx;

constexpr int kMaxThreads = 256;
constexpr int kMaxVecs = 4;  // 16-byte vectors of one head that a lane holds at most

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
  float eps, inv_n;  // with a weight: the norm's; 1 / n
};

// The turns of one token's pairs in shared memory, as the vectors' lanes read them: those of one
// vector in 16-byte pieces, and the pieces that the lanes read together consecutive, so that no two
// of them meet in a bank.  Where there are no vectors (`half` pairs do not fill them) turns are
// read one by one, in order.
template <typename T>
struct Turns;
template <>
struct Turns<float> {
  Turn<float> t[1];  // half of them
  __device__ static int slot(int k, int half, bool pairs) {
    const int per = pairs ? 2 : 4;  // pairs of one vector
    return half % per ? k : k % per * (half / per) + k / per;
  }
  static constexpr size_t bytes(int half) { return half * sizeof(Turn<float>); }
  __device__ void set(int k, int half, bool pairs, const Turn<float>& x) { t[slot(k, half, pairs)] = x; }
  __device__ Turn<float> get(int k, int half, bool pairs) const { return t[slot(k, half, pairs)]; }
};
// bf16: (cos, cos, sin, sin) of two pairs whose elements lie in the same halves of neighbouring
// words, for packed arithmetic.
template <>
struct Turns<__nv_bfloat16> {
  float f[4];
  __device__ static int slot(int k, int half, bool pairs) {
    if (half % (pairs ? 4 : 8)) return 4 * (k / 2) + (k & 1);
    // pairs: pair j of a vector is word j.  half layout: the vector's elements 2 j and 2 j + 1
    const int j = pairs ? k & 3 : k & 7, v = pairs ? k >> 2 : k >> 3, n = pairs ? half >> 2 : half >> 3;
    const int word = pairs ? j : j >> 1, piece = pairs ? word >> 1 : 2 * (word >> 1) + (j & 1);
    return 4 * (piece * n + v) + (word & 1);
  }
  static constexpr size_t bytes(int half) { return (half + 1) / 2 * 16; }
  __device__ void set(int k, int half, bool pairs, const Turn<__nv_bfloat16>& x) {
    float* at = f + slot(k, half, pairs);
    at[0] = x.c;
    at[2] = x.s;
  }
  __device__ Turn<__nv_bfloat16> get(int k, int half, bool pairs) const {
    const float* at = f + slot(k, half, pairs);
    return {at[0], at[2]};
  }
};
template <typename T>
__device__ __forceinline__ const Turns<T>* turns_of(const unsigned char* all, int token, int half) {
  return reinterpret_cast<const Turns<T>*>(all + token * Turns<T>::bytes(half));
}

// A head in 16-byte pieces by the `width` lanes of a group (lane `l` of it, vectors l, l + width,
// ..).  Loads first, then, by `finish`, the norm, the rotation and the stores.  `other` holds the
// partners in the half layout; kSwap: they are `swap` lanes away instead (or in the same vector).
template <typename T, int NV, bool kSwap>
struct Held;

template <int NV, bool kSwap>
struct Held<float, NV, kSwap> {
  uint4 own[NV], other[NV];
  __device__ __forceinline__ void load(const float* src, const Kind& k, bool pairs, bool on, int l, int width) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (l + i * width) * 4;
      if (!on || e >= k.n) continue;
      own[i] = *reinterpret_cast<const uint4*>(src + e);
      if (!pairs && e >= k.at && e < k.at + k.rot) {
        const int half = k.rot / 2;
        other[i] = *reinterpret_cast<const uint4*>(src + (e < k.at + half ? e + half : e - half));
      }
    }
  }
  // w: the norm's weights, null for none (the same for a whole warp, whose lanes meet in the sum).
  __device__ __forceinline__ void finish(float* low, float* high, const Kind& k, bool pairs, int,
                                         const float* w, bool on, int l, int width,
                                         const Turns<float>* turns) {
    const int half = k.rot / 2;
    float r = 1.f;
    if (w) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!on || (l + i * width) * 4 >= k.n) continue;
        float x[4];
        Vec16<float>::unpack(own[i], x);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum = fmaf(x[j], x[j], sum);
      }
      for (int o = width / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      r = 1.f / sqrtf(sum / (float)k.n + k.eps);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (l + i * width) * 4;
      if (!on || e >= k.n) continue;
      float x[4];
      Vec16<float>::unpack(own[i], x);
      if (w) {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = x[j] * r * __ldg(w + e + j);
      }
      if (e >= k.at && e < k.at + k.rot) {
        const int q = e - k.at;
        if (pairs) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const Turn<float>& t = turns->t[j * (half / 2) + q / 4];
            const float a = x[2 * j], b = x[2 * j + 1];
            x[2 * j] = t.out(a, b);
            x[2 * j + 1] = t.out(b, -a);
          }
        } else {
          const bool first = q < half;
          const int v = (first ? q : q - half) / 4;
          float y[4];
          Vec16<float>::unpack(other[i], y);
          if (w) {
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = y[j] * r * __ldg(w + (first ? e + half : e - half) + j);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            x[j] = turns->t[j * (half / 4) + v].out(x[j], first ? y[j] : -y[j]);
        }
      }
      *reinterpret_cast<uint4*>(e < k.split ? low + e : high + (e - k.split)) = Vec16<float>::pack(x);
    }
  }
};

// Eight bf16 as four pairs of floats for packed arithmetic: {elements 0 and 2, 1 and 3, 4 and 6, 5
// and 7} (the same halves of neighbouring words).
__device__ __forceinline__ void unpack_pairs(const uint4& u, uint64_t* x) {
  const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[2 * i] = f2_pack(__uint_as_float(v[2 * i] << 16), __uint_as_float(v[2 * i + 1] << 16));
    x[2 * i + 1] =
        f2_pack(__uint_as_float(v[2 * i] & 0xffff0000u), __uint_as_float(v[2 * i + 1] & 0xffff0000u));
  }
}
__device__ __forceinline__ uint4 pack_pairs(const uint64_t* x) {
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float a0, a1, b0, b1;
    f2_unpack(x[2 * i], a0, a1);
    f2_unpack(x[2 * i + 1], b0, b1);
    const __nv_bfloat162 p = __floats2bfloat162_rn(a0, b0), q = __floats2bfloat162_rn(a1, b1);
    v[2 * i] = *reinterpret_cast<const uint32_t*>(&p);
    v[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&q);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ uint64_t f2_swap_lanes(uint64_t x, int lanes) {
  float a, b;
  f2_unpack(x, a, b);
  return f2_pack(__shfl_xor_sync(0xffffffffu, a, lanes), __shfl_xor_sync(0xffffffffu, b, lanes));
}

template <int NV, bool kSwap>
struct Held<__nv_bfloat16, NV, kSwap> {
  using T = __nv_bfloat16;
  uint4 own[NV], other[kSwap ? 1 : NV];
  __device__ __forceinline__ void load(const T* src, const Kind& k, bool pairs, bool on, int l, int width) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (l + i * width) * 8;
      own[i] = make_uint4(0u, 0u, 0u, 0u);
      if (!on || e >= k.n) continue;
      own[i] = *reinterpret_cast<const uint4*>(src + e);
      if (!kSwap && !pairs && e >= k.at && e < k.at + k.rot) {
        const int half = k.rot / 2;
        other[i] = *reinterpret_cast<const uint4*>(src + (e < k.at + half ? e + half : e - half));
      }
    }
  }
  __device__ __forceinline__ void finish(T* low, T* high, const Kind& k, bool pairs, int swap, const T* w,
                                         bool on, int l, int width, const Turns<T>* turns) {
    const int half = k.rot / 2;
    uint64_t r2 = 0;
    if (w) {
      uint64_t s2 = f2_pack(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        uint64_t x[4];
        unpack_pairs(own[i], x);
#pragma unroll
        for (int j = 0; j < 4; ++j) s2 = f2_fma(x[j], x[j], s2);
      }
      float s0, s1;
      f2_unpack(s2, s0, s1);
      float sum = s0 + s1;
      for (int o = width / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float mean = fmaf(sum, k.inv_n, k.eps);
      float r = rsqrtf(mean);                        // and a step of Newton's iteration
      r = fmaf(0.5f * r, fmaf(-mean * r, r, 1.f), r);
      // (a mean of 0, its square root infinite, or past the step's range: the plain value)
      if (!(mean > 1e-30f && mean < 1e30f)) r = 1.f / sqrtf(mean);
      r2 = f2_pack(r, r);
    }
    const int at = k.at, end = k.at + k.rot;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (l + i * width) * 8;
      const bool valid = on && e < k.n;
      uint64_t x[4];
      unpack_pairs(own[i], x);
      if (w) {
        uint64_t f[4];
        unpack_pairs(valid ? __ldg(reinterpret_cast<const uint4*>(w + e)) : make_uint4(0u, 0u, 0u, 0u), f);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = f2_mul(f2_mul(x[j], r2), f[j]);
      }
      // (a vector of the warp's is rotated: where lanes swap, all of them take part)
      if (i * width * 8 < end && (i + 1) * width * 8 > at) {
        const bool turned = valid && e >= at && e < end;
        const int q = e - at;
        if (pairs) {
          if (turned) {
            const float4* t = reinterpret_cast<const float4*>(turns->f) + (q >> 3);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float4 cs = t[j * (half >> 2)];
              const uint64_t c = f2_pack(cs.x, cs.y), sn = f2_pack(cs.z, cs.w),
                             neg = f2_pack(-cs.z, -cs.w);
              const uint64_t a = x[2 * j], b = x[2 * j + 1];
              x[2 * j] = f2_fma(a, c, f2_mul(b, neg));
              x[2 * j + 1] = f2_fma(b, c, f2_mul(a, sn));
            }
          }
        } else {
          const bool first = q < half;
          uint64_t y[4];
          if (kSwap) {
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = f2_swap_lanes(x[j], swap);
          } else if (turned) {
            unpack_pairs(other[i], y);
            if (w) {
              uint64_t f[4];
              unpack_pairs(__ldg(reinterpret_cast<const uint4*>(w + (first ? e + half : e - half))), f);
#pragma unroll
              for (int j = 0; j < 4; ++j) y[j] = f2_mul(f2_mul(y[j], r2), f[j]);
            }
          }
          if (turned) {
            const float4* t = reinterpret_cast<const float4*>(turns->f) + ((first ? q : q - half) >> 3);
            const float sg = first ? -1.f : 1.f;
            const uint64_t sign = f2_pack(sg, sg);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float4 cs = t[j * (half >> 3)];
              x[j] = f2_fma(x[j], f2_pack(cs.x, cs.y), f2_mul(f2_mul(y[j], sign), f2_pack(cs.z, cs.w)));
            }
          }
        }
      }
      if (valid) *reinterpret_cast<uint4*>(e < k.split ? low + e : high + (e - k.split)) = pack_pairs(x);
    }
  }
};

// The same for one vector of any size and alignment, an element (or a pair) at a time; a lane
// reads both elements of a pair before it writes either, so the vector may be turned in place.
template <typename T>
__device__ void one_by_one(const T* src, T* low, T* high, const T* w, const Kind& k, bool pairs,
                           const Turns<T>* turns, int lane) {
  float r = 1.f;
  if (w) {
    float sum = 0.f;
    for (int e = lane; e < k.n; e += 32) {
      const float x = to_float(src[e]);
      sum = fmaf(x, x, sum);
    }
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    r = 1.f / sqrtf(sum / (float)k.n + k.eps);
  }
  auto get = [&](int e) {
    const float x = to_float(src[e]);
    return w ? x * r * to_float(w[e]) : x;
  };
  auto put = [&](int e, float y) { store_float(e < k.split ? low + e : high + (e - k.split), y); };
  for (int e = lane; e < k.n; e += 32)
    if (e < k.at || e >= k.at + k.rot) put(e, get(e));
  const int half = k.rot / 2;
  for (int i = lane; i < half; i += 32) {
    const int ea = k.at + (pairs ? 2 * i : i), eb = pairs ? ea + 1 : ea + half;
    const float a = get(ea), b = get(eb);
    const Turn<T> t = turns->get(i, half, pairs);
    put(ea, t.out(a, b));
    put(eb, t.out(b, -a));
  }
}

// Heads [h0, h0 + nh) of tokens [t0, t0 + nt), one list.
template <typename T>
struct Heads {
  const T* src;
  T* low;
  T* high;
  const T* w;
  int64_t token, stride, low_token, low_stride, high_token, high_stride;
  int64_t t0;
  int h0, nh, nt;
};

// Turns the list with all of the block's warps.  `ready` is called once by every thread, between
// the first loads and their use; on[i] then says whether token t0 + i takes part, and its turns
// are the i-th.
template <typename T, int NV, bool kSwap, typename Ready>
__device__ __forceinline__ void turn_heads(const Heads<T>& hd, const Kind& k, bool pairs, int width,
                                           int swap, const unsigned char* turns, const bool* on, Ready ready) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  const int half = k.rot / 2, n = hd.nh * hd.nt;
  const T* src0 = hd.src + hd.t0 * hd.token + hd.h0 * hd.stride;
  T* low0 = hd.low + hd.t0 * hd.low_token + hd.h0 * hd.low_stride;
  T* high0 = hd.high + hd.t0 * hd.high_token + hd.h0 * hd.high_stride;
  auto src = [&](int i, int h) { return src0 + i * hd.token + h * hd.stride; };
  auto low = [&](int i, int h) { return low0 + i * hd.low_token + h * hd.low_stride; };
  auto high = [&](int i, int h) { return high0 + i * hd.high_token + h * hd.high_stride; };
  if (width == 0) {
    ready();
    for (int q = warp; q < n; q += nw) {
      const int i = q / hd.nh, h = q - i * hd.nh;
      if (on[i])
        one_by_one<T>(src(i, h), low(i, h), high(i, h), hd.w, k, pairs, turns_of<T>(turns, i, half), lane);
    }
    return;
  }
  const int groups = 32 / width, l = lane & (width - 1), g = lane / width;
  // heads of a group on their way at once (float32 rotations are long: fewer copies of them)
  constexpr int kHold = sizeof(T) == 4 ? (NV == 1 ? 2 : 1) : NV == 1 ? 4 : NV == 2 ? 2 : 1;
  Held<T, NV, kSwap> held[kHold];
  const int step = nw * groups;
  int ti[kHold], hi[kHold];
#pragma unroll
  for (int u = 0; u < kHold; ++u) {
    const int q = warp * groups + u * step + g;
    ti[u] = q / hd.nh;
    hi[u] = q - ti[u] * hd.nh;
  }
  bool first = true;
  // (the bound is the same for a whole warp: its lanes meet in shuffles)
  for (int q0 = warp * groups; first || q0 < n; q0 += kHold * step) {
#pragma unroll
    for (int u = 0; u < kHold; ++u)
      held[u].load(src(ti[u], hi[u]), k, pairs, q0 + u * step + g < n, l, width);
    if (first) ready();
    first = false;
    __syncwarp();  // in place: every lane's loads come before any lane's stores
#pragma unroll
    for (int u = 0; u < kHold; ++u) {
      if (q0 + u * step < n) {
        const bool is = q0 + u * step + g < n && on[ti[u]];
        held[u].finish(low(ti[u], hi[u]), high(ti[u], hi[u]), k, pairs, swap, hd.w, is, l, width,
                       turns_of<T>(turns, ti[u], half));
      }
      // the next head of this lane's
      hi[u] += kHold * step;
      while (hi[u] >= hd.nh) {
        hi[u] -= hd.nh;
        ++ti[u];
      }
    }
  }
}

constexpr int kMaxTokens = 8;  // of a block

// Angles of the block's tokens, all at once.
template <typename T>
__device__ __forceinline__ void make_turns(unsigned char* turns, const double* pos, const bool* on, int nt,
                                           int half, bool pairs, const InvFreq& inv, double mag) {
  for (int x = threadIdx.x; x < nt * half; x += blockDim.x) {
    const int i = x / half, k = x - i * half;
    if (on[i])
      const_cast<Turns<T>*>(turns_of<T>(turns, i, half))
          ->set(k, half, pairs, Turn<T>::make(__dmul_rn(pos[i], inv.v[k]), mag));
  }
}

struct RopeParams {
  const void* in;
  void* out;
  int64_t in_token, in_head, out_token, out_head;
  int T, heads, per_block, tokens;
  Kind kind;
  int pairs, width, swap;
  const int32_t* positions;
  double sign, mag;
};

template <typename T, int NV, bool kSwap>
__global__ void __launch_bounds__(kMaxThreads)
    rope_kernel(const RopeParams p, const __grid_constant__ InvFreq inv) {
  extern __shared__ __align__(16) unsigned char turns[];
  __shared__ double pos[kMaxTokens];
  __shared__ bool on[kMaxTokens];
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
  const int nt = (int)min((int64_t)p.tokens, p.T - t0);
  const int h0 = (int)blockIdx.y * p.per_block, nh = min(p.per_block, p.heads - h0);
  const Heads<T> hd{(const T*)p.in, (T*)p.out,   (T*)p.out,  nullptr,     p.in_token, p.in_head,
                    p.out_token,    p.out_head, p.out_token, p.out_head, t0,          h0,
                    nh,             nt};
  griddep_wait();
  griddep_launch_dependents();
  turn_heads<T, NV, kSwap>(hd, p.kind, p.pairs, p.width, p.swap, turns, on, [&]() {
    if (threadIdx.x < nt) {
      pos[threadIdx.x] = (double)p.positions[t0 + threadIdx.x] * p.sign;
      on[threadIdx.x] = true;
    }
    __syncthreads();
    make_turns<T>(turns, pos, on, nt, p.kind.rot / 2, p.pairs, inv, p.mag);
    __syncthreads();
  });
}

struct NormRopeParams {
  const void *q, *kv, *q_w, *kv_w, *k_w;
  void *q_nope, *q_pe, *c_kv, *k_pe;
  int64_t q_token, q_head, kv_token, ckv_row, kpe_row;
  int64_t nope_token, nope_head, pe_token, pe_head;
  int T, B, H, per_block, tokens;
  Kind q_kind, c_kind, k_kind;
  int pairs, q_width, q_swap, c_vec, k_vec;
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
__device__ __forceinline__ int sequence_of(const int32_t* __restrict__ q_start, int B, int64_t t, int lane) {
  uint32_t lo = 0, n = (uint32_t)B + 1;  // the answer is lo - 1 .. lo + n - 1
  while (n > 0) {
    const uint32_t step = (n + 31) / 32, i = lo + (uint32_t)lane * step;
    const bool le = (uint32_t)lane * step < n && __ldg(q_start + i) <= t;
    const uint32_t m = __ballot_sync(0xffffffffu, le);
    const uint32_t c = (uint32_t)__popc(m);  // probes at or below t (entries ascend)
    if (c == 0) break;
    const uint32_t last = lo + (c - 1) * step;
    const uint32_t end = min(lo + n, last + step);
    lo = last + 1;
    n = end - lo;
  }
  return (int)lo - 1;
}

template <typename T, int NV, bool kSwap>
__global__ void __launch_bounds__(kMaxThreads, 3)
    norm_rope_kernel(const NormRopeParams p, const __grid_constant__ InvFreq inv) {
  extern __shared__ __align__(16) unsigned char turns[];
  __shared__ int64_t rows[kMaxTokens];  // the tokens' cache rows, -1: none
  __shared__ double pos[kMaxTokens];
  __shared__ bool on[kMaxTokens];
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
  const int nt = (int)min((int64_t)p.tokens, p.T - t0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int h0 = (int)blockIdx.y * p.per_block, nh = max(0, min(p.per_block, p.H - h0));
  const bool keys = p.kv && blockIdx.y == gridDim.y - 1;
  const Heads<T> hd{(const T*)p.q, (T*)p.q_nope, (T*)p.q_pe,  (const T*)p.q_w, p.q_token, p.q_head,
                    p.nope_token,  p.nope_head,  p.pe_token, p.pe_head,       t0,        h0,
                    max(nh, 1),    nh > 0 ? nt : 0};
  griddep_wait();
  griddep_launch_dependents();
  auto ready = [&]() {
    for (int i = warp; i < nt; i += nw) {
      const int64_t t = t0 + i;
      const int b = sequence_of(p.q_start, p.B, t, lane);
      if (lane > 0) continue;
      bool is = b >= 0 && b < p.B;
      int64_t row = -1;
      if (is) {
        const int64_t at = t - p.q_start[b];
        const int64_t dep = p.depth ? p.depth[t] : at;
        const int P = p.prefix_len[b];
        const bool sound = P >= 0 && at >= 0;  // (a q_start that does not ascend finds anything)
        if (!sound) report(p.status, TV_ERR_BOUNDS);
        is = dep >= 0 && sound;  // (a node of an invalid tree is left alone)
        pos[i] = (double)P + (double)dep;
        if (is && keys) {
          const int64_t j = (int64_t)P + at;
          if (p.cache.page_table) {
            const int64_t pg =
                j / p.cache.page_size < p.cache.max_pages
                    ? p.cache.page_table[(int64_t)b * p.cache.max_pages + j / p.cache.page_size]
                    : -1;
            if (pg >= 0) row = pg * p.cache.page_size + j % p.cache.page_size;
          } else if (j < p.cache.kv_stride_b) {
            row = (int64_t)b * p.cache.kv_stride_b + j;
          }
          if (row >= p.num_rows) row = -1;
          if (row < 0) report(p.status, TV_ERR_BOUNDS);
        }
      }
      on[i] = is;
      rows[i] = row;
    }
    __syncthreads();
    make_turns<T>(turns, pos, on, nt, p.k_kind.rot / 2, p.pairs, inv, p.mag);
    __syncthreads();
  };
  turn_heads<T, NV, kSwap>(hd, p.q_kind, p.pairs, p.q_width, p.q_swap, turns, on, ready);
  if (!keys) return;
  // the tokens' latent rows and rope parts, a warp each
  const int half = p.k_kind.rot / 2;
  for (int x = nw - 1 - warp; x < 2 * nt; x += nw) {
    const int i = x >> 1;
    const int64_t row = rows[i];
    if (row < 0) continue;
    const bool latent = (x & 1) == 0;
    const Kind& k = latent ? p.c_kind : p.k_kind;
    const T* src = (const T*)p.kv + (t0 + i) * p.kv_token + (latent ? 0 : p.c_kind.n);
    T* dst = latent ? (T*)p.c_kv + row * p.ckv_row : (T*)p.k_pe + row * p.kpe_row;
    const T* w = (const T*)(latent ? p.kv_w : p.k_w);
    const Turns<T>* tt = turns_of<T>(turns, i, half);
    if (latent ? p.c_vec : p.k_vec) {
      Held<T, kMaxVecs, false> held;
      held.load(src, k, p.pairs, true, lane, 32);
      held.finish(dst, dst, k, p.pairs, 0, w, true, lane, 32, tt);
    } else {
      one_by_one<T>(src, dst, dst, w, k, p.pairs, tt, lane);
    }
  }
}

template <typename T>
bool fits(const void* p) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0;
}

// Lanes that hold a head of a kind (a power of two) and their vectors, with as few lanes idle as
// up to `vecs` vectors a lane allow, fewer vectors first; 0: it has to go one by one.
template <typename T>
int lanes_for(const Kind& k, bool pairs, int vecs, int* per_lane) {
  constexpr int N = Vec16<T>::N;
  const int part = pairs ? k.rot : k.rot / 2, n = k.n / N;
  *per_lane = 1;
  if (k.n % N || k.split % N || k.at % N || part % N) return 0;
  int best = 0, waste = 1 << 30;
  for (int v = 1; v <= vecs; ++v)
    for (int w = 1; w <= 32; w *= 2)
      if (w * v >= n && w * v - n < waste) {
        waste = w * v - n;
        best = w;
        *per_lane = v;
      }
  return best;
}

// How many lanes away the partners of a rotated part are, if one exchange of lanes brings them (1
// where they are in the lane's own vector), else 0: the part lies in one of a lane's vectors, at a
// multiple of its size, a power of two.
template <typename T>
int swap_lanes(const Kind& k, bool pairs, int width) {
  constexpr int N = Vec16<T>::N;
  if (sizeof(T) == 4 || width == 0) return 0;
  if (pairs) return 1;
  const int at = k.at / N, n = k.rot / N;
  if ((n & (n - 1)) || at % n || at / width != (at + n - 1) / width) return 0;
  return n / 2;
}

// Tokens and heads per block, and threads.  `fit` blocks of 256 threads fit an SM: a block takes as
// many tokens as fill the GPU once (eight at most), and where the tokens are fewer than two per SM
// their heads go to several blocks.
struct Grid {
  int tokens, per_block, groups, threads;
};
Grid grid_for(int64_t tokens, int heads, int per_warp, int turn_bytes, int fit) {
  const int64_t sms = current_sm_count();
  Grid s;
  const int room = std::max(1, 16384 / turn_bytes);  // 16 KB of turns
  s.tokens = (int)std::min<int64_t>(std::min(kMaxTokens, room), (tokens + fit * sms - 1) / (fit * sms));
  const int64_t want = 2 * sms;
  const int groups =
      tokens >= want ? 1 : (int)std::min<int64_t>(std::max(heads, 1), (want + tokens - 1) / tokens);
  s.per_block = std::max(1, (heads + groups - 1) / groups);
  s.groups = std::max(1, (heads + s.per_block - 1) / s.per_block);
  const int warps = (s.per_block * s.tokens + per_warp - 1) / per_warp;
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
  p.kind = {a->d_head, a->rot_offset, a->rot_dim, a->d_head, 0.f, 0.f};
  const bool in_place = a->in == a->out;
  if (in_place) {  // the elements outside the rotated part are there already
    p.in = (const T*)a->in + a->rot_offset;
    p.out = (T*)a->out + a->rot_offset;
    p.kind = {a->rot_dim, 0, a->rot_dim, a->rot_dim, 0.f, 0.f};
  }
  p.pairs = a->layout == TV_ROPE_INTERLEAVED;
  int vecs = 1;
  p.width = lanes_for<T>(p.kind, p.pairs, kMaxVecs, &vecs);
  if (!(fits<T>(p.in) && fits<T>(p.out) && p.in_token % N == 0 && p.in_head % N == 0 &&
        p.out_token % N == 0 && p.out_head % N == 0))
    p.width = 0;
  p.swap = swap_lanes<T>(p.kind, p.pairs, p.width);
  p.T = a->T;
  p.positions = a->positions;
  p.sign = a->inverse ? -1.0 : 1.0;
  const InvFreq& inv = table_of(a->scaling, a->rot_dim, &p.mag);
  const Grid s = grid_for(a->T, a->n_heads, p.width ? 32 / p.width : 1, (int)Turns<T>::bytes(a->rot_dim / 2), 4);
  p.per_block = s.per_block;
  p.tokens = s.tokens;
  const dim3 grid((unsigned)(((int64_t)a->T + s.tokens - 1) / s.tokens), (unsigned)s.groups);
  const size_t smem = Turns<T>::bytes(a->rot_dim / 2) * s.tokens;
  auto go = [&](auto kernel) { return start(kernel, grid, s.threads, smem, st, p, inv); };
  if constexpr (sizeof(T) == 2)
    if (p.swap > 0)
      return vecs == 1   ? go(rope_kernel<T, 1, true>)
             : vecs == 2 ? go(rope_kernel<T, 2, true>)
             : vecs == 3 ? go(rope_kernel<T, 3, true>)
                         : go(rope_kernel<T, 4, true>);
  return vecs == 1   ? go(rope_kernel<T, 1, false>)
         : vecs == 2 ? go(rope_kernel<T, 2, false>)
         : vecs == 3 ? go(rope_kernel<T, 3, false>)
                     : go(rope_kernel<T, 4, false>);
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
  p.q_kind = {a->d_nope + a->d_rope, a->d_nope, a->rot_dim, a->d_nope, a->eps, 1.f / (float)(a->d_nope + a->d_rope)};
  p.c_kind = {a->d_latent, 0, 0, a->d_latent, a->eps, 1.f / (float)a->d_latent};
  p.k_kind = {a->d_rope, 0, a->rot_dim, a->d_rope, a->eps, 1.f / (float)a->d_rope};
  p.pairs = a->layout == TV_ROPE_INTERLEAVED;
  int vecs = 1, kv_vecs;
  p.q_width = a->q ? lanes_for<T>(p.q_kind, p.pairs, kMaxVecs, &vecs) : 0;
  if (!(fits<T>(a->q) && fits<T>(a->q_nope) && fits<T>(a->q_pe) && fits<T>(a->q_weight) &&
        p.q_token % N == 0 && p.q_head % N == 0))
    p.q_width = 0;
  p.q_swap = swap_lanes<T>(p.q_kind, p.pairs, p.q_width);
  const bool kv_ok = fits<T>(a->kv) && p.kv_token % N == 0 && a->d_latent % N == 0;
  p.c_vec = lanes_for<T>(p.c_kind, true, kMaxVecs, &kv_vecs) && kv_ok && fits<T>(a->c_kv) &&
            p.ckv_row % N == 0 && fits<T>(a->kv_weight);
  p.k_vec = lanes_for<T>(p.k_kind, p.pairs, kMaxVecs, &kv_vecs) && kv_ok && fits<T>(a->k_pe) &&
            p.kpe_row % N == 0 && fits<T>(a->k_weight);
  p.cache = {a->cache.page_table, a->cache.page_size, a->cache.max_pages, a->cache.kv_stride_b};
  p.num_rows = a->cache.num_rows;
  p.q_start = a->q_start;
  p.prefix_len = a->prefix_len;
  p.depth = a->depth;
  p.status = a->status;
  const InvFreq& inv = table_of(a->scaling, a->rot_dim, &p.mag);
  const Grid s = grid_for(a->T, p.H, p.q_width ? 32 / p.q_width : 1, (int)Turns<T>::bytes(a->rot_dim / 2), 3);
  p.per_block = s.per_block;
  p.tokens = s.tokens;
  const dim3 grid((unsigned)(((int64_t)a->T + s.tokens - 1) / s.tokens), (unsigned)s.groups);
  const size_t smem = Turns<T>::bytes(a->rot_dim / 2) * s.tokens;
  auto go = [&](auto kernel) { return start(kernel, grid, s.threads, smem, st, p, inv); };
  if constexpr (sizeof(T) == 2)
    if (p.q_swap > 0)
      return vecs == 1   ? go(norm_rope_kernel<T, 1, true>)
             : vecs == 2 ? go(norm_rope_kernel<T, 2, true>)
             : vecs == 3 ? go(norm_rope_kernel<T, 3, true>)
                         : go(norm_rope_kernel<T, 4, true>);
  return vecs == 1   ? go(norm_rope_kernel<T, 1, false>)
         : vecs == 2 ? go(norm_rope_kernel<T, 2, false>)
         : vecs == 3 ? go(norm_rope_kernel<T, 3, false>)
                     : go(norm_rope_kernel<T, 4, false>);
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
