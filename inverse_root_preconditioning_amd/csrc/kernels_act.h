// Activations y = f(a) and gated activations y = f(a) b with their gradients,
// elementwise over matrices, the inputs optionally kept as MX8 rows.
#pragma once

#include "kernels_mx8.h"

namespace shp {

// exp(-v) = e unit for 0 <= v <= 120.  FINE: to about an ulp, v (given in two floats)
// times log2(e) in two floats, so that the error of a large exponent does not
// reach the result.  Else within 2^-15: v's own rounding and that of the
// product, up to 300 ulps where v is large, which a bf16 result (half a step: 2^-9) does not show.
// The instruction has no subnormal results: e is 0 below 2^-126, but for FAR, where unit is 2^-64 for large v and e
// a normal number, so that what it is multiplied by is not lost.
template <bool FINE, bool FAR>
__device__ __forceinline__ float exp_minus(float v, float v_low, float& unit) {
#pragma clang fp contract(off)
  constexpr float kHi = 1.44269504088896341f, kLo = 1.9259629911e-8f;  // log2(e) and what fp32 leaves of it
  const float t = -v * kHi;  // rounded by itself, so that `low` is what it lacks
  const bool far = FAR && v > 80.f;  // t below -115, so that t + 64 is exact
  unit = far ? 0x1p-64f : 1.f;
  const float e = __builtin_amdgcn_exp2f(far ? t + 64.f : t);
  if constexpr (!FINE) return e;
  const float low = __builtin_fmaf(-v_low, kHi, __builtin_fmaf(-v, kLo, __builtin_fmaf(-v, kHi, -t)));
  return __builtin_fmaf(e, low * 0.693147180559945309f, e);
}

// x within +-limit; a NaN stays one.
__device__ __forceinline__ float clamp_abs(float x, float limit) {
  x = x > limit ? limit : x;
  return x < -limit ? -limit : x;
}

// Magnitudes up to which every factor of f and f' is a normal number.  v is at most 80 there, so that such values'
// results are the same bits in either form, whatever stands beside them.
template <int ACT>
constexpr float kNear = ACT == SHAMPOO_ACT_SILU ? 80.f : ACT == SHAMPOO_ACT_GELU ? 12.5f : 9.5f;

// f(x) and, with SLOPE, f'(x); FINE for fp32 results (see exp_minus), FAR where x may lie beyond kNear and its result
// is to keep its relative precision down to 2^-126; without it the tails end with the exponential, at
// results of some 2^-119.  Beyond the clamps f is 0 or x and f' 0 or 1 to the last bit, and no intermediate
// result overflows into a NaN for any finite x.  (-infinity: f = -infinity 0, a NaN, but for the relus; f' = 0.)
template <int ACT, bool SLOPE, bool FINE, bool FAR>
__device__ __forceinline__ void activation(float x, float& f, float& d) {
  if constexpr (ACT == SHAMPOO_ACT_RELU) {
    f = x < 0.f ? 0.f : x;
    if (SLOPE) d = x > 0.f ? 1.f : x <= 0.f ? 0.f : x;  // NaN stays: a kept group of NaN is no row of zeros
  } else if constexpr (ACT == SHAMPOO_ACT_RELU2) {
    const float r = x < 0.f ? 0.f : x;
    f = r * r;
    if (SLOPE) d = 2.f * r;
  } else if constexpr (ACT == SHAMPOO_ACT_GELU) {
    // x Phi(x), with Phi(-z) = exp(-z^2/2) t Q(t), t = 1 / (1 + 0.225 z): Q is
    // the polynomial of degree 10 nearest to erfcx(z / sqrt 2) / (2 t) on all of
    // z >= 0 (relative 1.0e-8; reweighted least squares at 400 Chebyshev
    // points of t).  The tail keeps its relative precision, which 1 + erf loses.
    const float c = clamp_abs(x, 15.f), z = fabsf(c);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.225f, z, 1.f));
    float q = 0.016711030155420303f;
    q = __builtin_fmaf(q, t, -0.07665678858757019f);
    q = __builtin_fmaf(q, t, 0.11226222664117813f);
    q = __builtin_fmaf(q, t, -0.0657426118850708f);
    q = __builtin_fmaf(q, t, 0.07158230245113373f);
    q = __builtin_fmaf(q, t, 0.03579634428024292f);
    q = __builtin_fmaf(q, t, 0.06539952754974365f);
    q = __builtin_fmaf(q, t, 0.07589364796876907f);
    q = __builtin_fmaf(q, t, 0.08523055911064148f);
    q = __builtin_fmaf(q, t, 0.08976174890995026f);
    q = __builtin_fmaf(q, t, 0.08976201713085175f);
    const float h = 0.5f * z, s = h * z;
    float unit;
    const float e = exp_minus<FINE, FAR>(s, __builtin_fmaf(h, z, -s), unit);
    float a = e, last = 1.f;
    if constexpr (FAR) {  // a negative x takes e as it is and the unit last
      a = x < 0.f ? (x < -15.f ? 0.f : e) : e * unit;
      last = x < 0.f ? unit : 1.f;
    }
    const float tail = a * (q * t);
    const float p = x < 0.f ? tail : 1.f - tail;
    f = x * p;
    if (SLOPE) d = __builtin_fmaf(c * a, 0.398942280401432678f, p);
    if constexpr (FAR) {
      f *= last;
      if (SLOPE) d *= last;
    }
  } else {
    // x p with p = 1 / (1 + exp(-v)): v = x, or 2 sqrt(2/pi) (x + 0.044715 x^3)
    constexpr bool kTanh = ACT == SHAMPOO_ACT_GELU_TANH;
    constexpr float kA = 1.59576912160573071f, kALow = -4.534068054e-8f, kB = 0.044715f, kBLow = 1.546144435e-9f;
    constexpr float kLimit = kTanh ? 11.f : 111.f;  // v at most 113 and 111: x exp(-v) is 0 in fp32 from 109 on
    const float c = clamp_abs(x, kLimit);
    float v, v_low = 0.f;
    if constexpr (kTanh && FINE) {
#pragma clang fp contract(off)
      // A c (1 + B c^2) in two floats: every product's error by a fused one, the sum's by its own terms
      const float q = c * c, q_low = __builtin_fmaf(c, c, -q);
      const float m = kB * q, m_low = __builtin_fmaf(kB, q, -m) + __builtin_fmaf(kB, q_low, kBLow * q);
      const float w = 1.f + m, back = w - 1.f;
      const float w_low = (1.f - (w - back)) + (m - back) + m_low;
      const float u = kA * c, u_low = __builtin_fmaf(kA, c, -u) + kALow * c;
      v = u * w;
      v_low = __builtin_fmaf(u, w, -v) + __builtin_fmaf(u, w_low, u_low * w);
      v_low = v < 0.f ? -v_low : v_low;
    } else {
      v = kTanh ? kA * __builtin_fmaf(kB * c, c * c, c) : c;
    }
    float unit;
    const float e = exp_minus<FINE, FAR>(fabsf(v), v_low, unit);
    const float r = __builtin_amdgcn_rcpf(1.f + (FAR ? e * unit : e));
    float a = e, last = 1.f;
    if constexpr (FAR) {  // a negative x takes e as it is and the unit last
      a = x < 0.f ? (x < -kLimit ? 0.f : e) : e * unit;
      last = x < 0.f ? unit : 1.f;
    }
    const float er = a * r;
    const float p = x < 0.f ? er : r;
    f = x * p;
    if (SLOPE) {
      const float slope = kTanh ? kA * __builtin_fmaf(3.f * kB, c * c, 1.f) : 1.f;
      d = __builtin_fmaf(c * slope, er * r, p);
    }
    if constexpr (FAR) {
      f *= last;
      if (SLOPE) d *= last;
    }
  }
}

// each(far): a lane's V values x, in the form for far values where results are fp32 and the wave has one.  Taken
// always it cost 4 to 6% (silu of 4096 x 8192 39 -> 41 us).
template <int ACT, bool FINE, int V, class X, class F>
__device__ __forceinline__ void near_or_far(X&& x, F&& each) {
  if constexpr (FINE && ACT != SHAMPOO_ACT_RELU && ACT != SHAMPOO_ACT_RELU2) {
    bool far = false;
#pragma unroll
    for (int e = 0; e < V; ++e) far |= fabsf(x(e)) > kNear<ACT>;
    if (__builtin_expect(__any(far), 0)) {
      each(std::true_type{});
      return;
    }
  }
  each(std::false_type{});
}

struct ActArgs {
  const void *a, *b, *dy;
  void *y, *da, *db;
  int64_t lda, ldb, lddy, ldy, ldda, lddb;
  int64_t rows;
  uint32_t cols;
  Mx8Rows ka, kb;  // kept inputs
  RowShape shape;
};

// Elementwise, in the pieces and with the grid of the MX8 conversion; the kept copies are
// made from the same registers, so that an input is read once, and backward
// reads only dy and codes.  Bound by HBM: gated silu of 8192 x 8192 bf16, inputs kept in 8 bits,
// 100 us forward (5.5 TB/s) and 102 backward (5.3); stores through the caches 217 us for both.  Ungated, forward and
// backward, of 8192 x 8192 bf16: relu 39, 59; silu 42, 60; gelu_tanh 46, 66; and gelu 53 to 67, 70 to 79, whose vector
// instructions fill a third of their slots, some at a quarter of the rate.
constexpr int kActPasses = 4;

template <bool BF16, int ACT, bool GATED, bool KEEP>
__global__ void __launch_bounds__(256) act_forward_kernel(const ActArgs P) {
  constexpr int V = BF16 ? 8 : 4;
  const uint32_t rb = blockIdx.x / P.shape.col_blocks, cb = blockIdx.x - rb * P.shape.col_blocks;
  const int lanes = 1 << P.shape.lanes_log2, per_pass = 256 >> P.shape.lanes_log2;
  const uint32_t col = (cb * lanes + (threadIdx.x & (lanes - 1))) * V;
  const int64_t row0 = (int64_t)rb * kActPasses * per_pass + (threadIdx.x >> P.shape.lanes_log2);
  Piece<BF16, V> a[kActPasses], b[kActPasses];
#pragma unroll
  for (int i = 0; i < kActPasses; ++i) {
    const int64_t r = min(row0 + i * per_pass, P.rows - 1);
    a[i] = load_row<BF16, V>(row_at<BF16>(P.a, r, P.lda), P.cols, col);
    if constexpr (GATED) b[i] = load_row<BF16, V>(row_at<BF16>(P.b, r, P.ldb), P.cols, col);
  }
#pragma unroll
  for (int i = 0; i < kActPasses; ++i) {
    const int64_t r = row0 + i * per_pass;
    if constexpr (KEEP) {
      Mx8Piece<V> q;
      q.encode(a[i]);
      if (r < P.rows) q.store(P.ka, r, col);
      if constexpr (GATED) {
        q.encode(b[i]);
        if (r < P.rows) q.store(P.kb, r, col);
      }
    }
    if (r < P.rows) {
      float y[V], unused = 0.f;
      near_or_far<ACT, !BF16, V>([&](int e) { return elem(a[i], e); }, [&](auto far) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          activation<ACT, false, !BF16, decltype(far)::value>(elem(a[i], e), y[e], unused);
          if constexpr (GATED) y[e] *= elem(b[i], e);
        }
      });
      store_row<BF16, V>(row_at<BF16>(P.y, r, P.ldy), P.cols, col, y);
    }
  }
}

template <bool BF16, int ACT, bool GATED, bool KEEP>
__global__ void __launch_bounds__(256) act_backward_kernel(const ActArgs P) {
  constexpr int V = BF16 ? 8 : 4;
  const uint32_t rb = blockIdx.x / P.shape.col_blocks, cb = blockIdx.x - rb * P.shape.col_blocks;
  const int lanes = 1 << P.shape.lanes_log2, per_pass = 256 >> P.shape.lanes_log2;
  const uint32_t col = (cb * lanes + (threadIdx.x & (lanes - 1))) * V;
  const int64_t row0 = (int64_t)rb * kActPasses * per_pass + (threadIdx.x >> P.shape.lanes_log2);
  if (col >= P.cols) return;
  Piece<BF16, V> dy[kActPasses], a[kActPasses], b[kActPasses];
  Mx8Piece<V> qa[kActPasses], qb[kActPasses];
#pragma unroll
  for (int i = 0; i < kActPasses; ++i) {
    const int64_t r = min(row0 + i * per_pass, P.rows - 1);
    dy[i] = load_row<BF16, V>(row_at<BF16>(P.dy, r, P.lddy), P.cols, col);
    if constexpr (KEEP) {
      qa[i].load(P.ka, r, col);
      if constexpr (GATED) qb[i].load(P.kb, r, col);
    } else {
      a[i] = load_row<BF16, V>(row_at<BF16>(P.a, r, P.lda), P.cols, col);
      if constexpr (GATED) b[i] = load_row<BF16, V>(row_at<BF16>(P.b, r, P.ldb), P.cols, col);
    }
  }
#pragma unroll
  for (int i = 0; i < kActPasses; ++i) {
    const int64_t r = row0 + i * per_pass;
    if (r >= P.rows) return;
    float av[V], bv[V], da[V], db[V];
    if constexpr (KEEP) {
      qa[i].decode(av);
      if constexpr (GATED) qb[i].decode(bv);
    }
    auto x = [&](int e) { return KEEP ? av[e] : elem(a[i], e); };
    near_or_far<ACT, !BF16, V>(x, [&](auto far) __attribute__((always_inline)) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if constexpr (!KEEP) {
          av[e] = elem(a[i], e);
          if constexpr (GATED) bv[e] = elem(b[i], e);
        }
        float f, d;
        activation<ACT, true, !BF16, decltype(far)::value>(av[e], f, d);
        const float g = elem(dy[i], e);
        da[e] = g * d;
        if constexpr (GATED) {
          da[e] *= bv[e];
          db[e] = g * f;
        }
      }
    });
    if (P.da != nullptr) store_row<BF16, V>(row_at<BF16>(P.da, r, P.ldda), P.cols, col, da);
    if constexpr (GATED) {
      if (P.db != nullptr) store_row<BF16, V>(row_at<BF16>(P.db, r, P.lddb), P.cols, col, db);
    }
  }
}

}  // namespace shp
