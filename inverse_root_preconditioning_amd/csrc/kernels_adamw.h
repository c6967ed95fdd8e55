// AdamW over many tensors and the norm of many tensors: HBM-bound kernels that
// walk a list of 2048-element segments.
#pragma once

#include "vector_io.h"

namespace shp {

constexpr int kGroup = SHAMPOO_GROUP;
constexpr int kSegment = SHAMPOO_SEGMENT;

// ---------------------------------------------------------------------------
// The hash behind the stochastic rounding: two rounds of xor-shift and
// multiplication by odd constants over a counter, so that every state-buffer
// position of every (seed, step) has its own 32 bits.
// ---------------------------------------------------------------------------
constexpr uint32_t kHashC1 = 0x2F6B4D1Du, kHashC2 = 0x5A3C91E7u, kHashC3 = 0x6D41B7A5u, kHashC4 = 0x3B9F0D4Bu;

__host__ __device__ __forceinline__ uint32_t hash_finish(uint32_t x) {
  x = (x ^ (x >> 16)) * kHashC2;
  x = (x ^ (x >> 15)) * kHashC3;
  return x ^ (x >> 16);
}

// ---------------------------------------------------------------------------
// 8-bit moments.  A float times 2^-kDown has the code in its bits 20 to 27 (the
// codes' subnormals are the float's), so rounding is an integer addition
// below bit 20 and a shift; the 16 random bits are centred in their 20-bit
// range, which leaves representable values alone.
// ---------------------------------------------------------------------------
struct MomentM {  // sign, E4M3 of bias 7
  static constexpr int kBack = 7, kDown = 120;
  static constexpr uint32_t kMask = 127;
};
struct MomentV {  // unsigned E5M3 of bias 15
  static constexpr int kBack = 15, kDown = 112;
  static constexpr uint32_t kMask = 255;
};

// 2^(e - 127) for 1 <= e <= 254.
__host__ __device__ __forceinline__ float pow2_field(int e) { return __builtin_bit_cast(float, (uint32_t)e << 23); }

// Scale byte of a group from the bits of its largest magnitude.
template <class F>
__device__ __forceinline__ int mx8_scale(uint32_t top_bits) {
  const int e = (int)(top_bits >> 23);
  return e == 255 ? 255 : max(e - F::kBack, 1);
}

template <class F>
__device__ __forceinline__ uint32_t mx8_encode(float x, int s, uint32_t rnd16) {
  const float up = s == 255 ? 0.f : pow2_field(254 - s);
  const float t = (fabsf(x) * up) * pow2_field(127 - F::kDown);
  uint32_t code = (__builtin_bit_cast(uint32_t, t) + (rnd16 << 4) + 8u) >> 20;
  if (F::kMask == 127) {
    code |= x < 0.f ? 128u : 0u;
  } else {
    code = max(code, 1u);
  }
  return s == 255 ? 0u : code;
}

template <class F>
__device__ __forceinline__ float mx8_decode(uint32_t code, int s) {
  float v = __builtin_bit_cast(float, (code & F::kMask) << 20) * pow2_field(127 + F::kDown);
  if (F::kMask == 127 && code >= 128) v = -v;
  return v * (s == 255 ? __builtin_nanf("") : pow2_field(s));  // s >= 1; 0 stands only beside codes of 0
}

// V consecutive elements of a tensor as floats (WHOLE: all of them; else those
// below `left`, the others 0), at any element's address.
template <bool BF16, int V, bool WHOLE>
__device__ __forceinline__ void load_elems(const void* p, int64_t at, int left, float (&x)[V]) {
  if constexpr (!WHOLE) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      x[e] = 0.f;
      if (e < left) {
        if constexpr (BF16) {
          x[e] = __builtin_bit_cast(float, (uint32_t)ldg(static_cast<const uint16_t*>(p) + at + e) << 16);
        } else {
          x[e] = ldg(static_cast<const float*>(p) + at + e);
        }
      }
    }
  } else if constexpr (BF16) {
    typedef uint32_t Words __attribute__((ext_vector_type(V / 2)));
    const Words w = ldg_once<Words, 2>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
    for (int e = 0; e < V; ++e)
      x[e] = __builtin_bit_cast(float, (e & 1) ? (w[e / 2] & 0xffff0000u) : (w[e / 2] << 16));
  } else {
#pragma unroll
    for (int q = 0; q < V / 4; ++q) {
      const floatx4 w = ldg_once<floatx4, 4>(static_cast<const float*>(p) + at + 4 * q);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[4 * q + e] = w[e];
    }
  }
}

template <int V, bool WHOLE>
__device__ __forceinline__ void store_f32(void* p, int64_t at, int left, const float (&x)[V]) {
  float* const o = static_cast<float*>(p) + at;
  if constexpr (WHOLE) {
#pragma unroll
    for (int q = 0; q < V / 4; ++q)
      stg_once<floatx4, 4>(o + 4 * q, floatx4{x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]});
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (e < left) stg(o + e, x[e]);
  }
}

// Bits of V bf16 values, two a word.
template <int V, bool WHOLE>
__device__ __forceinline__ void store_bf16(void* p, int64_t at, int left, const uint32_t (&w)[V / 2]) {
  typedef uint32_t Words __attribute__((ext_vector_type(V / 2)));
  uint16_t* const o = static_cast<uint16_t*>(p) + at;
  if constexpr (WHOLE) {
    Words x;
#pragma unroll
    for (int e = 0; e < V / 2; ++e) x[e] = w[e];
    stg_once<Words, 2>(o, x);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (e < left) stg(o + e, (uint16_t)(w[e / 2] >> (16 * (e & 1))));
  }
}

struct AdamwArgs {
  const shampoo_tensor *params, *grads, *copies;
  const float* hyper;
  const shampoo_segment* segments;
  int64_t ntensors;
  void *m, *v;
  uint8_t *m_scale, *v_scale;
  const float* grad_scale;
  double omb1, omb2;                             // 1 - beta
  float lr, beta1, beta2, eps, rbc1, rsbc2;      // rbc1 = 1 / (1 - beta1^t), rsbc2 = 1 / sqrt(1 - beta2^t)
  uint32_t key;
};

// One workgroup a segment (of 2048: 4096 are 1 to 5% slower on large sets and 14%
// on 2700 of them, whose last workgroups then leave the GPU half empty),
// everything read and written once and past the caches.  A lane takes 4
// consecutive elements, or 8 where all but the 8-bit moments are bf16 (16 bytes
// either way: 8 floats a lane would read half cache lines).  The square root
// and the reciprocal are the hardware's (1 ulp): they reach the parameter only,
// far below its rounding.  The root takes a subnormal v for 0: with TINY, for an
// eps that does not cover that, it is taken of v 2^64 (done for every eps that
// costs bf16 with 8-bit moments 5%).
//
// HBM-bound.  302e6 parameters: fp32 throughout 1.48 ms (5.7 TB/s, the rate of a
// large copy; 1.58 ms through the caches), bf16 with 8-bit moments 0.52 ms
// (5.9 TB/s; 5% more with 4 elements a lane).
template <bool PARAM_BF16, bool GRAD_BF16, bool MX8, bool COPY, bool TINY>
__global__ void __launch_bounds__(256) adamw_kernel(const AdamwArgs P) {
// Which operations are fused is written out: the codes that the moments round
// to must not depend on the compiler's choice.
#pragma clang fp contract(off)
    constexpr int V = MX8 && PARAM_BF16 && GRAD_BF16 ? 8 : 4, kRounds = kSegment / (256 * V);
  constexpr int kLanes = kGroup / V;
  typedef uint32_t Codes __attribute__((ext_vector_type(V / 4)));
  const shampoo_segment seg = P.segments[blockIdx.x];
  if ((uint64_t)seg.tensor >= (uint64_t)P.ntensors || seg.index < 0) return;
  float c = 1.f;
  if (P.grad_scale != nullptr) {
    c = *P.grad_scale;
    if (!(fabsf(c) <= FLT_MAX)) return;
  }
  const shampoo_tensor tp = P.params[seg.tensor], tg = P.grads[seg.tensor];
  void* const copy = COPY ? P.copies[seg.tensor].ptr : nullptr;
  const int64_t first = (int64_t)seg.index * kSegment, pos0 = tp.offset + first;
  const int len = (int)min((int64_t)kSegment, min(tp.n, tg.n) - first);
  const float eta = P.lr * P.hyper[2 * seg.tensor], keep = 1.f - eta * P.hyper[2 * seg.tensor + 1];
  // The scale c goes into the constants (in double) where that cannot overflow:
  // g c g k2 keeps v finite for a huge g with a small c, and takes four roundings at most.
  const float step = eta * P.rbc1, k1 = (float)(P.omb1 * c), k2 = (float)(P.omb2 * c);

  auto rounds = [&](auto WHOLE) __attribute__((always_inline)) {
    constexpr bool kWhole = decltype(WHOLE)::value;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const int i = (r * 256 + (int)threadIdx.x) * V, left = len - i;
      const int64_t at = first + i, pos = pos0 + i, grp = pos / kGroup;
      float p[V], g[V], m[V], v[V];
      load_elems<PARAM_BF16, V, kWhole>(tp.ptr, at, left, p);
      load_elems<GRAD_BF16, V, kWhole>(tg.ptr, at, left, g);
      if constexpr (MX8) {
        // The state buffers are padded to whole groups, so that whole vectors
        // are there wherever a tensor has elements.
        Codes mc = 0, vc = 0;
        int ms = 1, vs = 1;
        if (kWhole || left > 0) {
          mc = ldg_once<Codes, V>(static_cast<const uint8_t*>(P.m) + pos);
          vc = ldg_once<Codes, V>(static_cast<const uint8_t*>(P.v) + pos);
          ms = ldg(P.m_scale + grp);
          vs = ldg(P.v_scale + grp);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          m[e] = mx8_decode<MomentM>((mc[e / 4] >> (8 * (e % 4))) & 255u, ms);
          v[e] = mx8_decode<MomentV>((vc[e / 4] >> (8 * (e % 4))) & 255u, vs);
          if (!kWhole && e >= left) m[e] = v[e] = 0.f;
        }
      } else {
        load_elems<false, V, kWhole>(P.m, pos, left, m);
        load_elems<false, V, kWhole>(P.v, pos, left, v);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        m[e] = __builtin_fmaf(g[e], k1, P.beta1 * m[e]);
        v[e] = __builtin_fmaf(g[e] * c, g[e] * k2, P.beta2 * v[e]);
      }
      uint32_t h[V];
      if constexpr (MX8 || PARAM_BF16) {
        // V consecutive positions share their upper 32 bits
        const uint32_t x = (uint32_t)pos * kHashC1 + (uint32_t)((uint64_t)pos >> 32) * kHashC4 + P.key;
#pragma unroll
        for (int e = 0; e < V; ++e) h[e] = hash_finish(x + (uint32_t)e * kHashC1);
      }
      if constexpr (MX8) {
        uint32_t mt = 0, vt = 0;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          mt = max(mt, __builtin_bit_cast(uint32_t, m[e]) & 0x7fffffffu);
          vt = max(vt, __builtin_bit_cast(uint32_t, v[e]) & 0x7fffffffu);
        }
        const int ms = mx8_scale<MomentM>(group_max<kLanes>(mt)), vs = mx8_scale<MomentV>(group_max<kLanes>(vt));
        Codes mc = 0, vc = 0;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const uint32_t a = mx8_encode<MomentM>(m[e], ms, h[e] & 0xffffu), b = mx8_encode<MomentV>(v[e], vs, h[e] >> 16);
          if (kWhole || e < left) {  // the padding stays 0
            mc[e / 4] |= a << (8 * (e % 4));
            vc[e / 4] |= b << (8 * (e % 4));
          }
        }
        if (kWhole || left > 0) {
          stg_once<Codes, V>(static_cast<uint8_t*>(P.m) + pos, mc);
          stg_once<Codes, V>(static_cast<uint8_t*>(P.v) + pos, vc);
          if (threadIdx.x % kLanes == 0) {
            stg(P.m_scale + grp, (uint8_t)ms);
            stg(P.v_scale + grp, (uint8_t)vs);
          }
        }
      } else {
        store_f32<V, kWhole>(P.m, pos, left, m);
        store_f32<V, kWhole>(P.v, pos, left, v);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float root = TINY && v[e] < FLT_MIN ? __builtin_amdgcn_sqrtf(v[e] * 0x1p64f) * 0x1p-32f
                                                  : __builtin_amdgcn_sqrtf(v[e]);
        const float d = m[e] * __builtin_amdgcn_rcpf(__builtin_fmaf(root, P.rsbc2, P.eps));
        p[e] = __builtin_fmaf(-step, d, p[e] * keep);
      }
      if constexpr (PARAM_BF16) {
        uint32_t w[V / 2];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const uint32_t b = (__builtin_bit_cast(uint32_t, p[e]) + ((h[e] * kHashC2) >> 16)) >> 16;
          const uint32_t q = p[e] != p[e] ? 0x7fc0u : b;
          w[e / 2] = (e & 1) ? w[e / 2] | (q << 16) : q;
        }
        store_bf16<V, kWhole>(tp.ptr, at, left, w);
      } else {
        store_f32<V, kWhole>(tp.ptr, at, left, p);
        if constexpr (COPY) {
          uint32_t w[V / 2];
#pragma unroll
          for (int e = 0; e < V / 2; ++e) w[e] = pack_bf16x2(p[2 * e], p[2 * e + 1]);
          store_bf16<V, kWhole>(copy, at, left, w);
        }
      }
    }
  };
  if (len == kSegment) {
    rounds(std::true_type{});
  } else {
    rounds(std::false_type{});
  }
}

struct MomentsArgs {
  const uint8_t *codes[2], *scales[2];  // m, v
  void* out[2];
  int64_t n;
  int first;  // 0: blockIdx.y = 0 is m; 1: only v
};

// 8 codes a lane; m and v in one launch.  5.9 TB/s to bf16.
template <bool BF16>
__global__ void __launch_bounds__(256) mx8_decode_kernel(const MomentsArgs P) {
  const bool is_v = P.first + (int)blockIdx.y != 0;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (i >= P.n) return;
  const uint8_t* const codes = is_v ? P.codes[1] : P.codes[0];
  const uint8_t* const scales = is_v ? P.scales[1] : P.scales[0];
  void* const out = is_v ? P.out[1] : P.out[0];
  const u32x2 c = ldg_once<u32x2, 1>(codes + i);
  const int s = ldg(scales + i / kGroup);
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t code = (c[e / 4] >> (8 * (e % 4))) & 255u;
    x[e] = is_v ? mx8_decode<MomentV>(code, s) : mx8_decode<MomentM>(code, s);
  }
  if constexpr (BF16) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(x[2 * e], x[2 * e + 1]);
    store_bf16<8, true>(out, i, 8, w);
  } else {
    store_f32<8, true>(out, i, 8, x);
  }
}

// ---------------------------------------------------------------------------
// Norm.  Pass 1: each workgroup (1024 of them; 8192 are 6% slower) sums the
// squares of a contiguous run of segments in double (a product of two floats
// is exact there, and no fp32 gradient overflows it); pass 2: one workgroup
// adds the partial sums.  Both in a fixed order.  1.2e9 bf16 values take
// 0.37 ms (6.5 TB/s, reads alone).
// ---------------------------------------------------------------------------
template <int kThreads>
__device__ __forceinline__ double block_sum_f64(double v, double* red) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
  if ((threadIdx.x % kWave) == 0) red[threadIdx.x / kWave] = v;
  __syncthreads();
  double t = 0.;
#pragma unroll
  for (int i = 0; i < kThreads / kWave; ++i) t += red[i];
  __syncthreads();
  return t;
}

// out: the norm, and the factor that brings it down to max_norm.
__device__ __forceinline__ void store_norm(double sum, float max_norm, float* out) {
  const double norm = sqrt(sum);
  const float f = (float)norm;
  float coef = norm > max_norm ? (float)(max_norm / norm) : 1.f;
  if (!(f <= FLT_MAX)) coef = __builtin_nanf("");
  stg(out, f);
  stg(out + 1, coef);
}

template <bool BF16>
__global__ void __launch_bounds__(256) grad_norm_partial_kernel(const shampoo_tensor* tensors,
                                                                const shampoo_segment* segments, int64_t nseg,
                                                                double* partial) {
  __shared__ double red[4];
  // kSegs segments at a time: 16 bytes a lane twice, whatever the type
  constexpr int V = BF16 ? 8 : 4, kRounds = kSegment / (256 * V), kSegs = 2 / kRounds;
  static_assert(kSegs * kRounds == 2, "two loads a lane");
  const int64_t s0 = nseg * blockIdx.x / gridDim.x, s1 = nseg * (blockIdx.x + 1) / gridDim.x;
  double sum[2] = {0., 0.};
  shampoo_segment seg[kSegs];
  shampoo_tensor t[kSegs];
  auto describe = [&](int64_t s) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < kSegs; ++k) {
      seg[k] = segments[min(s + k, nseg - 1)];
      t[k] = tensors[seg[k].tensor];
    }
  };
  describe(s0);
  for (int64_t s = s0; s < s1; s += kSegs) {
    float x[kSegs][kRounds][V];
    int64_t first[kSegs];
    int len[kSegs];
    bool whole = true;
#pragma unroll
    for (int k = 0; k < kSegs; ++k) {
      first[k] = (int64_t)seg[k].index * kSegment;
      len[k] = s + k < s1 ? (int)min((int64_t)kSegment, t[k].n - first[k]) : 0;
      whole = whole && len[k] == kSegment;
    }
    // one branch for all: each would wait for its loads where it ends
    auto load = [&](auto WHOLE) __attribute__((always_inline)) {
#pragma unroll
      for (int k = 0; k < kSegs; ++k)
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
          const int i = (r * 256 + (int)threadIdx.x) * V;
          load_elems<BF16, V, decltype(WHOLE)::value>(t[k].ptr, first[k] + i, len[k] - i, x[k][r]);
        }
    };
    if (whole) {
      load(std::true_type{});
    } else {
      load(std::false_type{});
    }
    describe(s + kSegs);  // the next descriptors, under these loads
#pragma unroll
    for (int k = 0; k < kSegs; ++k)
#pragma unroll
      for (int r = 0; r < kRounds; ++r)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const double g = x[k][r][e];
          sum[e & 1] = __builtin_fma(g, g, sum[e & 1]);
        }
  }
  const double total = block_sum_f64<256>(sum[0] + sum[1], red);
  if (threadIdx.x == 0) stg(partial + blockIdx.x, total);
}

__global__ void __launch_bounds__(256) grad_norm_final_kernel(const double* partial, int count, float max_norm,
                                                              float* out) {
  __shared__ double red[4];
  double sum = 0.;
  for (int i = threadIdx.x; i < count; i += 256) sum += ldg(partial + i);
  sum = block_sum_f64<256>(sum, red);
  if (threadIdx.x == 0) store_norm(sum, max_norm, out);
}

// A few segments: both passes in one workgroup, a wave a segment (49 vectors of
// 1024 floats: 4.8 us, the latency of three dependent loads a segment).
template <bool BF16>
__global__ void __launch_bounds__(1024) grad_norm_small_kernel(const shampoo_tensor* tensors,
                                                               const shampoo_segment* segments, int nseg,
                                                               float max_norm, float* out) {
  __shared__ double red[16];
  constexpr int V = BF16 ? 8 : 4;
  const int lane = threadIdx.x % kWave;
  double sum = 0.;
  for (int s = threadIdx.x / kWave; s < nseg; s += 16) {
    const shampoo_segment seg = segments[s];
    const shampoo_tensor t = tensors[seg.tensor];
    const int64_t first = (int64_t)seg.index * kSegment;
    const int len = (int)min((int64_t)kSegment, t.n - first);
#pragma unroll 4
    for (int i = lane * V; i < len; i += kWave * V) {
      float x[V];
      if (i + V <= len) {
        load_elems<BF16, V, true>(t.ptr, first + i, V, x);
      } else {
        load_elems<BF16, V, false>(t.ptr, first + i, len - i, x);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) sum = __builtin_fma((double)x[e], (double)x[e], sum);
    }
  }
  sum = block_sum_f64<1024>(sum, red);
  if (threadIdx.x == 0) store_norm(sum, max_norm, out);
}

}  // namespace shp
