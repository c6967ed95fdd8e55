// AdamW over many tensors and the norm of many tensors: HBM-bound kernels that
// walk a list of 4096-element segments, one workgroup a segment.
#pragma once

#include "common.h"

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

__device__ __forceinline__ float load_elem(const void* p, int64_t i, int bf16) {
  if (!bf16) return ldg(static_cast<const float*>(p) + i);
  return __builtin_bit_cast(float, (uint32_t)ldg(static_cast<const uint16_t*>(p) + i) << 16);
}

__device__ __forceinline__ float group_max_abs_bits(float x, uint32_t& bits) {
  bits = __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) bits = max(bits, (uint32_t)__shfl_xor((int)bits, off, kWave));
  return x;
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
  int param_bf16, grad_bf16, mx8;
};

__global__ void __launch_bounds__(256) adamw_kernel(const AdamwArgs P) {
// Which operations are fused is written out: the codes that the moments round
// to must not depend on the compiler's choice.
#pragma clang fp contract(off)
  const shampoo_segment seg = P.segments[blockIdx.x];
  if ((uint64_t)seg.tensor >= (uint64_t)P.ntensors || seg.index < 0) return;
  float c = 1.f;
  if (P.grad_scale != nullptr) {
    c = *P.grad_scale;
    if (!(fabsf(c) <= FLT_MAX)) return;
  }
  const shampoo_tensor tp = P.params[seg.tensor], tg = P.grads[seg.tensor];
  const int64_t first = (int64_t)seg.index * kSegment;
  const int64_t left = min(tp.n, tg.n) - first;
  const int len = (int)min((int64_t)kSegment, left);
  const float eta = P.lr * P.hyper[2 * seg.tensor], keep = 1.f - eta * P.hyper[2 * seg.tensor + 1];
  const float step = eta * P.rbc1, k1 = (float)(P.omb1 * c), k2 = (float)(P.omb2 * c);
  for (int i0 = 0; i0 < len; i0 += 256) {
    const int i = i0 + threadIdx.x;
    const bool in = i < len;
    const int64_t at = first + i, pos = tp.offset + at, grp = pos / kGroup;
    float g = 0.f, m = 0.f, v = 0.f;
    if (in) {
      g = load_elem(tg.ptr, at, P.grad_bf16);
      if (P.mx8) {
        m = mx8_decode<MomentM>(ldg(static_cast<const uint8_t*>(P.m) + pos), ldg(P.m_scale + grp));
        v = mx8_decode<MomentV>(ldg(static_cast<const uint8_t*>(P.v) + pos), ldg(P.v_scale + grp));
      } else {
        m = ldg(static_cast<const float*>(P.m) + pos);
        v = ldg(static_cast<const float*>(P.v) + pos);
      }
      // The scale c goes into the constants (in double) where that cannot overflow:
      // g c g k2 keeps v finite for a huge g with a small c, and takes four roundings at most.
      m = __builtin_fmaf(g, k1, P.beta1 * m);
      v = __builtin_fmaf(g * c, g * k2, P.beta2 * v);
    }
    const uint32_t h =
        hash_finish((uint32_t)pos * kHashC1 + (uint32_t)((uint64_t)pos >> 32) * kHashC4 + P.key);
    if (P.mx8) {
      uint32_t mb, vb;
      group_max_abs_bits(m, mb);
      group_max_abs_bits(v, vb);
      const int ms = mx8_scale<MomentM>(mb), vs = mx8_scale<MomentV>(vb);
      if (in) {
        stg(static_cast<uint8_t*>(P.m) + pos, (uint8_t)mx8_encode<MomentM>(m, ms, h & 0xffffu));
        stg(static_cast<uint8_t*>(P.v) + pos, (uint8_t)mx8_encode<MomentV>(v, vs, h >> 16));
        if ((i % kGroup) == 0) {
          stg(P.m_scale + grp, (uint8_t)ms);
          stg(P.v_scale + grp, (uint8_t)vs);
        }
      }
    } else if (in) {
      stg(static_cast<float*>(P.m) + pos, m);
      stg(static_cast<float*>(P.v) + pos, v);
    }
    if (!in) continue;
    const float d = m / (sqrtf(v) * P.rsbc2 + P.eps);
    const float p = load_elem(tp.ptr, at, P.param_bf16) * keep - step * d;
    if (P.param_bf16) {
      const uint32_t b = (__builtin_bit_cast(uint32_t, p) + ((h * kHashC2) >> 16)) >> 16;
      stg(static_cast<uint16_t*>(tp.ptr) + at, (uint16_t)(p != p ? 0x7fc0u : b));
    } else {
      stg(static_cast<float*>(tp.ptr) + at, p);
      if (P.copies != nullptr) stg(static_cast<uint16_t*>(P.copies[seg.tensor].ptr) + at, f32_to_bf16_bits(p));
    }
  }
}

template <class F>
__global__ void __launch_bounds__(256) mx8_decode_kernel(const uint8_t* codes, const uint8_t* scales, int64_t n,
                                                         void* out, int bf16) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const float v = mx8_decode<F>(ldg(codes + i), ldg(scales + i / kGroup));
  if (bf16) {
    stg(static_cast<uint16_t*>(out) + i, f32_to_bf16_bits(v));
  } else {
    stg(static_cast<float*>(out) + i, v);
  }
}

// ---------------------------------------------------------------------------
// Norm.  Pass 1: each workgroup sums the squares of a contiguous run of
// segments in double (a product of two floats is exact there, and no fp32
// gradient overflows it); pass 2: one workgroup adds the partial sums.  Both
// in a fixed order.
// ---------------------------------------------------------------------------
__device__ __forceinline__ double block_sum_f64(double v, double* red) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
  if ((threadIdx.x % kWave) == 0) red[threadIdx.x / kWave] = v;
  __syncthreads();
  double t = 0.;
#pragma unroll
  for (int i = 0; i < 4; ++i) t += red[i];
  __syncthreads();
  return t;
}

__global__ void __launch_bounds__(256) grad_norm_partial_kernel(const shampoo_tensor* tensors,
                                                                const shampoo_segment* segments, int64_t nseg,
                                                                int bf16, double* partial) {
  __shared__ double red[4];
  double sum = 0.;
  const int64_t s1 = nseg * (blockIdx.x + 1) / gridDim.x;
  for (int64_t s = nseg * blockIdx.x / gridDim.x; s < s1; ++s) {
    const shampoo_segment seg = segments[s];
    const shampoo_tensor t = tensors[seg.tensor];
    const int64_t first = (int64_t)seg.index * kSegment;
    const int len = (int)min((int64_t)kSegment, t.n - first);
    for (int i = threadIdx.x; i < len; i += 256) {
      const double g = load_elem(t.ptr, first + i, bf16);
      sum += g * g;
    }
  }
  sum = block_sum_f64(sum, red);
  if (threadIdx.x == 0) stg(partial + blockIdx.x, sum);
}

__global__ void __launch_bounds__(256) grad_norm_final_kernel(const double* partial, int count, float max_norm,
                                                              float* out) {
  __shared__ double red[4];
  double sum = 0.;
  for (int i = threadIdx.x; i < count; i += 256) sum += ldg(partial + i);
  sum = block_sum_f64(sum, red);
  if (threadIdx.x != 0) return;
  const double norm = sqrt(sum);
  const float f = (float)norm;
  float coef = norm > max_norm ? (float)(max_norm / norm) : 1.f;
  if (!(f <= FLT_MAX)) coef = __builtin_nanf("");
  stg(out, f);
  stg(out + 1, coef);
}

}  // namespace shp
