// MX4 (E2M1 values, one E8M0 scale byte per 32) matrices: quantisation and the
// product C = alpha A B^T + beta C on the scaled MFMA of gfx950.
#pragma once

#include "common.h"

namespace shp {

constexpr int kMx4Pad = SHAMPOO_MX4_PAD;
constexpr int kMx4Group = SHAMPOO_GROUP;

typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx8 __attribute__((ext_vector_type(8)));

__host__ __device__ __forceinline__ int64_t mx4_padded(int64_t k) { return (k + kMx4Pad - 1) / kMx4Pad * kMx4Pad; }

// 2^(s - 127) for a scale byte s <= 254 (s = 0 is a subnormal float).
__device__ __forceinline__ float mx4_pow2(int s) {
  return __builtin_bit_cast(float, s == 0 ? 0x00400000u : (uint32_t)s << 23);
}

// Scale byte of a group from the bits of its largest magnitude.
__device__ __forceinline__ int mx4_scale(uint32_t top_bits) {
  const int e = (int)(top_bits >> 23);
  return e == 255 ? 255 : max(e - 2, 0);
}

// E2M1 code of x / 2^(s - 127), to nearest even, at most 6.
__device__ __forceinline__ uint32_t mx4_encode(float x, int s) {
  if (s == 255) return 0;
  const float a = fabsf(x) * __builtin_bit_cast(float, (uint32_t)(254 - s) << 23);
  uint32_t c;
  if (a < 2.f) {
    c = (uint32_t)rintf(2.f * a);
  } else if (a < 4.f) {
    c = (uint32_t)rintf(a) + 2;
  } else {
    c = min((uint32_t)rintf(0.5f * a) + 4, 7u);
  }
  return c | (x < 0.f ? 8u : 0u);
}

__device__ __forceinline__ float mx4_value(uint32_t code, int s) {
  const uint32_t c = code & 7;
  // 0, 0.5, then 1 and a mantissa bit below the exponent c >> 1
  float v = c < 2 ? 0.5f * (float)c : __builtin_bit_cast(float, ((126u + (c >> 1)) << 23) | ((c & 1u) << 22));
  if (code & 8) v = -v;
  return s == 255 ? __builtin_nanf("") : v * mx4_pow2(s);
}

struct Mx4QuantArgs {
  const void* x;
  int64_t rows, cols;       // of the quantised matrix
  int64_t row_step, col_step;  // element strides of x along them
  int64_t padded;           // mx4_padded(cols)
  uint8_t *codes, *scales;
  int bf16;
};

// One lane an element, 32 lanes a group.
__global__ void __launch_bounds__(256) mx4_quantize_kernel(const Mx4QuantArgs P) {
  const int64_t groups = P.padded / kMx4Group;
  const int64_t id = (int64_t)blockIdx.x * 8 + threadIdx.x / kMx4Group;
  const int lane = threadIdx.x % kMx4Group;
  const bool in = id < P.rows * groups;
  const int64_t r = in ? id / groups : 0, k = in ? (id - r * groups) * kMx4Group + lane : 0;
  float x = 0.f;
  if (in && k < P.cols) {
    const int64_t at = r * P.row_step + k * P.col_step;
    x = P.bf16 ? __builtin_bit_cast(float, (uint32_t)ldg(static_cast<const uint16_t*>(P.x) + at) << 16)
               : ldg(static_cast<const float*>(P.x) + at);
  }
  uint32_t top = __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, kWave));
  const int s = mx4_scale(top);
  const uint32_t c = mx4_encode(x, s), hi = (uint32_t)__shfl_xor((int)c, 1, kWave);
  if (!in) return;
  if ((lane & 1) == 0) stg(P.codes + r * (P.padded / 2) + k / 2, (uint8_t)(c | (hi << 4)));
  if (lane == 0) stg(P.scales + id, (uint8_t)s);
}

__global__ void __launch_bounds__(256) mx4_dequantize_kernel(const uint8_t* codes, const uint8_t* scales,
                                                             int64_t rows, int64_t cols, int64_t padded, void* out,
                                                             int bf16, int64_t ld) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t r = id / (padded / 2), b = id - r * (padded / 2);
  if (r >= rows) return;
  const uint32_t c = ldg(codes + id);
  const int s = ldg(scales + r * (padded / kMx4Group) + 2 * b / kMx4Group);
  for (int h = 0; h < 2; ++h) {
    const int64_t k = 2 * b + h;
    if (k >= cols) return;
    const float v = mx4_value((c >> (4 * h)) & 15u, s);
    if (bf16) {
      stg(static_cast<uint16_t*>(out) + r * ld + k, f32_to_bf16_bits(v));
    } else {
      stg(static_cast<float*>(out) + r * ld + k, v);
    }
  }
}

struct Mx4ProductArgs {
  const uint8_t *a, *as, *b, *bs;
  int64_t M, N, padded;  // padded: columns of the operands as stored
  void* c;
  int64_t ldc;
  float alpha, beta;
  int bf16;
};

// C += with lane l of a wave holding 32 consecutive columns of one row of each
// operand and their scale byte: row l % 16, columns 32 (l / 16) onwards of a
// 128-column step.  The result's lane l has column l % 16, rows 4 (l / 16)
// to 4 (l / 16) + 3.
__device__ __forceinline__ floatx4 mfma_mx4(const intx4& a, const intx4& b, const floatx4& c, int sa, int sb) {
  const intx8 x = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, y = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 0, sa, 0, sb);
}

// One wave a 16 x 16 tile, operands straight from memory.
__global__ void __launch_bounds__(256) mx4_product_kernel(const Mx4ProductArgs P) {
  const int lane = threadIdx.x % kWave;
  const int64_t tiles_n = (P.N + 15) / 16;
  const int64_t tile = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave;
  const int64_t tm = tile / tiles_n, tn = tile - tm * tiles_n;
  if (tm * 16 >= P.M) return;
  const int64_t row = min(tm * 16 + lane % 16, P.M - 1), col = min(tn * 16 + lane % 16, P.N - 1);
  floatx4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int64_t k = 32 * (lane / 16); k < P.padded; k += 128) {
    const intx4 a = ldg(reinterpret_cast<const intx4*>(P.a + (row * P.padded + k) / 2));
    const intx4 b = ldg(reinterpret_cast<const intx4*>(P.b + (col * P.padded + k) / 2));
    const int sa = ldg(P.as + (row * P.padded + k) / kMx4Group), sb = ldg(P.bs + (col * P.padded + k) / kMx4Group);
    acc = mfma_mx4(a, b, acc, sa, sb);
  }
  const int64_t n = tn * 16 + lane % 16;
  for (int r = 0; r < 4; ++r) {
    const int64_t m = tm * 16 + 4 * (lane / 16) + r;
    if (m >= P.M || n >= P.N) continue;
    float v = P.alpha * acc[r];
    const int64_t at = m * P.ldc + n;
    if (P.bf16) {
      uint16_t* c = static_cast<uint16_t*>(P.c) + at;
      if (P.beta != 0.f) v += P.beta * __builtin_bit_cast(float, (uint32_t)ldg(c) << 16);
      stg(c, f32_to_bf16_bits(v));
    } else {
      float* c = static_cast<float*>(P.c) + at;
      if (P.beta != 0.f) v += P.beta * ldg(c);
      stg(c, v);
    }
  }
}

}  // namespace shp
