// MX8 rows (E4M3 values, one E8M0 scale byte per 32 columns): conversion of
// pieces held in registers, and the kernels that convert whole matrices.
#pragma once

#include "vector_io.h"

namespace shp {

constexpr int kMx8Group = SHAMPOO_GROUP;

__host__ __device__ __forceinline__ int64_t mx8_padded(int64_t cols) {
  return (cols + kMx8Group - 1) / kMx8Group * kMx8Group;
}

typedef short i16x2 __attribute__((ext_vector_type(2)));

// Scale byte of a group from the bits of its largest magnitude (as fp32): that
// one comes to lie in [2^7, 2^8), below E4M3's largest, 448, so that nothing
// saturates; the 13 binades below it are held to a relative 2^-4, what lies lower to 2^-17 of the largest.
__device__ __forceinline__ uint32_t mx8_row_scale(uint32_t top_bits) {
  const int e = (int)(top_bits >> 23);
  return e == 255 ? 255u : (uint32_t)max(e - 7, 1);
}

// An MX8 matrix that is written or read beside a matrix of the same shape.
struct Mx8Rows {
  uint8_t *codes, *scales;
  uint32_t padded;
};

// V consecutive codes of a row, and the scale of their group.
template <int V>
struct Mx8Piece {
  typedef uint32_t Words __attribute__((ext_vector_type(V / 4)));
  Words c;
  uint32_t s;

  // Codes of a piece whose group lies in 32 / V consecutive lanes; nearest even
  // after the exact division by the scale.
  template <bool BF16>
  __device__ __forceinline__ void encode(const Piece<BF16, V>& x) {
    s = mx8_row_scale(group_max<kMx8Group / V>(x.top()));
    const float scale = __builtin_bit_cast(float, s << 23);
    static_for<V / 4>([&](auto I) __attribute__((always_inline)) {
      constexpr int i = decltype(I)::value;
      i16x2 w = {0, 0};
      if constexpr (BF16) {
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, __builtin_bit_cast(bf16x2_t, (uint32_t)x.w[2 * i]), scale, false);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, __builtin_bit_cast(bf16x2_t, (uint32_t)x.w[2 * i + 1]), scale, true);
      } else {
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, elem(x, 4 * i), elem(x, 4 * i + 1), scale, false);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, elem(x, 4 * i + 2), elem(x, 4 * i + 3), scale, true);
      }
      c[i] = s == 255 ? 0x7f7f7f7fu : __builtin_bit_cast(uint32_t, w);  // NaN, four times
    });
  }
  __device__ __forceinline__ void store(const Mx8Rows& m, int64_t row, uint32_t col) const {
    if (col < m.padded) {
      stg_once<Words, 4>(m.codes + row * (int64_t)m.padded + col, c);
      if (col % kMx8Group == 0) stg(m.scales + row * (int64_t)(m.padded / kMx8Group) + col / kMx8Group, (uint8_t)s);
    }
  }
  __device__ __forceinline__ void load(const Mx8Rows& m, int64_t row, uint32_t col) {
    c = (Words)0u;
    s = 1;
    if (col < m.padded) {
      c = ldg_once<Words, 4>(m.codes + row * (int64_t)m.padded + col);
      s = ldg(m.scales + row * (int64_t)(m.padded / kMx8Group) + col / kMx8Group);
    }
  }
  // The same without a branch: beyond the row's end codes that are there, to be cleared when they have come.
  __device__ __forceinline__ void load_near(const Mx8Rows& m, int64_t row, uint32_t col) {
    const uint32_t from = min(col, m.padded - V);
    c = ldg_once<Words, 4>(m.codes + row * (int64_t)m.padded + from);
    s = ldg(m.scales + row * (int64_t)(m.padded / kMx8Group) + from / kMx8Group);
  }
  __device__ __forceinline__ void clear() {
    c = (Words)0u;
    s = 1;
  }
  // The values; where s = 255 those of the codes quantisation writes beside it, NaN.
  __device__ __forceinline__ void decode(float (&x)[V]) const {
    const float scale = __builtin_bit_cast(float, s << 23);
    static_for<V / 4>([&](auto I) __attribute__((always_inline)) {
      constexpr int i = decltype(I)::value;
      const f32x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((uint32_t)c[i], scale, false);
      const f32x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((uint32_t)c[i], scale, true);
      x[4 * i] = lo[0];
      x[4 * i + 1] = lo[1];
      x[4 * i + 2] = hi[0];
      x[4 * i + 3] = hi[1];
    });
  }
};

// What a pass over a matrix in pieces needs: 2^lanes_log2 lanes take a stretch
// of a row, a row has col_blocks of them.
struct RowShape {
  uint32_t col_blocks;
  int lanes_log2;
};

struct Mx8Args {
  const void* x;
  void* out;
  int64_t rows, ld;
  uint32_t cols;
  Mx8Rows m;
  RowShape shape;
};

// Bound by HBM: each element is read once, each code written once.  Lanes hold
// consecutive pieces of 16 bytes, so that a group is 4 (bf16) or 8 (fp32) lanes, whose
// largest magnitude is found by DPP without LDS; 4 rows a thread keep 4 loads in
// flight.  16384 x 8192 bf16: 70 us to codes and 65 back, 5.8 and 6.2 TB/s; with
// stores through the caches 155 us for both.
constexpr int kMx8Passes = 4;  // rows a thread takes

template <bool BF16>
__global__ void __launch_bounds__(256) mx8_quantize_kernel(const Mx8Args P) {
  constexpr int V = BF16 ? 8 : 4;
  const uint32_t rb = blockIdx.x / P.shape.col_blocks, cb = blockIdx.x - rb * P.shape.col_blocks;
  const int lanes = 1 << P.shape.lanes_log2, per_pass = 256 >> P.shape.lanes_log2;
  const uint32_t col = (cb * lanes + (threadIdx.x & (lanes - 1))) * V;
  const int64_t row0 = (int64_t)rb * kMx8Passes * per_pass + (threadIdx.x >> P.shape.lanes_log2);
  Piece<BF16, V> x[kMx8Passes];
#pragma unroll
  for (int i = 0; i < kMx8Passes; ++i) {
    const int64_t r = min(row0 + i * per_pass, P.rows - 1);
    x[i] = load_row<BF16, V>(row_at<BF16>(P.x, r, P.ld), P.cols, col);
  }
#pragma unroll
  for (int i = 0; i < kMx8Passes; ++i) {
    const int64_t r = row0 + i * per_pass;
    Mx8Piece<V> q;
    q.encode(x[i]);
    if (r < P.rows) q.store(P.m, r, col);
  }
}

template <bool BF16>
__global__ void __launch_bounds__(256) mx8_dequantize_kernel(const Mx8Args P) {
  constexpr int V = BF16 ? 8 : 4;
  const uint32_t rb = blockIdx.x / P.shape.col_blocks, cb = blockIdx.x - rb * P.shape.col_blocks;
  const int lanes = 1 << P.shape.lanes_log2, per_pass = 256 >> P.shape.lanes_log2;
  const uint32_t col = (cb * lanes + (threadIdx.x & (lanes - 1))) * V;
  const int64_t row0 = (int64_t)rb * kMx8Passes * per_pass + (threadIdx.x >> P.shape.lanes_log2);
  if (col >= P.cols) return;
  Mx8Piece<V> q[kMx8Passes];
#pragma unroll
  for (int i = 0; i < kMx8Passes; ++i) q[i].load(P.m, min(row0 + i * per_pass, P.rows - 1), col);
#pragma unroll
  for (int i = 0; i < kMx8Passes; ++i) {
    const int64_t r = row0 + i * per_pass;
    if (r >= P.rows) return;
    float x[V];
    q[i].decode(x);
    if (q[i].s == 255) {  // whatever the codes are
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] = __builtin_nanf("");
    }
    store_row<BF16, V>(row_at<BF16>(P.out, r, P.ld), P.cols, col, x);
  }
}

}  // namespace shp
