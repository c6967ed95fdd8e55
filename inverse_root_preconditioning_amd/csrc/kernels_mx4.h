// MX4 (E2M1 values, one E8M0 scale byte per 32) matrices: quantisation and the
// product C = alpha A B^T + beta C on the scaled MFMA of gfx950.
#pragma once

#include "vector_io.h"

namespace shp {

constexpr int kMx4Pad = SHAMPOO_MX4_PAD;
constexpr int kMx4Group = SHAMPOO_GROUP;

typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx8 __attribute__((ext_vector_type(8)));

__host__ __device__ __forceinline__ int64_t mx4_padded(int64_t k) { return (k + kMx4Pad - 1) / kMx4Pad * kMx4Pad; }

// Scale byte of a group from the bits of its largest magnitude (as fp32).
__device__ __forceinline__ uint32_t mx4_scale(uint32_t top_bits) {
  const int e = (int)(top_bits >> 23);
  return e == 255 ? 255u : (uint32_t)max(e - 2, 0);
}

// The conversions take 2^(s - 127) as a float of exponent field s, also where
// that is a subnormal (s = 0): they use the field alone.  They round to
// nearest even and saturate at 6.
__device__ __forceinline__ float mx4_scale_float(uint32_t s) { return __builtin_bit_cast(float, s << 23); }

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                __builtin_bit_cast(u16x2, b)));
}
__device__ __forceinline__ uint32_t abs_halves(uint32_t a) { return a & 0x7fff7fffu; }

// Byte SEL of `old` replaced by the codes of two values.
template <int SEL>
__device__ __forceinline__ uint32_t mx4_codes_bf16(uint32_t old, uint32_t pair, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2_t, pair), scale, SEL);
}
template <int SEL>
__device__ __forceinline__ uint32_t mx4_codes_f32(uint32_t old, float a, float b, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, a, b, scale, SEL);
}

struct Mx4QuantArgs {
  const void* x;
  int64_t rows, cols, ld;
  int64_t padded_cols, padded_rows;  // mx4_padded
  uint8_t *codes, *scales;           // of x
  uint8_t *codes_t, *scales_t;       // of its transpose
  uint32_t col_blocks;
  int lanes_log2;                    // rows kernel: lanes on a row
};

// V consecutive elements of a row: bf16, two a word, or fp32 bits.
template <bool BF16, int V>
struct Mx4Piece {
  static constexpr int kElems = V, kWords = BF16 ? V / 2 : V;
  typedef uint32_t Words __attribute__((ext_vector_type(kWords)));
  Words w;
  __device__ __forceinline__ void load(const void* x, int64_t at) {
    if constexpr (BF16) {
      w = ldg_any<Words, 2>(static_cast<const uint16_t*>(x) + at);
    } else {
      w = ldg_any<Words, 4>(static_cast<const float*>(x) + at);
    }
  }
  // The piece at (row, col) of a matrix whose edge it may cross (or pass), zero
  // outside.  No branch on the lane: V elements that are there, shifted down.
  __device__ __forceinline__ void load_edge(const void* x, int64_t rows, int64_t cols, int64_t ld, int64_t row,
                                            int64_t col) {
    if (cols >= V) {
      const int64_t from = min(col, cols - V);
      const uint32_t d = row < rows ? (uint32_t)min<int64_t>(col - from, V) : (uint32_t)V;
      load(x, min(row, rows - 1) * ld + from);
      if constexpr (BF16) {
        if (d & 1) {
#pragma unroll
          for (int i = 0; i < kWords; ++i) w[i] = (w[i] >> 16) | (i + 1 < kWords ? w[i + 1] << 16 : 0u);
        }
      }
#pragma unroll
      for (int b = 1; b < kWords; b *= 2) {
        if (d & (BF16 ? 2 * b : b)) {
#pragma unroll
          for (int i = 0; i < kWords; ++i) w[i] = i + b < kWords ? w[i + b] : 0u;
        }
      }
      if (d == V) w = (Words)0u;
    } else {
      w = (Words)0u;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (row < rows && col + e < cols) {
          if constexpr (BF16) {
            w[e / 2] |= (uint32_t)ldg(static_cast<const uint16_t*>(x) + row * ld + col + e) << (16 * (e & 1));
          } else {
            w[e] = ldg(static_cast<const uint32_t*>(x) + row * ld + col + e);
          }
        }
      }
    }
  }
  // Bits, as fp32, of the largest magnitude.
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
    if constexpr (BF16) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) m = max_halves(m, abs_halves(w[i]));
      return max(m & 0xffff0000u, m << 16);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) m = max(m, w[i] & 0x7fffffffu);
      return m;
    }
  }
  // V / 2 bytes of codes.
  __device__ __forceinline__ uint32_t encode(float scale) const {
    uint32_t c = 0;
    static_for<V / 2>([&](auto I) __attribute__((always_inline)) {
      constexpr int i = decltype(I)::value;
      if constexpr (BF16) {
        c = mx4_codes_bf16<i>(c, w[i], scale);
      } else {
        c = mx4_codes_f32<i>(c, __builtin_bit_cast(float, (uint32_t)w[2 * i]),
                             __builtin_bit_cast(float, (uint32_t)w[2 * i + 1]), scale);
      }
    });
    return c;
  }
};

// Rows only: 8 elements a lane, 4 lanes a group; a workgroup takes `lanes` x 8
// columns of 4 x 256 / lanes rows.  Memory-bound: 16384 x 8192 bf16 in 60 us
// (5.6 TB/s), fp32 in 110 us (5.5).
template <bool BF16>
__global__ void __launch_bounds__(256) mx4_quantize_rows_kernel(const Mx4QuantArgs P) {
  constexpr int kPasses = 4;
  const uint32_t rb = blockIdx.x / P.col_blocks, cb = blockIdx.x - rb * P.col_blocks;
  const int lanes = 1 << P.lanes_log2, per_pass = 256 >> P.lanes_log2;
  const int64_t col = ((int64_t)cb * lanes + (threadIdx.x & (lanes - 1))) * 8;
  const int64_t row0 = (int64_t)rb * kPasses * per_pass + (threadIdx.x >> P.lanes_log2);
  Mx4Piece<BF16, 8> x[kPasses];
  if (((int64_t)rb + 1) * kPasses * per_pass <= P.rows && ((int64_t)cb + 1) * lanes * 8 <= P.cols) {
#pragma unroll
    for (int i = 0; i < kPasses; ++i) x[i].load(P.x, (row0 + i * per_pass) * P.ld + col);
  } else {
#pragma unroll
    for (int i = 0; i < kPasses; ++i) x[i].load_edge(P.x, P.rows, P.cols, P.ld, row0 + i * per_pass, col);
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int64_t r = row0 + i * per_pass;
    const uint32_t s = mx4_scale(group_max<4>(x[i].top()));
    uint32_t c = x[i].encode(mx4_scale_float(s));
    if (s == 255) c = 0;
    if (r < P.rows && col < P.padded_cols) {
      stg(reinterpret_cast<uint32_t*>(P.codes + r * (P.padded_cols / 2) + col / 2), c);
      if ((threadIdx.x & 3) == 0) stg(P.scales + r * (P.padded_cols / kMx4Group) + col / kMx4Group, (uint8_t)s);
    }
  }
}

// Columns, and rows as well with ROWS, from one reading: a wave holds 32 rows of
// 64 pieces of V elements in registers, so that a group along a column lies
// within a lane and one along a row within 32 / V lanes.  The 4 waves of a workgroup
// are stacked, and the 16 bytes that a lane has for a column of the transpose
// meet their neighbours in LDS, so that 64 bytes are stored at a time.  Rows up
// to padded_rows are zero groups.
template <bool BF16, int V, bool ROWS>
__global__ void __launch_bounds__(256, 2) mx4_quantize_cols_kernel(const Mx4QuantArgs P) {
  constexpr int kLanes = kMx4Group / V, kCols = kWave * V;
  constexpr int kPitch = 64;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kCols * (kPitch + 4)];
  const uint32_t rb = blockIdx.x / P.col_blocks, cb = blockIdx.x - rb * P.col_blocks;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int64_t base = (int64_t)rb * 128, row0 = base + wave * 32;
  const int64_t col0 = (int64_t)cb * kCols, col = col0 + lane * V;

  auto quantize = [&](auto WHOLE) __attribute__((always_inline)) {
    constexpr bool kWhole = decltype(WHOLE)::value;
    Mx4Piece<BF16, V> x[32];
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      if constexpr (kWhole) {
        x[r].load(P.x, (row0 + r) * P.ld + col);
      } else {
        x[r].load_edge(P.x, P.rows, P.cols, P.ld, row0 + r, col);
      }
    }
    if constexpr (ROWS) {
      const int part = lane % kLanes;
      const int64_t pitch = P.padded_cols / 2, spitch = P.padded_cols / kMx4Group;
      uint8_t* const codes = P.codes + row0 * pitch + col / 2;
      uint8_t* const scales = P.scales + row0 * spitch + col / kMx4Group;
      uint32_t mine = 0;
#pragma unroll
      for (int r = 0; r < 32; ++r) {
        if (r % 4 == 0) __builtin_amdgcn_sched_barrier(0);  // keeps the rows' temporaries out of each other's way
        const uint32_t s = mx4_scale(group_max<kLanes>(x[r].top()));
        uint32_t c = x[r].encode(mx4_scale_float(s));
        if (s == 255) c = 0;
        if (kWhole || (row0 + r < P.rows && col < P.padded_cols)) {
          if constexpr (V == 8) {
            stg(reinterpret_cast<uint32_t*>(codes + r * pitch), c);
          } else if constexpr (V == 4) {
            stg(reinterpret_cast<uint16_t*>(codes + r * pitch), (uint16_t)c);
          } else {
            stg(codes + r * pitch, (uint8_t)c);
          }
        }
        // each lane of a group keeps the scale of one of kLanes rows, then all store
        if (part == r % kLanes) mine = s;
        if (r % kLanes == kLanes - 1) {
          const int q = r - (kLanes - 1) + part;
          if (kWhole || (row0 + q < P.rows && col < P.padded_cols)) stg(scales + q * spitch, (uint8_t)mine);
        }
      }
    }
    static_for<V>([&](auto I) __attribute__((always_inline)) {
      constexpr int i = decltype(I)::value;
      uint32_t top = 0;
      u32x4 out;
      if constexpr (BF16) {
        uint32_t m = 0;
#pragma unroll
        for (int r = 0; r < 32; ++r) m = max_halves(m, abs_halves(x[r].w[i / 2]));
        top = (i & 1) ? m & 0xffff0000u : m << 16;
      } else {
#pragma unroll
        for (int r = 0; r < 32; ++r) top = max(top, x[r].w[i] & 0x7fffffffu);
      }
      const uint32_t s = mx4_scale(top);
      const float scale = mx4_scale_float(s);
      static_for<4>([&](auto D) __attribute__((always_inline)) {
        constexpr int d = decltype(D)::value;
        uint32_t c = 0;
        static_for<4>([&](auto B) __attribute__((always_inline)) {
          constexpr int b = decltype(B)::value, r = 8 * d + 2 * b;
          if constexpr (BF16) {
            // rows r and r + 1 of this column: both low or both high halves
            const uint32_t pair = __builtin_amdgcn_perm(x[r + 1].w[i / 2], x[r].w[i / 2],
                                                        (i & 1) ? 0x07060302u : 0x05040100u);
            c = mx4_codes_bf16<b>(c, pair, scale);
          } else {
            c = mx4_codes_f32<b>(c, __builtin_bit_cast(float, (uint32_t)x[r].w[i]),
                                 __builtin_bit_cast(float, (uint32_t)x[r + 1].w[i]), scale);
          }
        });
        out[d] = s == 255 ? 0u : c;
      });
      // at place (wave + lane) % 4 of the column's four: lanes are V columns apart
      const int c = lane * V + i;
      *reinterpret_cast<u32x4*>(lds + c * kPitch + 16 * ((wave + lane) & 3)) = out;
      lds[kCols * kPitch + c * 4 + wave] = (uint8_t)s;
    });
  };
  if (base + 128 <= P.rows && col0 + kCols <= P.cols) {
    quantize(std::true_type{});
  } else {
    quantize(std::false_type{});
  }
  __syncthreads();
  const int64_t pitch = P.padded_rows / 2, spitch = P.padded_rows / kMx4Group;
#pragma unroll 4
  for (int q = threadIdx.x; q < kCols * 4; q += 256) {
    const int c = q / 4, u = q % 4;
    if (col0 + c < P.cols)
      stg(reinterpret_cast<u32x4*>(P.codes_t + (col0 + c) * pitch + base / 2 + 16 * u),
          *reinterpret_cast<const u32x4*>(lds + c * kPitch + 16 * ((u + c / V) & 3)));
  }
  for (int c = threadIdx.x; c < kCols; c += 256) {
    if (col0 + c < P.cols)
      stg(reinterpret_cast<uint32_t*>(P.scales_t + (col0 + c) * spitch + base / kMx4Group),
          *reinterpret_cast<const uint32_t*>(lds + kCols * kPitch + c * 4));
  }
}

struct Mx4DequantArgs {
  const uint8_t *codes, *scales;
  int64_t rows, cols, padded, ld;
  void* out;
  uint32_t col_blocks;
  int lanes_log2;
};

// 16 bytes of output a lane (8 bf16, 4 floats), the rows kernel's shape.
// Memory-bound: 16384 x 8192 to bf16 in 62 us (5.5 TB/s), to fp32 in 108 us
// (5.6; 153 us with 8 floats a lane, half cache lines a store).
template <bool BF16>
__global__ void __launch_bounds__(256) mx4_dequantize_kernel(const Mx4DequantArgs P) {
  constexpr int kPasses = 4, E = BF16 ? 8 : 4;
  const uint32_t rb = blockIdx.x / P.col_blocks, cb = blockIdx.x - rb * P.col_blocks;
  const int lanes = 1 << P.lanes_log2, per_pass = 256 >> P.lanes_log2;
  const int64_t col = ((int64_t)cb * lanes + (threadIdx.x & (lanes - 1))) * E;
  const int64_t row0 = (int64_t)rb * kPasses * per_pass + (threadIdx.x >> P.lanes_log2);
  if (col >= P.cols) return;
  uint32_t c[kPasses], s[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int64_t r = min(row0 + i * per_pass, P.rows - 1);
    const uint8_t* const from = P.codes + r * (P.padded / 2) + col / 2;
    if constexpr (BF16) {
      c[i] = ldg(reinterpret_cast<const uint32_t*>(from));
    } else {
      c[i] = ldg(reinterpret_cast<const uint16_t*>(from));
    }
    s[i] = ldg(P.scales + r * (P.padded / kMx4Group) + col / kMx4Group);
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int64_t r = row0 + i * per_pass;
    if (r >= P.rows) return;
    const float scale = mx4_scale_float(s[i]);
    const bool bad = s[i] == 255;
    const int64_t at = r * P.ld + col;
    if constexpr (BF16) {
      u32x4 w;
      static_for<4>([&](auto B) __attribute__((always_inline)) {
        constexpr int b = decltype(B)::value;
        w[b] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[i], scale, b));
      });
      if (bad) w = u32x4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
      uint16_t* const o = static_cast<uint16_t*>(P.out) + at;
      if (col + E <= P.cols) {
        stg_any<u32x4, 2>(o, w);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (col + e < P.cols) stg(o + e, (uint16_t)(w[e / 2] >> (16 * (e & 1))));
      }
    } else {
      floatx4 v;
      static_for<2>([&](auto B) __attribute__((always_inline)) {
        constexpr int b = decltype(B)::value;
        const f32x2_t t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], scale, b);
        v[2 * b] = bad ? __builtin_nanf("") : t[0];
        v[2 * b + 1] = bad ? __builtin_nanf("") : t[1];
      });
      float* const o = static_cast<float*>(P.out) + at;
      if (col + E <= P.cols) {
        stg_any<floatx4, 4>(o, v);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (col + e < P.cols) stg(o + e, v[e]);
      }
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
  uint32_t tiles_m, tiles_n;
  // Columns are split over blockIdx.y, split_blocks blocks of 1024 to each; with
  // more than one split C holds one [M][N] partial product after the other.
  int split_blocks;
};

// acc += A B^T over 64 columns for a 32 x 32 block.  Lane l of a wave holds 32
// consecutive columns of one row of each operand (row l % 32, half l / 32 of
// the step) and their scale in byte `SEL` of a dword.  The result's lane l has
// the second operand's row l % 32 and, in element e, the first operand's row
// 8 (e / 4) + 4 (l / 32) + e % 4.
template <int SEL>
__device__ __forceinline__ floatx16 mfma_mx4(const intx4& a, const intx4& b, const floatx16& c, int sa, int sb) {
  const intx8 x = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, y = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, SEL, sa, SEL, sb);
}

// ---------------------------------------------------------------------------
// C = alpha A B^T + beta C on tiles of 64 T x 64 T: 4 waves (2 x 2), each T x T
// blocks of the 32 x 32 x 64 scaled MFMA.  Chunks of 256 columns (128 bytes a row)
// go straight into one of two LDS buffers (global_load_lds_dwordx4) while the
// other is multiplied.
//
//  - Within a chunk lane half h takes the 32-column groups 4 h + s at step s
//    = 0 ... 3, in both operands, so that its 4 scale bytes of a chunk are one
//    dword and the MFMA picks byte s.  (The order of the sum over k is free.)
//  - Scales are staged 1024 columns at a time, a quarter of the next block in
//    each chunk: 8 lanes read 32 bytes of a row.  Taken chunk by chunk (8 bytes a
//    row, 32 cache lines a load) they cost as much of the vector cache's time
//    as half of the codes.
//  - Fragments of the next step are read while the current one multiplies; the
//    barrier between chunks stands before the last step, whose fragments are
//    then in registers.  It frees the chunk's buffer: A's half of the chunk
//    after next is loaded into it under this step's MFMAs, B's under the next's.
//  - 16-byte pieces of a row are permuted by the row (mx4_swz_a, mx4_swz_b), so
//    that the rows a fragment read takes per clock lie in different banks.
//  - B is the MFMA's first operand and its rows are assigned to MFMA rows so
//    that a lane ends with 16 consecutive columns of one row of C.  Each wave
//    turns its 32-row slices through LDS into stores of whole rows.
//  - A workgroup of the 256-tile stays on its compute unit and takes every 256th
//    tile where the columns are whole scale blocks of 1024: the loads ahead of a
//    tile's last chunks are the next tile's, and its stores end under the next
//    tile's MFMAs (8192 x 8192 x 2048 91.4 -> 83.5 us, 8190 x 8190 x 2048 101.8
//    -> 94.7, 16384 x 8192 x 1024 121.8 -> 103.9, 16384 x 2048 x 8192 132.3 -> 129.4,
//    one box, in turn).
//
// Measured, 16384 x 2048 x 8192 to bf16: 128 to 142 us by box and heat, 3.9 to
// 4.3 PFLOP/s.  A launch takes 219 600 cycles, of which the MFMAs take 131 100
// (60%); the rest are waits, the output's among them: there is one wave a SIMD, and
// every chunk ends in a wait for all loads.  The clock is what power leaves: 1.7 to 1.8 GHz on
// random operands, 2.4 on zeros, where the same cycles take 93 us.  Fewer cycles
// alone need not pay: MFMAs fed from registers fall to 1.4 GHz on random operands
// (5.9 PFLOP/s; 9.0 on zeros), and 8 waves a tile, with 5% fewer cycles, took
// the same time.  8192 x 8192 x 2048: 83 to 91 us (3.0 to 3.3 PFLOP/s; MFMAs in
// 44% of the cycles), whose 128 MiB of output take 25 by themselves.
// 1024 x 1024 x 4096 on 64 x 64 tiles: 8.3 us, 1.3 us for 1024 columns.
// ---------------------------------------------------------------------------
constexpr int kMx4Chunk = 256;              // columns
constexpr int kMx4RowBytes = kMx4Chunk / 2;
constexpr int kMx4ScaleDwords = 8;          // of a row and block: 4 chunks

__device__ __forceinline__ int mx4_swz_a(int row) { return (row ^ ((row >> 3) & 3)) & 7; }
// Row of B that MFMA row r (0 ... 31) of a block takes, and its permutation:
// 16 consecutive r cover rows 0-7 and 16-23 of the block (or 8 further on), whose
// even and odd rows lie in different halves of the banks.
__device__ __forceinline__ int mx4_row_b(int r) { return 16 * ((r >> 2) & 1) + 4 * (r >> 3) + (r & 3); }
__device__ __forceinline__ int mx4_swz_b(int row) { return ((row >> 1) & 3) | ((row >> 2) & 4); }

// 16 (4) bytes a lane from memory to consecutive places in LDS.
__device__ __forceinline__ void to_lds16(const uint8_t* from, uint8_t* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}
__device__ __forceinline__ void to_lds4(const uint8_t* from, uint8_t* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (__attribute__((address_space(3))) void*)to, 4, 0, 0);
}

// 4 elements of a row of C at column n (all of them, or those below N).
template <bool BF16, bool WHOLE>
__device__ __forceinline__ floatx4 mx4_load4(const Mx4ProductArgs& P, int64_t m, int64_t n) {
  const uint16_t* const ch = static_cast<const uint16_t*>(P.c) + m * P.ldc + n;
  const float* const cf = static_cast<const float*>(P.c) + m * P.ldc + n;
  floatx4 o = {0.f, 0.f, 0.f, 0.f};
  if (WHOLE || n + 4 <= P.N) {
    if constexpr (BF16) {
      const u32x2 w = ldg_any<u32x2, 2>(ch);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] = __builtin_bit_cast(float, (e & 1) ? (w[e / 2] & 0xffff0000u) : (w[e / 2] << 16));
    } else {
      o = ldg_any<floatx4, 4>(cf);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (n + e < P.N) {
        if constexpr (BF16) {
          o[e] = __builtin_bit_cast(float, (uint32_t)ldg(ch + e) << 16);
        } else {
          o[e] = ldg(cf + e);
        }
      }
    }
  }
  return o;
}

template <bool BF16, bool WHOLE>
__device__ __forceinline__ void mx4_store4(const Mx4ProductArgs& P, int64_t m, int64_t n, const floatx4& v) {
  uint16_t* const ch = static_cast<uint16_t*>(P.c) + m * P.ldc + n;
  float* const cf = static_cast<float*>(P.c) + m * P.ldc + n;
  if (WHOLE || n + 4 <= P.N) {
    if constexpr (BF16) {
      stg_any<u32x2, 2>(ch, u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])});
    } else {
      stg_any<floatx4, 4>(cf, v);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (n + e < P.N) {
        if constexpr (BF16) {
          stg(ch + e, f32_to_bf16_bits(v[e]));
        } else {
          stg(cf + e, v[e]);
        }
      }
    }
  }
}

// Whether a workgroup goes on from tile to tile.  With beta the old values of C
// and the next tile's fragments together pass 512 registers (ten times slower);
// of smaller tiles several workgroups share a compute unit, and overlap anyway.
constexpr bool mx4_streams(int T, bool beta) { return T == 4 && !beta; }

template <int T, bool BF16, bool BETA>
__global__ void __launch_bounds__(256, 1) mx4_product_kernel(const Mx4ProductArgs P) {
  constexpr int BT = 64 * T, NT = 256;                         // tile edge, threads
  constexpr int kData = BT * kMx4RowBytes, kStage = 2 * kData;
  constexpr int kScale = BT * 4 * kMx4ScaleDwords;             // one operand's scale block
  constexpr int LD = kData / (NT * 16);                       // 16-byte loads a thread, operand and chunk
  constexpr int LS = kScale / 2 / (NT * 4);                    // 4-byte scale loads likewise
  constexpr int kSlice = T > 1 ? 64 : 32;                     // columns of a wave's output slice
  constexpr int kLds = 2 * kStage + 4 * kScale;
  static_assert(LD * NT * 16 == kData && LS * NT * 8 == kScale, "chunking");
  constexpr bool kStream = mx4_streams(T, BETA);              // a workgroup may take several tiles
  static_assert(4 * 32 * kSlice * 4 <= (kStream ? kData : kLds) && kLds <= 160 * 1024, "fits the LDS");
  __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];

  // Tiles in groups of 8 tile rows, column by column within a group: the 32
  // tiles that an XCD runs at a time share 8 panels of A and 4 of B.
  const uint32_t tiles = P.tiles_m * P.tiles_n;
  int64_t m0, n0;      // the tile that is multiplied
  int64_t lm, ln;      // the tile that is loaded next
  auto place = [&](uint32_t tile, int64_t& m, int64_t& n) __attribute__((always_inline)) {
    const uint32_t id = xcd_remap(tile, tiles);
    const uint32_t group = id / (8 * P.tiles_n), in_group = id - group * (8 * P.tiles_n);
    const uint32_t rows_here = min(8u, P.tiles_m - 8 * group);
    m = (int64_t)(8 * group + in_group % rows_here) * BT;
    n = (int64_t)(in_group / rows_here) * BT;
  };
  uint32_t tile = blockIdx.x;
  place(tile, m0, n0);

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = (wave >> 1) * 32 * T, wn = (wave & 1) * 32 * T;
  const int r32 = lane & 31, h = lane >> 5;

  const uint32_t pitch = (uint32_t)(P.padded / 2), spitch = (uint32_t)(P.padded / kMx4Group);
  const uint8_t *A, *B, *As, *Bs;
  int ma, nb;  // last valid rows, for the scales
  // Piece c of an operand's chunk: row c / 8, permuted 16-byte column c % 8.
  // Rows past the last one repeat it; they end in rows of C that are not stored.
  uint32_t offA[LD], offB[LD];
  auto aim_a = [&](int64_t m) __attribute__((always_inline)) {
    A = P.a + m * pitch + (int64_t)blockIdx.y * P.split_blocks * 512;
    const int limit = (int)min<int64_t>(BT, P.M - m) - 1;
#pragma unroll
    for (int it = 0; it < LD; ++it) {
      const int c = it * NT + tid, row = c >> 3;
      offA[it] = (uint32_t)min(row, limit) * pitch + 16 * ((c & 7) ^ mx4_swz_a(row));
    }
  };
  auto aim_b = [&](int64_t n) __attribute__((always_inline)) {
    B = P.b + n * pitch + (int64_t)blockIdx.y * P.split_blocks * 512;
    const int limit = (int)min<int64_t>(BT, P.N - n) - 1;
#pragma unroll
    for (int it = 0; it < LD; ++it) {
      const int c = it * NT + tid, row = c >> 3;
      offB[it] = (uint32_t)min(row, limit) * pitch + 16 * ((c & 7) ^ mx4_swz_b(row));
    }
  };
  auto aim_scales = [&](int64_t m, int64_t n) __attribute__((always_inline)) {
    As = P.as + m * spitch + (int64_t)blockIdx.y * P.split_blocks * 32;
    Bs = P.bs + n * spitch + (int64_t)blockIdx.y * P.split_blocks * 32;
    ma = (int)min<int64_t>(BT, P.M - m) - 1;
    nb = (int)min<int64_t>(BT, P.N - n) - 1;
  };
  aim_a(m0);
  aim_b(n0);
  aim_scales(m0, n0);
  // This split's 128-column halves of chunks, and its whole chunks.
  const int steps = min((int)(P.padded / 128) - (int)blockIdx.y * P.split_blocks * 8, P.split_blocks * 8);
  const int full = steps / 2;
  auto issue_a = [&](int buf, int chunk) __attribute__((always_inline)) {
    const uint8_t* const a = A + (int64_t)chunk * kMx4RowBytes;
#pragma unroll
    for (int it = 0; it < LD; ++it) to_lds16(a + offA[it], lds + buf + (it * NT + wave * 64) * 16);
  };
  auto issue_b = [&](int buf, int chunk) __attribute__((always_inline)) {
    const uint8_t* const b = B + (int64_t)chunk * kMx4RowBytes;
#pragma unroll
    for (int it = 0; it < LD; ++it) to_lds16(b + offB[it], lds + buf + kData + (it * NT + wave * 64) * 16);
  };
  // Quarter q of scale block blk, to the place of blocks of its parity: 32 T rows
  // of A (q = 0, 1) or B.  Dword p of a row goes to place p ^ 2 ((row / 8) % 4), so that the rows of a read, 8
  // dwords apart, spread over the banks.
  const int last = steps - 1;
  auto issue_scales = [&](int blk, int parity, int q) __attribute__((always_inline)) {
    const uint8_t* const from = q < 2 ? As : Bs;
    const int limit = q < 2 ? ma : nb;
    const uint32_t col = 4 * min(blk * kMx4ScaleDwords + ((tid & 7) ^ (2 * wave)), last);
    uint8_t* const to = lds + 2 * kStage + (parity & 1) * 2 * kScale;
#pragma unroll
    for (int it = 0; it < LS; ++it) {
      const uint32_t row = (uint32_t)min(((q & 1) * LS + it) * (NT / 8) + (tid >> 3), limit);
      to_lds4(from + row * spitch + col, to + ((q * LS + it) * NT + wave * 64) * 4);
    }
  };
  // The 128 columns after the whole chunks: pieces of the missing half re-read
  // the first one and are not used.  Their scales are the last dword of a row.
  auto issue_half = [&](int buf) __attribute__((always_inline)) {
    const int64_t k = (int64_t)full * kMx4RowBytes;
#pragma unroll
    for (int it = 0; it < LD; ++it) {
      const int c = it * NT + tid, row = c >> 3;
      const uint32_t upA = (c ^ mx4_swz_a(row)) & 4, upB = (c ^ mx4_swz_b(row)) & 4;
      to_lds16(A + k + (offA[it] - 16 * upA), lds + buf + (it * NT + wave * 64) * 16);
      to_lds16(B + k + (offB[it] - 16 * upB), lds + buf + kData + (it * NT + wave * 64) * 16);
    }
  };

  floatx16 acc[T][T];
#pragma unroll
  for (int i = 0; i < T; ++i)
#pragma unroll
    for (int j = 0; j < T; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  const int rb = mx4_row_b(r32);
  // LDS offsets of this lane's rows in a stage and in a scale block
  const int rowA = (wm + r32) * kMx4RowBytes, rowB = kData + (wn + rb) * kMx4RowBytes;
  const int swzA = mx4_swz_a(r32), swzB = mx4_swz_b(rb);
  const int scaleA = 2 * kStage + (wm + r32) * 4 * kMx4ScaleDwords;
  const int scaleB = 2 * kStage + kScale + (wn + rb) * 4 * kMx4ScaleDwords;
  constexpr int kBlock = 32 * kMx4RowBytes, kBlockScales = 32 * 4 * kMx4ScaleDwords;

  intx4 fa[2][T], fb[2][T];
  int sa[T], sb[T];
  auto read = [&](int buf, int slot, int q) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < T; ++i)
      fa[slot][i] = *reinterpret_cast<const intx4*>(lds + buf + rowA + i * kBlock + 16 * (q ^ swzA));
#pragma unroll
    for (int j = 0; j < T; ++j)
      fb[slot][j] = *reinterpret_cast<const intx4*>(lds + buf + rowB + j * kBlock + 16 * (q ^ swzB));
  };
  // This lane's scales at dword p of scale block parity blk.
  auto read_scales = [&](int blk, int p) __attribute__((always_inline)) {
    const int base = (blk & 1) * 2 * kScale;
    const int pa = 4 * (p ^ (2 * ((r32 >> 3) & 3))), pb = 4 * (p ^ (2 * ((rb >> 3) & 3)));
#pragma unroll
    for (int i = 0; i < T; ++i) sa[i] = *reinterpret_cast<const int*>(lds + base + scaleA + i * kBlockScales + pa);
#pragma unroll
    for (int j = 0; j < T; ++j) sb[j] = *reinterpret_cast<const int*>(lds + base + scaleB + j * kBlockScales + pb);
  };
  constexpr int kWaitAll = 0 | (7 << 4);            // vmcnt(0) lgkmcnt(0)
  constexpr int kWaitLds = 0xc00f | (7 << 4);       // lgkmcnt(0)
  auto meet = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(kWaitAll);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };

  if (full > 0) {
    issue_a(0, 0);
    issue_b(0, 0);
#pragma unroll
    for (int q = 0; q < 4; ++q) issue_scales(0, 0, q);
  }
  if (steps & 1) {
    issue_half(kStage);
#pragma unroll
    for (int q = 0; q < 4; ++q) issue_scales((full / 4) | 1, 1, q);  // clamped to the last dword
  }
  meet();
  if (steps & 1) {  // lane half h takes groups 2 h and 2 h + 1
    read_scales(1, min((((full / 4) | 1) * kMx4ScaleDwords), last) == last ? 0 : 2 * (full % 4));
#pragma unroll
    for (int i = 0; i < T; ++i) sa[i] = sa[i] >> (16 * h);
#pragma unroll
    for (int j = 0; j < T; ++j) sb[j] = sb[j] >> (16 * h);
    static_for<2>([&](auto S) __attribute__((always_inline)) {
      constexpr int s = decltype(S)::value;
      read(kStage, s, 2 * h + s);
#pragma unroll
      for (int i = 0; i < T; ++i)
#pragma unroll
        for (int j = 0; j < T; ++j) acc[i][j] = mfma_mx4<s>(fb[s][j], fa[s][i], acc[i][j], sb[j], sa[i]);
    });
    meet();
  }
  int cur = 0, block = 0;  // buffer of the next chunk; scale blocks before this tile's
  if (full > 0) {
    issue_a(kStage, min(1, full - 1));
    read_scales(0, h);
    read(0, 0, 4 * h);
  }
  for (;;) {
    // The chunks of this workgroup's tiles are one stream: the loads that run
    // ahead of a tile's last chunks are the next tile's first ones (its own first
    // ones again after the last tile, into buffers that nothing reads any more).
    const uint32_t next = tile + gridDim.x;
    const bool more = kStream && next < tiles;
    lm = m0;
    ln = n0;
    if (more) place(next, lm, ln);
    for (int c = 0; c < full; ++c) {
      if constexpr (kStream) {
        if (c + 4 == full) aim_scales(lm, ln);
        if (c + 2 == full) aim_a(lm);
        if (c + 1 == full) aim_b(ln);
      }
      const int other = kStage - cur;
      const int ahead1 = kStream && c + 1 == full ? 0 : min(c + 1, full - 1);
      const int ahead2 = min(kStream && c + 2 >= full ? c + 2 - full : c + 2, full - 1);
      const int ahead_scales = kStream && 4 * (c / 4 + 1) >= full ? 0 : c / 4 + 1;
      int ta[T], tb[T];
#pragma unroll
      for (int i = 0; i < T; ++i) ta[i] = sa[i];
#pragma unroll
      for (int j = 0; j < T; ++j) tb[j] = sb[j];
      static_for<4>([&](auto S) __attribute__((always_inline)) {
        constexpr int s = decltype(S)::value;
        constexpr int kReads = 2 * T, kMfma = T * T;
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (s == 0) issue_b(other, ahead1);
        if constexpr (s == 1) issue_scales(ahead_scales, block + c / 4 + 1, c % 4);
        if constexpr (s < 3) {
          read(cur, (s + 1) & 1, 4 * h + s + 1);
        } else {
          meet();
          issue_a(cur, ahead2);
          read_scales(block + (c + 1) / 4, 2 * ((c + 1) % 4) + h);
          read(other, 0, 4 * h);
        }
#pragma unroll
        for (int i = 0; i < T; ++i)
#pragma unroll
          for (int j = 0; j < T; ++j)
            acc[i][j] = mfma_mx4<s>(fb[s & 1][j], fa[s & 1][i], acc[i][j], tb[j], ta[i]);
        // one MFMA, one LDS read, and so on; then the loads
        static_for<(kReads < kMfma ? kReads : kMfma)>([&](auto) __attribute__((always_inline)) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, s < 3 ? 1 : 2, 0);
        });
        static_for<4>([&](auto) __attribute__((always_inline)) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x020, s == 1 ? (LS + 3) / 4 : (LD + 3) / 4, 0);
        });
        __builtin_amdgcn_sched_barrier(0);
      });
      cur = other;
    }

    // Output: 32 rows of kSlice columns of C at a time through this wave's slice
    // of LDS, 16-byte pieces permuted by the row.  A stream's slices lie in B's
    // half of the last chunk's buffer: the next tile's loads reach it only after
    // the barrier below.
    if constexpr (!kStream) meet();
    // no loads into LDS may be left when the workgroup ends
    if (kStream && !more) __builtin_amdgcn_s_waitcnt(kWaitAll);
    uint8_t* const slice = lds + (kStream ? kStage - cur + kData : 0) + wave * 32 * kSlice * 4;
    auto output = [&](auto WHOLE) __attribute__((always_inline)) {
      constexpr bool kWhole = decltype(WHOLE)::value;
      constexpr int kLanes = kSlice / 4, kRows = 64 / kLanes, kIter = 32 / kRows;  // kLanes lanes hold a row, 4 elements each
      const int piece = lane % kLanes, row0 = lane / kLanes;
#pragma unroll
      for (int i = 0; i < T; ++i) {
#pragma unroll
        for (int part = 0; part < 32 * T / kSlice; ++part) {
          const int64_t n = n0 + wn + part * kSlice + 4 * piece;
          const int64_t mi = m0 + wm + 32 * i + row0, split = (int64_t)blockIdx.y * P.M;
          // all of C's loads first: none can pass a store
          floatx4 old[BETA ? kIter : 1];
          if constexpr (BETA) {
#pragma unroll
            for (int r = 0; r < kIter; ++r)
              if (kWhole || (mi + r * kRows < P.M && n < P.N)) old[r] = mx4_load4<BF16, kWhole>(P, mi + r * kRows, n);
          }
#pragma unroll
          for (int jj = 0; jj < kSlice / 32; ++jj) {
            const int j = part * (kSlice / 32) + jj;
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<floatx4*>(slice + r32 * kSlice * 4 + 16 * ((8 * jj + 4 * h + q) ^ (r32 & (kLanes - 1)))) =
                  floatx4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          }
          floatx4 v[kIter];
#pragma unroll
          for (int r = 0; r < kIter; ++r) {
            const int row = r * kRows + row0;
            v[r] = *reinterpret_cast<const floatx4*>(slice + row * kSlice * 4 + 16 * (piece ^ (row & (kLanes - 1))));
          }
#pragma unroll
          for (int r = 0; r < kIter; ++r) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[r][e] *= P.alpha;
              if constexpr (BETA) v[r][e] += P.beta * old[r][e];
            }
            if (kWhole || (mi + r * kRows < P.M && n < P.N)) mx4_store4<BF16, kWhole>(P, split + mi + r * kRows, n, v[r]);
          }
        }
      }
    };
    if (m0 + BT <= P.M && n0 + BT <= P.N) {
      output(std::true_type{});
    } else {
      output(std::false_type{});
    }
    if (!more) return;

#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
      for (int j = 0; j < T; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    tile = next;
    m0 = lm;
    n0 = ln;
    block += full / 4;
    // every wave has read its slice; the stores are left under way
    __builtin_amdgcn_s_waitcnt(kWaitLds);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

// ---------------------------------------------------------------------------
// Few rows (M <= 16): the weight-streaming form, bound by the bytes of B (or by
// latency).  A workgroup takes 16 NT rows of B; its 4 waves split the columns
// and add their partial sums through LDS in a fixed order.  Lane l holds, at
// each 128-column step, columns 32 (l / 16) onwards of B's row l % 16 and of A's
// row l % 16.  A wave works in batches of BATCH steps, whose scales are one load
// of 4 BATCH bytes a row: read byte by byte they cost as many cache lines as
// the codes.  A may still be fp32 or bf16 (at most kMx4FewElems elements): then
// the workgroup quantises it into LDS while its first rows of B are on their
// way, which saves a launch and A's way through memory.  Measured, one bf16 row
// by 8192 x 2048: 4.2 us (a launch alone takes 2), by 8192 x 8192: 9.0 us
// (4.2 TB/s); 16 rows by 8192 x 8192, B read for two tiles at a time: 10.4 us.
// ---------------------------------------------------------------------------
enum { MX4_A_MX4 = 0, MX4_A_F32 = 1, MX4_A_BF16 = 2 };
constexpr int kMx4FewElems = 16384;

struct Mx4FewArgs {
  Mx4ProductArgs p;
  const void* x;  // A before quantisation
  int64_t ldx, K;
};

__device__ __forceinline__ floatx4 mfma_mx4_16(const intx4& a, const intx4& b, const floatx4& c, int sa, int sb) {
  const intx8 x = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, y = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 0, sa, 0, sb);
}

template <int AM, int NT, int BATCH>
__global__ void __launch_bounds__(256) mx4_few_rows_kernel(const Mx4FewArgs Q) {
  typedef uint32_t Scales __attribute__((ext_vector_type(BATCH)));
  const Mx4ProductArgs& P = Q.p;
  constexpr int W = 4;
  __shared__ float part[W][16][16 * NT + 1];
  __shared__ __attribute__((aligned(16))) uint8_t qa[AM == MX4_A_MX4 ? 16 : kMx4FewElems / 2 + kMx4FewElems / kMx4Group];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16 * NT;
  // The wave's steps: whole batches but for the matrix's last steps.
  const int steps = (int)(P.padded / 128), batches = (steps + BATCH - 1) / BATCH;
  const int s0 = batches * wave / W * BATCH, s1 = min(batches * (wave + 1) / W * BATCH, steps);
  int64_t brow[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) brow[j] = min(n0 + 16 * j + r16, P.N - 1) * P.padded;
  const int64_t arow = min<int64_t>(r16, P.M - 1) * P.padded;
  floatx4 acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = floatx4{0.f, 0.f, 0.f, 0.f};

  intx4 b[BATCH][NT], a[BATCH];
  Scales sb[NT], sa;
  auto load_whole = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int64_t k = (int64_t)(s + u) * 128 + 32 * g;
#pragma unroll
      for (int j = 0; j < NT; ++j) b[u][j] = ldg(reinterpret_cast<const intx4*>(P.b + (brow[j] + k) / 2));
      if constexpr (AM == MX4_A_MX4) a[u] = ldg(reinterpret_cast<const intx4*>(P.a + (arow + k) / 2));
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) sb[j] = ldg_any<Scales, 4>(P.bs + (brow[j] + s * 128) / kMx4Group);
    if constexpr (AM == MX4_A_MX4) sa = ldg_any<Scales, 4>(P.as + (arow + s * 128) / kMx4Group);
  };
  auto multiply = [&](int s, int u, const intx4& av, uint32_t sav, const intx4 (&bv)[NT], const uint32_t (&sbv)[NT])
      __attribute__((always_inline)) {
    intx4 x = av;
    uint32_t sx = sav >> (8 * g);
    if constexpr (AM != MX4_A_MX4) {
      const int at = min(r16, (int)P.M - 1) * (int)P.padded + (s + u) * 128 + 32 * g;
      x = *reinterpret_cast<const intx4*>(qa + at / 2);
      sx = qa[kMx4FewElems / 2 + at / kMx4Group];
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = mfma_mx4_16(bv[j], x, acc[j], (int)(sbv[j] >> (8 * g)), (int)sx);
  };

  const bool first = s0 + BATCH <= s1;
  if (first) load_whole(s0);
  if constexpr (AM != MX4_A_MX4) {
    // 8 elements a lane, 4 lanes a group
    const int per_row = (int)(P.padded / 8), pieces = (int)P.M * per_row;
    for (int q = threadIdx.x; q < pieces; q += 256) {
      const int row = q / per_row, k = (q - row * per_row) * 8;
      Mx4Piece<AM == MX4_A_BF16, 8> x;
      x.load_edge(Q.x, P.M, Q.K, Q.ldx, row, k);
      const uint32_t s = mx4_scale(group_max<4>(x.top())), c = x.encode(mx4_scale_float(s));
      *reinterpret_cast<uint32_t*>(qa + 4 * q) = s == 255 ? 0u : c;
      if ((q & 3) == 0) qa[kMx4FewElems / 2 + q / 4] = (uint8_t)s;
    }
    __syncthreads();
  }
  int s = s0;
  if (first) {
    for (;;) {
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        uint32_t t[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) t[j] = sb[j][u];
        multiply(s, u, a[u], sa[u], b[u], t);
      }
      s += BATCH;
      if (s + BATCH > s1) break;
      load_whole(s);
    }
  }
  for (; s < s1; ++s) {  // fewer than BATCH steps at the end of the matrix
    const int64_t k = (int64_t)s * 128;
    intx4 bv[NT], av = {0, 0, 0, 0};
    uint32_t t[NT], ta = 0;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      bv[j] = ldg(reinterpret_cast<const intx4*>(P.b + (brow[j] + k + 32 * g) / 2));
      t[j] = ldg(reinterpret_cast<const uint32_t*>(P.bs + (brow[j] + k) / kMx4Group));
    }
    if constexpr (AM == MX4_A_MX4) {
      av = ldg(reinterpret_cast<const intx4*>(P.a + (arow + k + 32 * g) / 2));
      ta = ldg(reinterpret_cast<const uint32_t*>(P.as + (arow + k) / kMx4Group));
    }
    multiply(s, 0, av, ta, bv, t);
  }
  // Lane l has columns n0 + 16 j + 4 g ... of C's row l % 16.
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[wave][r16][16 * j + 4 * g + e] = acc[j][e];
  __syncthreads();
  for (int q = threadIdx.x; q < NT * 256; q += 256) {
    const int col = q % (16 * NT);
    const int64_t m = q / (16 * NT), n = n0 + col;
    if (m >= P.M || n >= P.N) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += part[w][m][col];
    v *= P.alpha;
    const int64_t at = m * P.ldc + n;
    if (P.bf16) {
      uint16_t* const c = static_cast<uint16_t*>(P.c) + at;
      if (P.beta != 0.f) v += P.beta * __builtin_bit_cast(float, (uint32_t)ldg(c) << 16);
      stg(c, f32_to_bf16_bits(v));
    } else {
      float* const c = static_cast<float*>(P.c) + at;
      if (P.beta != 0.f) v += P.beta * ldg(c);
      stg(c, v);
    }
  }
}

// C = alpha sum + beta C over the partial products of a split, in their order:
// 2.5 us with its launch; 64 x 2048 x 8192 takes 6.7 us in 8 splits, 13.5 in one.
struct Mx4SumArgs {
  Mx4ProductArgs p;
  const float* parts;  // [splits][M][N]
  int splits;
};

__global__ void __launch_bounds__(256) mx4_sum_kernel(const Mx4SumArgs Q) {
  const Mx4ProductArgs& P = Q.p;
  const uint32_t total = (uint32_t)(P.M * P.N), id = blockIdx.x * 256 + threadIdx.x;  // a split is of small C only
  if (id >= total) return;
  float v = 0.f;
#pragma unroll 4
  for (int s = 0; s < Q.splits; ++s) v += ldg(Q.parts + (int64_t)s * total + id);
  v *= P.alpha;
  const uint32_t m = id / (uint32_t)P.N;
  const int64_t at = m * P.ldc + (id - m * (uint32_t)P.N);
  if (P.bf16) {
    uint16_t* const c = static_cast<uint16_t*>(P.c) + at;
    if (P.beta != 0.f) v += P.beta * __builtin_bit_cast(float, (uint32_t)ldg(c) << 16);
    stg(c, f32_to_bf16_bits(v));
  } else {
    float* const c = static_cast<float*>(P.c) + at;
    if (P.beta != 0.f) v += P.beta * ldg(c);
    stg(c, v);
  }
}

}  // namespace shp
