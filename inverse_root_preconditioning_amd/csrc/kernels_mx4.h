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
  uint32_t tiles_m, tiles_n;
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
// blocks of the 32 x 32 x 64 scaled MFMA.  Chunks of 256 columns (128 bytes a row,
// 8 scale bytes) go straight into one of two LDS buffers
// (global_load_lds_dwordx4) while the other is multiplied.
//
//  - Within a chunk lane half h takes the 32-column groups 4 h + s at step s
//    = 0 ... 3, in both operands, so that its 4 scale bytes of a chunk are one
//    dword and the MFMA picks byte s.  (The order of the sum over k is free.)
//  - Fragments of the next step are read while the current one multiplies; the
//    barrier between chunks stands before the last step, whose fragments are
//    then in registers: it frees the chunk's buffer for the loads after next
//    and lets the next chunk's first fragments be read under that step's MFMAs.
//  - 16-byte pieces of a row are permuted by the row (mx4_swz_a, mx4_swz_b), so
//    that the 8 rows a fragment read takes per clock lie in different banks.
//  - B is the MFMA's first operand and its rows are assigned to MFMA rows so
//    that a lane ends with 16 consecutive columns of one row of C.
// ---------------------------------------------------------------------------
constexpr int kMx4Chunk = 256;              // columns
constexpr int kMx4RowBytes = kMx4Chunk / 2;
constexpr int kMx4RowScales = kMx4Chunk / kMx4Group;

__device__ __forceinline__ int mx4_swz_a(int row) { return (row ^ ((row >> 3) & 3)) & 7; }
// Row of B that MFMA row r (0 ... 31) of a block takes, and its permutation:
// 8 consecutive r cover rows 0-3 and 16-19 of the block (plus a multiple of 4).
__device__ __forceinline__ int mx4_row_b(int r) { return 16 * ((r >> 2) & 1) + 4 * (r >> 3) + (r & 3); }
__device__ __forceinline__ int mx4_swz_b(int row) { return (row & 3) | ((row >> 2) & 4); }

// 16 consecutive elements of a row of C at column n (all of them, or those below N).
template <bool BF16, bool BETA, bool WHOLE>
__device__ __forceinline__ void mx4_store16(const Mx4ProductArgs& P, int64_t m, int64_t n, const floatx16& v) {
  const int64_t at = m * P.ldc + n;
  uint16_t* const ch = static_cast<uint16_t*>(P.c) + at;
  float* const cf = static_cast<float*>(P.c) + at;
  if constexpr (!WHOLE) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      if (n + e < P.N) {
        float o = P.alpha * v[e];
        if constexpr (BF16) {
          if constexpr (BETA) o += P.beta * __builtin_bit_cast(float, (uint32_t)ldg(ch + e) << 16);
          stg(ch + e, f32_to_bf16_bits(o));
        } else {
          if constexpr (BETA) o += P.beta * ldg(cf + e);
          stg(cf + e, o);
        }
      }
    }
  } else if constexpr (BF16) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      u32x4 old = {0, 0, 0, 0};
      if constexpr (BETA) old = ldg_any<u32x4, 2>(ch + 8 * q);
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float lo = P.alpha * v[8 * q + 2 * e], hi = P.alpha * v[8 * q + 2 * e + 1];
        if constexpr (BETA) {
          lo += P.beta * __builtin_bit_cast(float, old[e] << 16);
          hi += P.beta * __builtin_bit_cast(float, old[e] & 0xffff0000u);
        }
        w[e] = pack_bf16x2(lo, hi);
      }
      stg_any<u32x4, 2>(ch + 8 * q, w);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      floatx4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = P.alpha * v[4 * q + e];
      if constexpr (BETA) {
        const floatx4 old = ldg_any<floatx4, 4>(cf + 4 * q);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += P.beta * old[e];
      }
      stg_any<floatx4, 4>(cf + 4 * q, o);
    }
  }
}

// 16 (4) bytes a lane from memory to consecutive places in LDS.
__device__ __forceinline__ void to_lds16(const uint8_t* from, uint8_t* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}
__device__ __forceinline__ void to_lds4(const uint8_t* from, uint8_t* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (__attribute__((address_space(3))) void*)to, 4, 0, 0);
}

template <int T, bool BF16, bool BETA>
__global__ void __launch_bounds__(256, 1) mx4_product_kernel(const Mx4ProductArgs P) {
  constexpr int BT = 64 * T;                                   // tile edge
  constexpr int kData = BT * kMx4RowBytes, kScale = BT * kMx4RowScales;
  constexpr int kStage = 2 * (kData + kScale);                 // A, B, their scales
  constexpr int LD = kData / (256 * 16);                       // 16-byte loads a thread, operand and chunk
  constexpr int kScaleLoads = 2 * kScale / (256 * 4);          // of both operands
  static_assert(LD * 256 * 16 == kData && kScaleLoads * 256 * 4 == 2 * kScale, "chunking");
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kStage];

  // Tiles in groups of 8 tile rows, column by column within a group: the 32
  // tiles that an XCD runs at a time share 8 panels of A and 4 of B.
  const uint32_t id = xcd_remap(blockIdx.x, gridDim.x);
  const uint32_t group = id / (8 * P.tiles_n), in_group = id - group * (8 * P.tiles_n);
  const uint32_t rows_here = min(8u, P.tiles_m - 8 * group);
  const int64_t m0 = (int64_t)(8 * group + in_group % rows_here) * BT, n0 = (int64_t)(in_group / rows_here) * BT;

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = (wave >> 1) * 32 * T, wn = (wave & 1) * 32 * T;
  const int r32 = lane & 31, h = lane >> 5;

  const uint32_t pitch = (uint32_t)(P.padded / 2), spitch = (uint32_t)(P.padded / kMx4Group);
  const uint8_t* const A = P.a + m0 * pitch;
  const uint8_t* const B = P.b + n0 * pitch;
  const uint8_t* const As = P.as + m0 * spitch;
  const uint8_t* const Bs = P.bs + n0 * spitch;
  const int ma = (int)min<int64_t>(BT, P.M - m0) - 1, nb = (int)min<int64_t>(BT, P.N - n0) - 1;  // last valid rows

  // Piece c of an operand's chunk: row c / 8, permuted 16-byte column c % 8.
  uint32_t offA[LD], offB[LD], offS[kScaleLoads];
#pragma unroll
  for (int it = 0; it < LD; ++it) {
    const int c = it * 256 + tid, row = c >> 3;
    offA[it] = (uint32_t)min(row, ma) * pitch + 16 * ((c & 7) ^ mx4_swz_a(row));
    offB[it] = (uint32_t)min(row, nb) * pitch + 16 * ((c & 7) ^ mx4_swz_b(row));
  }
#pragma unroll
  for (int it = 0; it < kScaleLoads; ++it) {
    const int d = it * 256 + tid;  // dword d: row d / 2 of A, then of B
    offS[it] = (uint32_t)(d < 2 * BT ? min(d >> 1, ma) : min((d >> 1) - BT, nb)) * spitch + 4 * (d & 1);
  }
  const int steps = (int)(P.padded / 128);  // 128-column halves of chunks
  const int full = steps / 2;               // whole chunks
  // With one dword a thread covers both operands' scales when T = 1: the
  // operand then differs between the waves, which is uniform within one.
  auto scale_base = [&](int it) __attribute__((always_inline)) { return it * 256 + wave * 64 < 2 * BT ? As : Bs; };
  auto issue_a = [&](uint8_t* base, int chunk) __attribute__((always_inline)) {
    const uint8_t* const a = A + (int64_t)chunk * kMx4RowBytes;
#pragma unroll
    for (int it = 0; it < LD; ++it) to_lds16(a + offA[it], base + (it * 256 + wave * 64) * 16);
  };
  auto issue_b = [&](uint8_t* base, int chunk) __attribute__((always_inline)) {
    const uint8_t* const b = B + (int64_t)chunk * kMx4RowBytes;
#pragma unroll
    for (int it = 0; it < LD; ++it) to_lds16(b + offB[it], base + kData + (it * 256 + wave * 64) * 16);
#pragma unroll
    for (int it = 0; it < kScaleLoads; ++it)
      to_lds4(scale_base(it) + (int64_t)chunk * kMx4RowScales + offS[it],
             base + 2 * kData + (it * 256 + wave * 64) * 4);
  };
  // The 128 columns after the whole chunks: pieces and scales of the missing
  // half re-read the first one and are not used.
  auto issue_half = [&](uint8_t* base) __attribute__((always_inline)) {
    const int64_t k = (int64_t)full * kMx4RowBytes, ks = (int64_t)full * kMx4RowScales;
#pragma unroll
    for (int it = 0; it < LD; ++it) {
      const int c = it * 256 + tid, row = c >> 3;
      const uint32_t upA = (c ^ mx4_swz_a(row)) & 4, upB = (c ^ mx4_swz_b(row)) & 4;
      to_lds16(A + k + (offA[it] - 16 * upA), base + (it * 256 + wave * 64) * 16);
      to_lds16(B + k + (offB[it] - 16 * upB), base + kData + (it * 256 + wave * 64) * 16);
    }
#pragma unroll
    for (int it = 0; it < kScaleLoads; ++it)
      to_lds4(scale_base(it) + ks + offS[it] - 4 * (tid & 1), base + 2 * kData + (it * 256 + wave * 64) * 4);
  };

  floatx16 acc[T][T];
#pragma unroll
  for (int i = 0; i < T; ++i)
#pragma unroll
    for (int j = 0; j < T; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  const int rb = mx4_row_b(r32);
  // LDS offsets of this lane's fragments (piece 0 of its half) and scales
  const int fragA = (wm + r32) * kMx4RowBytes, swzA = mx4_swz_a(r32);
  const int fragB = kData + (wn + rb) * kMx4RowBytes, swzB = mx4_swz_b(rb);
  const int scaleA = 2 * kData + (wm + r32) * kMx4RowScales, scaleB = 2 * kData + kScale + (wn + rb) * kMx4RowScales;
  constexpr int kBlock = 32 * kMx4RowBytes, kBlockScales = 32 * kMx4RowScales;

  constexpr int kWaitAll = 0 | (7 << 4);  // vmcnt(0) lgkmcnt(0)
  auto meet = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(kWaitAll);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };
  intx4 fa[2][T], fb[2][T];
  int sa[T], sb[T];
  auto read = [&](const uint8_t* base, int slot, int q) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < T; ++i)
      fa[slot][i] = *reinterpret_cast<const intx4*>(base + fragA + i * kBlock + 16 * (q ^ swzA));
#pragma unroll
    for (int j = 0; j < T; ++j)
      fb[slot][j] = *reinterpret_cast<const intx4*>(base + fragB + j * kBlock + 16 * (q ^ swzB));
  };

  if (full > 0) {
    issue_a(lds, 0);
    issue_b(lds, 0);
  }
  if (steps & 1) issue_half(lds + kStage);
  meet();
  if (steps & 1) {  // lane half h takes groups 2 h and 2 h + 1
    const uint8_t* const base = lds + kStage;
#pragma unroll
    for (int i = 0; i < T; ++i)
      sa[i] = *reinterpret_cast<const uint16_t*>(base + scaleA + i * kBlockScales + 2 * h);
#pragma unroll
    for (int j = 0; j < T; ++j)
      sb[j] = *reinterpret_cast<const uint16_t*>(base + scaleB + j * kBlockScales + 2 * h);
    static_for<2>([&](auto S) __attribute__((always_inline)) {
      constexpr int s = decltype(S)::value;
      read(base, s, 2 * h + s);
#pragma unroll
      for (int i = 0; i < T; ++i)
#pragma unroll
        for (int j = 0; j < T; ++j) acc[i][j] = mfma_mx4<s>(fb[s][j], fa[s][i], acc[i][j], sb[j], sa[i]);
    });
    meet();
  }
  if (full > 0) {
    // Loads past the last chunk repeat it into the buffer that nothing reads any more.
    issue_a(lds + kStage, min(1, full - 1));
    issue_b(lds + kStage, min(1, full - 1));
    uint32_t cur = 0;
    auto read_scales = [&](const uint8_t* base) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < T; ++i)
        sa[i] = *reinterpret_cast<const int*>(base + scaleA + i * kBlockScales + 4 * h);
#pragma unroll
      for (int j = 0; j < T; ++j)
        sb[j] = *reinterpret_cast<const int*>(base + scaleB + j * kBlockScales + 4 * h);
    };
    read_scales(lds);
    read(lds, 0, 4 * h);
    for (int c = 0; c < full; ++c) {
      const uint8_t* const base = lds + cur;
      uint8_t* const other = lds + (kStage - cur);
      int ta[T], tb[T];
#pragma unroll
      for (int i = 0; i < T; ++i) ta[i] = sa[i];
#pragma unroll
      for (int j = 0; j < T; ++j) tb[j] = sb[j];
      static_for<4>([&](auto S) __attribute__((always_inline)) {
        constexpr int s = decltype(S)::value;
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (s < 3) {
          read(base, (s + 1) & 1, 4 * h + s + 1);
        } else {
          meet();
          issue_a(lds + cur, min(c + 2, full - 1));
          issue_b(lds + cur, min(c + 2, full - 1));
          read_scales(other);
          read(other, 0, 4 * h);
        }
#pragma unroll
        for (int i = 0; i < T; ++i)
#pragma unroll
          for (int j = 0; j < T; ++j)
            acc[i][j] = mfma_mx4<s>(fb[s & 1][j], fa[s & 1][i], acc[i][j], tb[j], ta[i]);
        if constexpr (s < 3) {
          constexpr int kPairs = 2 * T < T * T ? 2 * T : T * T;
          static_for<kPairs>([&](auto) __attribute__((always_inline)) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          });
          if constexpr (T * T > kPairs) __builtin_amdgcn_sched_group_barrier(0x008, T * T - kPairs, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      });
      cur = kStage - cur;
    }
  }

  const bool whole = m0 + BT <= P.M && n0 + BT <= P.N;
#pragma unroll
  for (int i = 0; i < T; ++i) {
    const int64_t m = m0 + wm + 32 * i + r32;
#pragma unroll
    for (int j = 0; j < T; ++j) {
      const int64_t n = n0 + wn + 32 * j + 16 * h;
      if (whole) {
        mx4_store16<BF16, BETA, true>(P, m, n, acc[i][j]);
      } else if (m < P.M && n < P.N) {
        mx4_store16<BF16, BETA, false>(P, m, n, acc[i][j]);
      }
    }
  }
}

}  // namespace shp
