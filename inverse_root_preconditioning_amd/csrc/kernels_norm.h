// Norms over rows and the join of a block's output y with its residual r,
//   z = N1(y),  h = scale r + gate z,  u = N2(h),
// with their gradients.  N(x) = (x - mean) s w + b, s = 1 / sqrt(mean of squares
// (RMS: mean = 0) or variance (layer) + eps); either norm may be absent, and
// the norm alone is the join without y: h = r.
//
// W waves hold a row of up to 64 W P V columns in registers, each lane P pieces
// of V consecutive elements, so that a row is read once however many sums over
// it the formulas need.
#pragma once

#include "kernels_mx8.h"

namespace shp {

// A norm's parameters; kind SHAMPOO_NORM_NONE: there is none.
struct NormSide {
  const void *w, *b;
  int kind, w_bf16, b_bf16;
  float eps;
};

struct JoinArgs {
  int64_t rows;
  uint32_t cols;
  float scale;
  const void *r, *y;  // the inputs; y unused without a join
  int64_t ldr, ldy;
  Mx8Rows kr, ky;     // their MX8 copies: written forward where codes is given, read backward with KEEP
  NormSide after, before;
  const void* gate;
  int gate_kind, gate_bf16;
  uint32_t gate_rows;        // rows that share a row of the gate
  float *stats1, *stats2;    // [rows][2]: mean and s of N1 and of N2
  // forward
  void *h, *u;
  int64_t ldh, ldu;
  // backward
  const void *dh, *du;
  int64_t lddh, lddu;
  void *dr, *dy, *dtoken;
  int64_t lddr, lddy;
  int dtoken_bf16;
  int has2;                  // du is there
  // Pieces of consecutive rows, `per_group` of them for each run of gate_rows
  // rows; a workgroup takes `per_block` pieces.
  int64_t pieces;
  uint32_t per_group, per_block, piece_rows;
  float *pa, *pb, *pw, *pc;  // partial sums: [pieces] of dt yn, dt; [workgroups] of du hn, du (NULL: not wanted)
  uint32_t pitch;            // floats between their rows
};

// ---------------------------------------------------------------------------
// Sums over a row
// ---------------------------------------------------------------------------

// The same number, which the compiler cannot take for the one of the last row:
// else it keeps every comparison with the row's end, 8 a piece, in registers
// over the loop (186 vector registers for 60, and scratch beyond 8 elements a lane).
__device__ __forceinline__ uint32_t anew(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Sum over a wave in every lane, in a fixed order.
__device__ __forceinline__ float wave_total(float v) {
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0xB1, 0xf, 0xf, true));
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x4E, 0xf, 0xf, true));
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x141, 0xf, 0xf, true));
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x140, 0xf, 0xf, true));
  const int b = __builtin_bit_cast(int, v);
  const float r0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 0));
  const float r1 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 16));
  const float r2 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 32));
  const float r3 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 48));
  return (r0 + r1) + (r2 + r3);
}

// Sums over the W waves of a row.  Two buffers in turn: a wave writes one again
// only after the barrier of the next sum, which every wave reaches after its
// reads of this one.
template <int W>
struct RowSums {
  float* lds;  // [2][2][W]
  int turn = 0;
  template <int N>
  __device__ __forceinline__ void total(float (&v)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = wave_total(v[n]);
    if constexpr (W > 1) {
      float* const at = lds + turn * 2 * W;
      const int wave = threadIdx.x / kWave;
      if (threadIdx.x % kWave == 0) {
#pragma unroll
        for (int n = 0; n < N; ++n) at[n * W + wave] = v[n];
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < N; ++n) {
        v[n] = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) v[n] += at[n * W + w];
      }
      turn ^= 1;
    }
  }
  __device__ __forceinline__ float total1(float v) {
    float a[1] = {v};
    total(a);
    return a[0];
  }
};

// ---------------------------------------------------------------------------
// Parameters
// ---------------------------------------------------------------------------

// V columns of a vector of parameters, 0 beyond its end; without the vector, `none`.
template <int V>
__device__ __forceinline__ void load_param(const void* p, int bf16, uint32_t cols, uint32_t col, float none,
                                           float (&x)[V]) {
  if (p == nullptr) {
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = col + e < cols ? none : 0.f;
  } else if (bf16) {
    const Piece<true, V> q = load_row<true, V>(p, cols, col);
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = elem(q, e);
  } else {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const Piece<false, 4> q = load_row<false, 4>(p, cols, col + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[4 * i + e] = elem(q, e);
    }
  }
}

// The gate's row for a row of the stream: NULL where it is one value (or none).
__device__ __forceinline__ const void* gate_row(const JoinArgs& A, uint32_t row) {
  if (A.gate_kind != SHAMPOO_GATE_ROWS) return nullptr;
  const int64_t at = (int64_t)(row / A.gate_rows) * A.cols;
  return static_cast<const uint8_t*>(A.gate) + at * (A.gate_bf16 ? 2 : 4);
}
__device__ __forceinline__ float gate_value(const JoinArgs& A, uint32_t row) {
  if (A.gate_kind != SHAMPOO_GATE_TOKEN) return 1.f;
  if (A.gate_bf16) return __builtin_bit_cast(float, (uint32_t)ldg(static_cast<const uint16_t*>(A.gate) + row) << 16);
  return ldg(static_cast<const float*>(A.gate) + row);
}

// Mean and s of a row held in pieces, zero beyond its end.
template <int W, int P, int V>
__device__ __forceinline__ void row_stats(const float (&x)[P][V], const NormSide& n, uint32_t cols, uint32_t lane,
                                          RowSums<W>& sums, float& mean, float& s) {
  const float over = 1.f / (float)cols;
  mean = 0.f;
  float ss = 0.f;
  if (n.kind == SHAMPOO_NORM_LAYER) {
    float t = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int e = 0; e < V; ++e) t += x[p][e];
    mean = sums.total1(t) * over;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t col = (p * W * kWave + lane) * V;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = col + e < cols ? x[p][e] - mean : 0.f;
        ss = __builtin_fmaf(d, d, ss);
      }
    }
  } else {
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int e = 0; e < V; ++e) ss = __builtin_fmaf(x[p][e], x[p][e], ss);
  }
  s = 1.f / sqrtf(sums.total1(ss) * over + n.eps);
}

// Rows that a workgroup holds at once: 4 of a wave each, or one.
template <int W>
constexpr int kRowLanes = W == 1 ? 4 : 1;
template <int W>
constexpr int kRowThreads = W == 1 ? 256 : 64 * W;

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------

template <bool SB, bool BB, int W, int P, bool JOIN>
__global__ void __launch_bounds__(kRowThreads<W>) join_forward_kernel(const JoinArgs A) {
  constexpr int V = SB ? 8 : 4, L = kRowLanes<W>;
  __shared__ float red[4 * W];
  RowSums<W> sums{red};
  const uint32_t lane0 = threadIdx.x % (kWave * W);
  const int64_t first = (int64_t)blockIdx.x * L + __builtin_amdgcn_readfirstlane(threadIdx.x / (kWave * W));
  for (int64_t row = first; row < A.rows; row += (int64_t)gridDim.x * L) {
    const uint32_t lane = anew(lane0);
    Piece<SB, V> r[P];
    Piece<BB, V> y[P];
    float x[P][V];
#pragma unroll
    for (int p = 0; p < P; ++p)
      r[p] = load_row<SB, V>(row_at<SB>(A.r, row, A.ldr), A.cols, (p * W * kWave + lane) * V);
    if constexpr (JOIN) {
#pragma unroll
      for (int p = 0; p < P; ++p)
        y[p] = load_row<BB, V>(row_at<BB>(A.y, row, A.ldy), A.cols, (p * W * kWave + lane) * V);
    }
    if (A.kr.codes != nullptr) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        Mx8Piece<V> q;
        q.encode(r[p]);
        q.store(A.kr, row, (p * W * kWave + lane) * V);
      }
    }
    if constexpr (JOIN) {
      if (A.ky.codes != nullptr) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
          Mx8Piece<V> q;
          q.encode(y[p]);
          q.store(A.ky, row, (p * W * kWave + lane) * V);
        }
      }
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int e = 0; e < V; ++e) x[p][e] = elem(y[p], e);
      float mean = 0.f, s = 1.f;
      if (A.after.kind != SHAMPOO_NORM_NONE) {
        row_stats<W, P, V>(x, A.after, A.cols, lane, sums, mean, s);
        if (A.stats1 != nullptr && lane == 0) {
          stg(A.stats1 + 2 * row, mean);
          stg(A.stats1 + 2 * row + 1, s);
        }
      }
      const void* const grow = gate_row(A, (uint32_t)row);
      const float token = gate_value(A, (uint32_t)row);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const uint32_t col = (p * W * kWave + lane) * V;
        float g[V], w[V], b[V];
        load_param(grow, A.gate_bf16, A.cols, col, token, g);
        load_param(A.after.w, A.after.w_bf16, A.cols, col, 1.f, w);
        load_param(A.after.b, A.after.b_bf16, A.cols, col, 0.f, b);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float z = __builtin_fmaf((x[p][e] - mean) * s, w[e], b[e]);
          x[p][e] = __builtin_fmaf(g[e], z, A.scale * elem(r[p], e));
        }
        store_row<SB, V>(row_at<SB>(A.h, row, A.ldh), A.cols, col, x[p]);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int e = 0; e < V; ++e) x[p][e] = elem(r[p], e);
    }
    if (A.before.kind != SHAMPOO_NORM_NONE) {
      float mean, s;
      row_stats<W, P, V>(x, A.before, A.cols, lane, sums, mean, s);
      if (A.stats2 != nullptr && lane == 0) {
        stg(A.stats2 + 2 * row, mean);
        stg(A.stats2 + 2 * row + 1, s);
      }
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const uint32_t col = (p * W * kWave + lane) * V;
        float w[V], b[V], u[V];
        load_param(A.before.w, A.before.w_bf16, A.cols, col, 1.f, w);
        load_param(A.before.b, A.before.b_bf16, A.cols, col, 0.f, b);
#pragma unroll
        for (int e = 0; e < V; ++e) u[e] = __builtin_fmaf((x[p][e] - mean) * s, w[e], b[e]);
        store_row<BB, V>(row_at<BB>(A.u, row, A.ldu), A.cols, col, u);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Backward.  With dt the gradient of h (from h itself and through N2),
//   dr = scale dt,  dz = gate dt,  dy = N1'(dz),
//   dw1 = sum dz yn,  db1 = sum dz,  dgate = sum dt z,  dw2 = sum du hn,  db2 = sum du
// (yn, hn: the normed rows).  A gate row is constant over a piece, so sum dt yn
// and sum dt give dw1, db1 and dgate alike; with a gate for each token they are
// taken of the gated dt.  Columns' sums stay in registers over all rows of a
// workgroup, then go to memory for join_sums_kernel: no atomics, a fixed order.
// ---------------------------------------------------------------------------

// A lane's sums, added over the rows held side by side, to row `at` of partial sums.
template <int W, int P, int V>
__device__ __forceinline__ void store_sums(const float (&acc)[P][V], float* to, uint32_t pitch, uint32_t lane, float* lds) {
  if constexpr (W > 1) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t col = (p * W * kWave + lane) * V;
      if (col < pitch) {
#pragma unroll
        for (int q = 0; q < V / 4; ++q)
          stg(reinterpret_cast<floatx4*>(to + col) + q,
              floatx4{acc[p][4 * q], acc[p][4 * q + 1], acc[p][4 * q + 2], acc[p][4 * q + 3]});
      }
    }
  } else {
    constexpr int kCols = kWave * V;
    const int wave = threadIdx.x / kWave;
#pragma unroll
    for (int p = 0; p < P; ++p) {
#pragma unroll
      for (int e = 0; e < V; ++e) lds[wave * kCols + lane * V + e] = acc[p][e];
      __syncthreads();
      for (int c = threadIdx.x; c < kCols; c += 256) {
        const uint32_t col = p * kCols + c;
        if (col < pitch) stg(to + col, (lds[c] + lds[kCols + c]) + (lds[2 * kCols + c] + lds[3 * kCols + c]));
      }
      __syncthreads();
    }
  }
}

// An input of the backward pass, from its MX8 copy or as it is.
template <bool KEEP, bool BF16, int V>
struct Kept {
  Piece<BF16, V> x;
  Mx8Piece<V> q;
  __device__ __forceinline__ void load(const void* from, int64_t ld, const Mx8Rows& m, int64_t row, uint32_t cols,
                                       uint32_t col) {
    if constexpr (KEEP) {
      q.load(m, row, col);
    } else {
      x = load_row<BF16, V>(row_at<BF16>(from, row, ld), cols, col);
    }
  }
  __device__ __forceinline__ void get(float (&v)[V]) const {
    if constexpr (KEEP) {
      q.decode(v);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = elem(x, e);
    }
  }
};

template <bool SB, bool BB, int W, int P, bool JOIN, bool KEEP, bool BIAS>
__global__ void __launch_bounds__(kRowThreads<W>) join_backward_kernel(const JoinArgs A) {
  constexpr int V = SB ? 8 : 4, L = kRowLanes<W>;
  __shared__ __attribute__((aligned(16))) float lds[W == 1 ? 4 * kWave * V : 4 * W];
  RowSums<W> sums{lds};
  const uint32_t lane0 = threadIdx.x % (kWave * W);
  const int part = __builtin_amdgcn_readfirstlane(threadIdx.x / (kWave * W));
  const float over = 1.f / (float)A.cols;
  const bool has1 = JOIN && A.after.kind != SHAMPOO_NORM_NONE, has2 = A.has2 != 0;
  const bool need_y = JOIN && (has1 || A.gate_kind != SHAMPOO_GATE_NONE || has2);
  float aw[P][V] = {}, ac[P][V] = {}, aa[P][V], ab[P][V];
  const int64_t begin = (int64_t)blockIdx.x * A.per_block;
  const int64_t end = begin + A.per_block < A.pieces ? begin + A.per_block : A.pieces;
  for (int64_t piece = begin; piece < end; ++piece) {
    const int64_t group = piece / A.per_group;
    const int64_t group0 = group * A.gate_rows, group1 = group0 + A.gate_rows;
    const int64_t row0 = group0 + (piece - group * A.per_group) * A.piece_rows;
    const int64_t row1 = row0 + A.piece_rows < group1 ? row0 + A.piece_rows : group1;
    if constexpr (JOIN) {
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int e = 0; e < V; ++e) aa[p][e] = ab[p][e] = 0.f;
    }
    for (int64_t row = row0 + part; row < row1; row += L) {
      const uint32_t lane = anew(lane0);
      Piece<SB, V> dh[P];
      Piece<BB, V> du[P];
      Kept<KEEP, SB, V> r[P];
      Kept<KEEP, BB, V> y[P];
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const uint32_t col = (p * W * kWave + lane) * V;
        if (has2) {
          du[p] = load_row<BB, V>(row_at<BB>(A.du, row, A.lddu), A.cols, col);
          r[p].load(A.r, A.ldr, A.kr, row, A.cols, col);
        }
        if constexpr (JOIN) {
          if (need_y) y[p].load(A.y, A.ldy, A.ky, row, A.cols, col);
          dh[p].w = 0u;
          if (A.dh != nullptr) dh[p] = load_row<SB, V>(row_at<SB>(A.dh, row, A.lddh), A.cols, col);
        }
      }
      float mean1 = 0.f, s1 = 1.f, mean2 = 0.f, s2 = 1.f, token = 1.f;
      if (has1) {
        mean1 = ldg(A.stats1 + 2 * row);
        s1 = ldg(A.stats1 + 2 * row + 1);
      }
      if (has2) {
        mean2 = ldg(A.stats2 + 2 * row);
        s2 = ldg(A.stats2 + 2 * row + 1);
      }
      const void* grow = nullptr;
      if constexpr (JOIN) {
        grow = gate_row(A, (uint32_t)row);
        token = gate_value(A, (uint32_t)row);
      }
      float yn[P][V], hn[P][V], dt[P][V];
      float t[2] = {0.f, 0.f};
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const uint32_t col = (p * W * kWave + anew(lane)) * V;
        if constexpr (JOIN) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            yn[p][e] = 0.f;
            dt[p][e] = elem(dh[p], e);
          }
          if (need_y) {
            y[p].get(yn[p]);
#pragma unroll
            for (int e = 0; e < V; ++e) yn[p][e] = (yn[p][e] - mean1) * s1;
          }
        }
        if (has2) {
          r[p].get(hn[p]);
          if constexpr (JOIN) {
            float g[V], w[V], b[V];
            load_param(grow, A.gate_bf16, A.cols, col, token, g);
            load_param(A.after.w, A.after.w_bf16, A.cols, col, 1.f, w);
            load_param(A.after.b, A.after.b_bf16, A.cols, col, 0.f, b);
#pragma unroll
            for (int e = 0; e < V; ++e)
              hn[p][e] = __builtin_fmaf(g[e], __builtin_fmaf(yn[p][e], w[e], b[e]), A.scale * hn[p][e]);
          }
          float w[V];
          load_param(A.before.w, A.before.w_bf16, A.cols, col, 1.f, w);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            hn[p][e] = (hn[p][e] - mean2) * s2;
            const float d = elem(du[p], e), g = d * w[e];
            aw[p][e] = __builtin_fmaf(d, hn[p][e], aw[p][e]);
            if constexpr (BIAS) ac[p][e] += d;
            t[0] = __builtin_fmaf(g, hn[p][e], t[0]);
            t[1] += g;
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (has2) {
        sums.total(t);
        const float m0 = t[0] * over, m1 = A.before.kind == SHAMPOO_NORM_LAYER ? t[1] * over : 0.f;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const uint32_t col = (p * W * kWave + anew(lane)) * V;
          float w[V];
          load_param(A.before.w, A.before.w_bf16, A.cols, col, 1.f, w);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float g = elem(du[p], e) * w[e];
            const float d = s2 * (g - m1 - hn[p][e] * m0);
            if constexpr (JOIN) {
              dt[p][e] += d;
            } else {
              dt[p][e] = d;
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if (A.dr != nullptr) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
          float o[V];
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] = A.scale * dt[p][e];
          store_row<SB, V>(row_at<SB>(A.dr, row, A.lddr), A.cols, (p * W * kWave + lane) * V, o);
        }
      }
      if constexpr (JOIN) {
        t[0] = t[1] = 0.f;
        float dtoken = 0.f;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const uint32_t col = (p * W * kWave + anew(lane)) * V;
          float g[V], w[V], b[V];
          load_param(grow, A.gate_bf16, A.cols, col, 1.f, g);
          load_param(A.after.w, A.after.w_bf16, A.cols, col, 1.f, w);
          load_param(A.after.b, A.after.b_bf16, A.cols, col, 0.f, b);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            dtoken = __builtin_fmaf(dt[p][e], __builtin_fmaf(yn[p][e], w[e], b[e]), dtoken);
            const float d = dt[p][e] * token;
            aa[p][e] = __builtin_fmaf(d, yn[p][e], aa[p][e]);
            if constexpr (BIAS) ab[p][e] += d;
            dt[p][e] = d * g[e] * w[e];  // dz w1
            t[0] = __builtin_fmaf(dt[p][e], yn[p][e], t[0]);
            t[1] += dt[p][e];
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        float m0 = 0.f, m1 = 0.f;
        if (has1) {
          sums.total(t);
          m0 = t[0] * over;
          m1 = A.after.kind == SHAMPOO_NORM_LAYER ? t[1] * over : 0.f;
        }
        if (A.dtoken != nullptr) {
          dtoken = sums.total1(dtoken);
          if (lane == 0) {
            if (A.dtoken_bf16) {
              stg(static_cast<uint16_t*>(A.dtoken) + row, f32_to_bf16_bits(dtoken));
            } else {
              stg(static_cast<float*>(A.dtoken) + row, dtoken);
            }
          }
        }
        if (A.dy != nullptr) {
#pragma unroll
          for (int p = 0; p < P; ++p) {
            float o[V];
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = s1 * (dt[p][e] - m1 - yn[p][e] * m0);
            store_row<BB, V>(row_at<BB>(A.dy, row, A.lddy), A.cols, (p * W * kWave + lane) * V, o);
          }
        }
      }
    }
    if constexpr (JOIN) {
      if (A.pa != nullptr) store_sums<W, P, V>(aa, A.pa + piece * (int64_t)A.pitch, A.pitch, lane0, lds);
      if constexpr (BIAS) {
        if (A.pb != nullptr) store_sums<W, P, V>(ab, A.pb + piece * (int64_t)A.pitch, A.pitch, lane0, lds);
      }
    }
  }
  if (has2) {
    if (A.pw != nullptr) store_sums<W, P, V>(aw, A.pw + (int64_t)blockIdx.x * A.pitch, A.pitch, lane0, lds);
    if constexpr (BIAS) {
      if (A.pc != nullptr) store_sums<W, P, V>(ac, A.pc + (int64_t)blockIdx.x * A.pitch, A.pitch, lane0, lds);
    }
  }
}

}  // namespace shp
