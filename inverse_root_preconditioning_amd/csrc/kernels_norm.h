// Norms over rows and the join of a block's output y with its residual r,
//   z = N1(y),  h = scale r + gate z,  u = N2(h),
// with their gradients.  N(x) = (x - mean) s w + b, s = 1 / sqrt(mean of squares
// (RMS: mean = 0) or variance (layer) + eps); either norm may be absent, and
// the norm alone is the join without y: h = r.
//
// `waves` waves (1 to 16) hold a row of up to 64 waves P V columns in registers,
// each lane P pieces of V consecutive elements, so that a row is read once
// however many sums over it the formulas need; the parameters' columns stay in
// registers over all the rows that a workgroup takes.  The waves are a number of
// the call, so that few lanes are idle whatever the width.
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
  uint32_t cols, flags;
  uint32_t waves, lanes;     // of a row; rows that a workgroup holds side by side
  float scale;
  const void *r, *y;  // the inputs; y unused without a join
  int64_t ldr, ldy;
  Mx8Rows kr, ky;     // their MX8 copies: written forward where codes is given, read backward with KEEP
  NormSide after, before;
  const void* gate;
  int gate_bf16;
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
  // The rows' division: `per_group` pieces of each run of gate_rows rows; a
  // workgroup takes `per_block` pieces.
  uint32_t pieces, per_group, per_block;
  float *pa, *pb, *pw, *pc;  // partial sums: [pieces] of dt yn, dt; [workgroups] of du hn, du (NULL: not wanted)
  uint32_t pitch;            // floats between their rows
};

// The same value, which the compiler cannot take for the one of the row before.
// Else every comparison with the row's end and every flag that a row's work tests
// is kept in scalar registers over the loop, which then do not suffice: a hundred moves
// a row from where they are put instead, a third of the instructions.
__device__ __forceinline__ uint32_t anew(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}
__device__ __forceinline__ uint32_t anew_uniform(uint32_t v) {
  asm volatile("" : "+s"(v));
  return v;
}

// What there is to do, in one word.
enum : uint32_t {
  kJoinNorm1 = 1,     // N1
  kJoinMean1 = 2,     // with a mean
  kJoinNorm2 = 4,     // N2 (backward: and its gradient)
  kJoinMean2 = 8,
  kJoinRuns = 16,     // a gate row for runs of rows
  kJoinToken = 32,    // a gate for each row
  kJoinDh = 64,       // a gradient of h
  kJoinNeedY = 128,   // the branch is read backward
  kJoinCodesR = 256,  // MX8 copies are written
  kJoinCodesY = 512
};

// ---------------------------------------------------------------------------
// Sums over a row
// ---------------------------------------------------------------------------

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

constexpr int kMaxWaves = 16;
constexpr int kSumsFloats = 4 * kMaxWaves;  // LDS of a row's sums

// Sums over the waves of a row, in a fixed order.  Two buffers in turn: a wave
// writes one again only after the barrier of the next sum, which every wave
// reaches after its reads of this one.  What lies beyond the row's waves is 0.
struct RowSums {
  float* lds;  // [2][2][kMaxWaves] of this row
  uint32_t waves, wave;
  uint32_t turn = 0;
  // Called by every thread, with one more barrier before the first sum.
  __device__ __forceinline__ RowSums(float* all, uint32_t part, uint32_t n, uint32_t rows)
      : lds(all + part * kSumsFloats), waves(n), wave(__builtin_amdgcn_readfirstlane(threadIdx.x / kWave) - part * n) {
    if (waves > 1) {
      for (uint32_t i = threadIdx.x; i < rows * kSumsFloats; i += blockDim.x) all[i] = 0.f;
      __syncthreads();
    }
  }
  template <int N>
  __device__ __forceinline__ void total(float (&v)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = wave_total(v[n]);
    if (waves > 1) {
      float* const at = lds + turn * 2 * kMaxWaves;
      if (threadIdx.x % kWave == 0) {
#pragma unroll
        for (int n = 0; n < N; ++n) at[n * kMaxWaves + wave] = v[n];
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const floatx4* const q = reinterpret_cast<const floatx4*>(at + n * kMaxWaves);
        floatx4 t = q[0];
        if (waves > 4) t += q[1];
        if (waves > 8) t += q[2] + q[3];
        v[n] = (t[0] + t[1]) + (t[2] + t[3]);
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
// Pieces of a row
// ---------------------------------------------------------------------------

// The places of a lane's P pieces.  Loads are of V elements that are there (at
// the row's end those before it), so that no branch stands between them; `fix`
// puts right what a piece beyond the end, or over it, has read, when it has come.
// WHOLE: the columns are a multiple of V.
template <int P, int V, bool WHOLE>
struct Places {
  uint32_t cols, width, lane;  // of the row; its lanes; this one
  __device__ __forceinline__ Places(const JoinArgs& A, uint32_t which) : cols(A.cols), width(A.waves * kWave), lane(which) {}
  __device__ __forceinline__ uint32_t col(int p) const { return (p * width + lane) * V; }

  // ONCE: it is read once, and where rows begin at a line's start or near it, its lines by one
  // wave each: past the caches.  Elsewhere two waves share a line, which would come twice
  // (2050 bf16 columns: norm 45 us that way, 34 through the caches).
  template <bool BF16, bool ONCE = true>
  __device__ __forceinline__ Piece<BF16, V> load(const void* row, int p) const {
    Piece<BF16, V> x;
    if (WHOLE || cols >= V) {
      const uint32_t from = min(col(p), cols - V);
      if constexpr (ONCE && WHOLE) {
        x.load_once(row, from);
      } else {
        x.load_at(row, from);
      }
    } else {
      x = load_row<BF16, V>(row, cols, col(p));
    }
    return x;
  }
  template <bool BF16>
  __device__ __forceinline__ void fix(Piece<BF16, V>& x, int p) const {
    if constexpr (WHOLE) {
      if (col(p) >= cols) x.w = 0u;
    } else if (cols >= V) {
      const uint32_t over = col(p) + V;
      if (over > cols) x.shift_down(min(over - cols, (uint32_t)V));
    }
  }
  template <bool BF16>
  __device__ __forceinline__ void store(void* row, int p, const float (&x)[V]) const {
    if constexpr (WHOLE) {
      if (col(p) < cols) store_row<BF16, V, true>(row, cols, col(p), x);
    } else {
      store_row<BF16, V>(row, cols, col(p), x);
    }
  }
  // Whether element e of piece p is a column.
  __device__ __forceinline__ bool valid(int p, int e) const { return col(p) + (WHOLE ? 0 : e) < cols; }
};

// Piece p of a vector of parameters, 0 beyond its end; without the vector, `none`.
template <int P, int V, bool WHOLE>
__device__ __forceinline__ void load_param(const Places<P, V, WHOLE>& at, int p, const void* v, int bf16, float none,
                                           float (&x)[V]) {
  if (v == nullptr) {
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = at.valid(p, e) ? none : 0.f;
  } else if (bf16) {
    Piece<true, V> q = at.template load<true, false>(v, p);
    at.fix(q, p);
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = elem(q, e);
  } else {
    Piece<false, V> q = at.template load<false, false>(v, p);
    at.fix(q, p);
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = elem(q, e);
  }
}

// Parameters of a lane's pieces: kept in registers, or where those do not
// suffice, read again for every use.
template <int P, int V, bool WHOLE, bool BIAS, bool KEPT>
struct Parameters {
  static constexpr bool kKept = KEPT;
  typedef Places<P, V, WHOLE> At;
  float w[kKept ? P : 1][V], b[kKept ? P : 1][V];
  uint32_t run;

  // w and b of a norm; of N1 times the gate's row of a run, where the gate is
  // one for runs of rows, so that gate N1 = w yn + b.
  __device__ __forceinline__ void load(const At& at, const JoinArgs& A, const NormSide& n, bool gated, int p, float (&w)[V],
                                       float (&b)[V]) const {
    load_param(at, p, n.w, n.w_bf16, 1.f, w);
    if constexpr (BIAS) load_param(at, p, n.b, n.b_bf16, 0.f, b);
    if (gated) {
      const void* const row = static_cast<const uint8_t*>(A.gate) + (int64_t)run * A.cols * (A.gate_bf16 ? 2 : 4);
      float g[V];
      load_param(at, p, row, A.gate_bf16, 1.f, g);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        w[e] *= g[e];
        if constexpr (BIAS) b[e] *= g[e];
      }
    }
  }
  __device__ __forceinline__ void keep(const At& at, const JoinArgs& A, const NormSide& n, bool gated, uint32_t new_run) {
    run = new_run;
    if constexpr (kKept) {
#pragma unroll
      for (int p = 0; p < P; ++p) load(at, A, n, gated, p, w[p], b[p]);
    }
  }
  __device__ __forceinline__ void get(const At& at, const JoinArgs& A, const NormSide& n, bool gated, int p, float (&wp)[V],
                                      float (&bp)[V]) const {
    if constexpr (kKept) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        wp[e] = w[p][e];
        bp[e] = BIAS ? b[p][e] : 0.f;
      }
    } else {
      __builtin_amdgcn_sched_barrier(0);  // one piece's parameters at a time
      load(At(A, anew(at.lane)), A, n, gated, p, wp, bp);
      if constexpr (!BIAS) {
#pragma unroll
        for (int e = 0; e < V; ++e) bp[e] = 0.f;
      }
    }
  }
};

__device__ __forceinline__ float load_token(const JoinArgs& A, int64_t row) {
  if (A.gate_bf16) return __builtin_bit_cast(float, (uint32_t)ldg(static_cast<const uint16_t*>(A.gate) + row) << 16);
  return ldg(static_cast<const float*>(A.gate) + row);
}

// Mean and s of a row held in pieces, zero beyond its end.  What is normed is formed as (x - mean) s, whose
// difference is exact near the mean.  As x s - mean s it would keep the product's rounding: 0.03 where
// x = mean = 1000 and the variance is 0.
template <int P, int V, bool WHOLE>
__device__ __forceinline__ void row_stats(const Places<P, V, WHOLE>& at, const float (&x)[P][V], bool centred,
                                          float eps, RowSums& sums, float& mean, float& s) {
  const float over = 1.f / (float)at.cols;
  mean = 0.f;
  float ss = 0.f;
  if (centred) {
    float t = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int e = 0; e < V; ++e) t += x[p][e];
    t = sums.total1(t);
    mean = t * over;
    // as rounded once: exact where t / cols is
    mean = __builtin_fmaf(__builtin_fmaf(-mean, (float)anew_uniform(at.cols), t), over, mean);
#pragma unroll
    for (int p = 0; p < P; ++p) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = at.valid(p, e) ? x[p][e] - mean : 0.f;
        ss = __builtin_fmaf(d, d, ss);
      }
    }
  } else {
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int e = 0; e < V; ++e) ss = __builtin_fmaf(x[p][e], x[p][e], ss);
  }
  s = 1.f / sqrtf(sums.total1(ss) * over + eps);
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------

// A row is read once and stays in registers for both norms' sums and both outputs;
// its copies are made from the same registers.  Bound by HBM once rows fill the
// compute units: 16384 rows of 2048 bf16 with 8-bit copies 65 us as a join (5.2
// TB/s) and 32 as a norm (5.3); below that by a row's latency, loads, two sums a norm and their
// barriers: a single row of 2048 3.9 and 2.4 us, its launch included.  Several
// rows a workgroup only where each is a wave's, which needs no barrier.
template <bool SB, bool BB, int P, bool JOIN, bool WHOLE>
__global__ void __launch_bounds__(kWave * kMaxWaves) join_forward_kernel(const JoinArgs A) {
  constexpr int V = SB ? 8 : 4;
  typedef Places<P, V, WHOLE> At;
  __shared__ __attribute__((aligned(16))) float red[kSumsFloats];
  const uint32_t part = A.lanes > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) : 0;
  const uint32_t lane0 = threadIdx.x - part * kWave;
  RowSums sums(red, 0, A.waves, 1);
  const int64_t step = (int64_t)gridDim.x * A.lanes;
  int64_t row = (int64_t)blockIdx.x * A.lanes + part;
  if (row >= A.rows) return;  // a wave by itself, or the whole workgroup
  Piece<SB, V> r[P];
  Piece<BB, V> y[P];
  auto load = [&](const At& at, int64_t from) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      r[p] = at.template load<SB>(row_at<SB>(A.r, from, A.ldr), p);
      if constexpr (JOIN) y[p] = at.template load<BB>(row_at<BB>(A.y, from, A.ldy), p);
    }
  };
  Parameters<P, V, WHOLE, true, (P * V <= 8)> n1, n2;
  {
    const At at(A, lane0);
    load(at, row);
    if constexpr (JOIN)
      n1.keep(at, A, A.after, A.flags & kJoinRuns, __builtin_amdgcn_readfirstlane((uint32_t)row / A.gate_rows));
    n2.keep(at, A, A.before, false, 0);
  }
  while (true) {
    const At at(A, anew(lane0));
    const uint32_t flags = anew_uniform(A.flags);
    float x[P][V], rf[P][V];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      at.fix(r[p], p);
#pragma unroll
      for (int e = 0; e < V; ++e) rf[p][e] = elem(r[p], e);
      if (flags & kJoinCodesR) {
        Mx8Piece<V> q;
        q.encode(r[p]);
        q.store(A.kr, row, at.col(p));
      }
      if constexpr (JOIN) {
        at.fix(y[p], p);
#pragma unroll
        for (int e = 0; e < V; ++e) x[p][e] = elem(y[p], e);
        if (flags & kJoinCodesY) {
          Mx8Piece<V> q;
          q.encode(y[p]);
          q.store(A.ky, row, at.col(p));
        }
      }
    }
    const int64_t next = row + step;
    if (next < A.rows) load(at, next);  // in flight while this row is worked on
    if constexpr (JOIN) {
      float mean = 0.f, s = 1.f;
      if (flags & kJoinNorm1) {
        row_stats(at, x, (flags & kJoinMean1) != 0, A.after.eps, sums, mean, s);
        if (A.stats1 != nullptr && at.lane == 0) stg(reinterpret_cast<f32x2_t*>(A.stats1) + row, f32x2_t{mean, s});
      }
      if (flags & kJoinRuns) {
        const uint32_t now = __builtin_amdgcn_readfirstlane((uint32_t)row / A.gate_rows);
        if (now != n1.run) n1.keep(at, A, A.after, true, now);
      }
      const float token = flags & kJoinToken ? load_token(A, row) : 1.f;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float w[V], b[V];
        n1.get(at, A, A.after, flags & kJoinRuns, p, w, b);
        if (flags & kJoinToken) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float z = __builtin_fmaf((x[p][e] - mean) * s, w[e], b[e]);
            x[p][e] = __builtin_fmaf(token, z, A.scale * rf[p][e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e)
            x[p][e] = __builtin_fmaf((x[p][e] - mean) * s, w[e], __builtin_fmaf(A.scale, rf[p][e], b[e]));
        }
      }
#pragma unroll
      for (int p = 0; p < P; ++p) at.template store<SB>(row_at<SB>(A.h, row, A.ldh), p, x[p]);
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int e = 0; e < V; ++e) x[p][e] = rf[p][e];
    }
    if (flags & kJoinNorm2) {
      float mean, s;
      row_stats(at, x, (flags & kJoinMean2) != 0, A.before.eps, sums, mean, s);
      if (A.stats2 != nullptr && at.lane == 0) stg(reinterpret_cast<f32x2_t*>(A.stats2) + row, f32x2_t{mean, s});
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float u[V], w[V], b[V];
        n2.get(at, A, A.before, false, p, w, b);
#pragma unroll
        for (int e = 0; e < V; ++e) u[e] = __builtin_fmaf((x[p][e] - mean) * s, w[e], b[e]);
        at.template store<BB>(row_at<BB>(A.u, row, A.ldu), p, u);
      }
    }
    if (next >= A.rows) return;
    row = next;
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
// Bound by HBM: 16384 rows of 2048 bf16 from 8-bit copies 70 us as a join (4.8
// TB/s) and 35 as a norm (4.9).  128 registers a lane do not hold the row, the next
// one's loads, the parameters and four sums a column (with biases), nor 16 elements a lane with two: then
// the sums are in LDS.  Joins of 2^25 bf16 elements, us with the sums in registers (fewer waves, no
// next row, or scratch memory) and in LDS: with biases rows of 2048 78, 80; 2050 159, 113; 5120 139, 97; 8192
// 113, 81; without, of 16384 216, 98.  With biases those take 238: two of the four sums do not fit.
// ---------------------------------------------------------------------------

// A lane's sums over its columns: in registers, or its own places in LDS.
template <int P, int V, bool IN_LDS>
struct ColumnSums {
  static constexpr int kFloats = IN_LDS ? P * V * kWave * kMaxWaves : 0;  // of a workgroup
  float v[IN_LDS ? 1 : P][V];
  float* all;
  floatx4* at;
  __device__ __forceinline__ explicit ColumnSums(float* lds)
      : all(lds), at(reinterpret_cast<floatx4*>(lds) + threadIdx.x) {}
  // Column c of the first piece, from the lanes of a row whose first is thread `from`.
  __device__ __forceinline__ float column(uint32_t from, uint32_t c) const {
    return all[(c % V / 4 * kWave * kMaxWaves + from + c / V) * 4 + c % 4];
  }
  __device__ __forceinline__ void clear() {
    const float zero[V] = {};
#pragma unroll
    for (int p = 0; p < P; ++p) put(p, zero);
  }
  __device__ __forceinline__ void get(int p, float (&x)[V]) const {
    if constexpr (IN_LDS) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        const floatx4 q = at[(p * (V / 4) + i) * kWave * kMaxWaves];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * i + e] = q[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] = v[p][e];
    }
  }
  __device__ __forceinline__ void put(int p, const float (&x)[V]) {
    if constexpr (IN_LDS) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i)
        at[(p * (V / 4) + i) * kWave * kMaxWaves] = floatx4{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) v[p][e] = x[e];
    }
  }
};

// A lane's sums, added over the rows held side by side, to a row of partial sums.
template <int P, int V, bool IN_LDS>
__device__ __forceinline__ void store_sums(const ColumnSums<P, V, IN_LDS>& sums, float* to, const JoinArgs& A,
                                           uint32_t lane, uint32_t part, float* lds) {
  const uint32_t cols = A.waves * kWave * V;  // of a piece
#pragma unroll
  for (int p = 0; p < P; ++p) {
    float acc[V];
    sums.get(p, acc);
    if (P > 1 || A.lanes == 1) {
      const uint32_t col = p * cols + lane * V;
      if (col < A.pitch) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
          stg(reinterpret_cast<floatx4*>(to + col) + i, floatx4{acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]});
      }
    } else {
      // sums in LDS are added where they are
      ColumnSums<1, V, true> there(IN_LDS ? sums.all : lds);
      if constexpr (!IN_LDS) there.put(0, acc);
      __syncthreads();
      for (uint32_t c = threadIdx.x; c < cols; c += blockDim.x) {
        if (c < A.pitch) {
          float v = 0.f;
          for (uint32_t i = 0; i < A.lanes; ++i) v += there.column(i * A.waves * kWave, c);
          stg(to + c, v);
        }
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
  template <class At>
  __device__ __forceinline__ void load(const At& at, const void* from, int64_t ld, const Mx8Rows& m, int64_t row, int p) {
    if constexpr (KEEP) {
      q.load_near(m, row, at.col(p));
    } else {
      x = at.template load<BF16>(row_at<BF16>(from, row, ld), p);
    }
  }
  __device__ __forceinline__ void clear() {
    if constexpr (KEEP) {
      q.clear();
    } else {
      x.w = 0u;
    }
  }
  template <class At>
  __device__ __forceinline__ void get(const At& at, const Mx8Rows& m, int p, float (&v)[V]) {
    if constexpr (KEEP) {
      if (at.col(p) >= m.padded) q.clear();
      q.decode(v);
    } else {
      at.fix(x, p);
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = elem(x, e);
    }
  }
};

template <bool SB, bool BB, int P, bool JOIN, bool KEEP, bool BIAS, bool WHOLE>
__global__ void __launch_bounds__(kWave * kMaxWaves) join_backward_kernel(const JoinArgs A) {
  constexpr int V = SB ? 8 : 4;
  typedef Places<P, V, WHOLE> At;
  // Parameters in registers and the next row's loads in flight, where there are registers for
  // them: 128 in a workgroup of 16 waves.
  constexpr bool kAhead = P * V <= 8;
  __shared__ __attribute__((aligned(16))) float red[kMaxWaves * kSumsFloats];
  // Columns' sums in LDS where 128 registers do not hold them, 128 KB of its 160: those for w2 and w1 (or the
  // gate) of 16 elements a lane, all four of 8 with biases.  Read and written once a row, by every
  // lane at its own place: no barrier, and some 1 us of the 12 that such a row takes a compute unit.
  constexpr bool kInLds = JOIN && (P * V == 16 || (BIAS && P * V == 8)), kAllInLds = kInLds && P * V == 8;
  typedef ColumnSums<P, V, kInLds> SumsW;
  typedef ColumnSums<P, V, kAllInLds> SumsB;
  // those, or for registers one such array in which rows side by side meet
  constexpr int kLds = kInLds ? 2 * SumsW::kFloats + 2 * SumsB::kFloats : kMaxWaves * kWave * V;
  __shared__ __attribute__((aligned(16))) float lds[kLds];
  const uint32_t L = A.lanes;
  const uint32_t part = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave / A.waves);
  const uint32_t lane0 = threadIdx.x - part * A.waves * kWave;
  RowSums sums(red, part, A.waves, L);
  const float over = 1.f / (float)A.cols;

  // One row's inputs, as they come from memory.
  Piece<SB, V> dh[P];
  Piece<BB, V> du[P];
  Kept<KEEP, SB, V> r[P];
  Kept<KEEP, BB, V> y[P];
  f32x2_t st1 = {0.f, 1.f}, st2 = {0.f, 1.f};
  auto load = [&](const At& at, uint32_t flags, int64_t row) __attribute__((always_inline)) {
    if (flags & kJoinNorm2) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        du[p] = at.template load<BB>(row_at<BB>(A.du, row, A.lddu), p);
        r[p].load(at, A.r, A.ldr, A.kr, row, p);
      }
      st2 = ldg(reinterpret_cast<const f32x2_t*>(A.stats2) + row);
    }
    if constexpr (JOIN) {
      if (flags & kJoinNeedY) {
#pragma unroll
        for (int p = 0; p < P; ++p) y[p].load(at, A.y, A.ldy, A.ky, row, p);
      }
      if (flags & kJoinDh) {
#pragma unroll
        for (int p = 0; p < P; ++p) dh[p] = at.template load<SB>(row_at<SB>(A.dh, row, A.lddh), p);
      }
      if (flags & kJoinNorm1) st1 = ldg(reinterpret_cast<const f32x2_t*>(A.stats1) + row);
    }
  };

  const uint32_t begin = blockIdx.x * A.per_block;
  const uint32_t end = min(begin + A.per_block, A.pieces);
  Parameters<P, V, WHOLE, BIAS, kAhead> n1;
  Parameters<P, V, WHOLE, false, kAhead> n2;
  n2.keep(At(A, lane0), A, A.before, false, 0);
  SumsW aw(lds), aa(lds + SumsW::kFloats);
  SumsB ac(lds + 2 * SumsW::kFloats), ab(lds + 2 * SumsW::kFloats + SumsB::kFloats);
  aw.clear();
  if constexpr (BIAS) ac.clear();
  for (uint32_t piece = begin; piece < end; ++piece) {
    const uint32_t group = __builtin_amdgcn_readfirstlane(piece / A.per_group);
    // every per_group-th set of L rows of the run: workgroups side by side read side by side
    const int64_t row0 = (int64_t)group * A.gate_rows + (int64_t)(piece - group * A.per_group) * L;
    const int64_t row1 = (int64_t)(group + 1) * A.gate_rows, step = (int64_t)A.per_group * L;
    {
      const At at(A, anew(lane0));
      if (kAhead) load(at, A.flags, min(row0 + part, row1 - 1));
      if constexpr (JOIN) n1.keep(at, A, A.after, A.flags & kJoinRuns, group);
    }
    if constexpr (JOIN) {
      aa.clear();
      if constexpr (BIAS) ab.clear();
    }
    for (int64_t base = row0; base < row1; base += step) {
      const int64_t row = base + part;
      const bool here = row < row1;  // else the waves of `part` only meet the others at the barriers
      const At at(A, anew(lane0));
      const uint32_t flags = anew_uniform(A.flags);
      if (!kAhead) load(at, flags, min(row, row1 - 1));
      if (!here) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
          du[p].w = 0u;
          dh[p].w = 0u;
          r[p].clear();
          y[p].clear();
        }
        st1 = st2 = f32x2_t{0.f, 1.f};
      }
      float yn[P][V], hn[P][V], dt[P][V], gu[P][V];
      float t[2] = {0.f, 0.f};
      const float mean1 = st1[0], s1 = st1[1], mean2 = st2[0], s2 = st2[1];
      float token = 1.f;
      if constexpr (JOIN) {
        if (here && (flags & kJoinToken)) token = load_token(A, row);
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int e = 0; e < V; ++e) yn[p][e] = dt[p][e] = 0.f;
        if (flags & kJoinDh) {
#pragma unroll
          for (int p = 0; p < P; ++p) {
            at.fix(dh[p], p);
#pragma unroll
            for (int e = 0; e < V; ++e) dt[p][e] = elem(dh[p], e);
          }
        }
        if (flags & kJoinNeedY) {
#pragma unroll
          for (int p = 0; p < P; ++p) {
            y[p].get(at, A.ky, p, yn[p]);
#pragma unroll
            for (int e = 0; e < V; ++e) yn[p][e] = (yn[p][e] - mean1) * s1;
          }
        }
      }
      if (flags & kJoinNorm2) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
          r[p].get(at, A.kr, p, hn[p]);
          at.fix(du[p], p);
          float w[V], b[V];
          if constexpr (JOIN) {
            n1.get(at, A, A.after, flags & kJoinRuns, p, w, b);
            if (flags & kJoinToken) {
#pragma unroll
              for (int e = 0; e < V; ++e)
                hn[p][e] = __builtin_fmaf(token, __builtin_fmaf(yn[p][e], w[e], b[e]),
                                          __builtin_fmaf(A.scale, hn[p][e], -mean2));
            } else {
#pragma unroll
              for (int e = 0; e < V; ++e) {
                hn[p][e] = __builtin_fmaf(A.scale, hn[p][e], BIAS ? b[e] - mean2 : -mean2);
                hn[p][e] = __builtin_fmaf(yn[p][e], w[e], hn[p][e]);
              }
            }
          }
          n2.get(at, A, A.before, false, p, w, b);
          float sw[V], sc[V];
          aw.get(p, sw);
          if constexpr (BIAS) ac.get(p, sc);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            hn[p][e] = JOIN ? hn[p][e] * s2 : (hn[p][e] - mean2) * s2;
            const float d = elem(du[p], e);
            gu[p][e] = d * w[e];
            sw[e] = __builtin_fmaf(d, hn[p][e], sw[e]);
            if constexpr (BIAS) sc[e] += d;
            t[0] = __builtin_fmaf(gu[p][e], hn[p][e], t[0]);
          }
          aw.put(p, sw);
          if constexpr (BIAS) ac.put(p, sc);
          if (flags & kJoinMean2) {
#pragma unroll
            for (int e = 0; e < V; ++e) t[1] += gu[p][e];
          }
        }
      }
      if (kAhead && base + step < row1) load(at, flags, min(row + step, row1 - 1));  // in flight while this row is worked on
      if (flags & kJoinNorm2) {
        float m1 = 0.f;
        if (flags & kJoinMean2) {
          sums.total(t);
          m1 = -s2 * (t[1] * over);
        } else {
          t[0] = sums.total1(t[0]);
        }
        const float m0 = -s2 * (t[0] * over);
#pragma unroll
        for (int p = 0; p < P; ++p) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            // s (g - mean(g) - hn mean(g hn))
            const float d = __builtin_fmaf(hn[p][e], m0, JOIN ? dt[p][e] + m1 : m1);
            dt[p][e] = __builtin_fmaf(gu[p][e], s2, d);
          }
        }
      }
      if (here && A.dr != nullptr) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
          float o[V];
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] = JOIN ? A.scale * dt[p][e] : dt[p][e];
          at.template store<SB>(row_at<SB>(A.dr, row, A.lddr), p, o);
        }
      }
      if constexpr (JOIN) {
        float dtoken = 0.f;
        t[0] = t[1] = 0.f;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          float w[V], b[V];
          n1.get(at, A, A.after, flags & kJoinRuns, p, w, b);
          if (flags & kJoinToken) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
              dtoken = __builtin_fmaf(dt[p][e], __builtin_fmaf(yn[p][e], w[e], b[e]), dtoken);
              dt[p][e] *= token;
            }
          }
          float sa[V], sb[V];
          aa.get(p, sa);
          if constexpr (BIAS) ab.get(p, sb);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            sa[e] = __builtin_fmaf(dt[p][e], yn[p][e], sa[e]);
            if constexpr (BIAS) sb[e] += dt[p][e];
            dt[p][e] *= w[e];  // dz w
            t[0] = __builtin_fmaf(dt[p][e], yn[p][e], t[0]);
          }
          aa.put(p, sa);
          if constexpr (BIAS) ab.put(p, sb);
          if (flags & kJoinMean1) {
#pragma unroll
            for (int e = 0; e < V; ++e) t[1] += dt[p][e];
          }
        }
        float m0 = 0.f, m1 = 0.f;
        if (flags & kJoinMean1) {
          sums.total(t);
          m0 = -s1 * (t[0] * over);
          m1 = -s1 * (t[1] * over);
        } else if (flags & kJoinNorm1) {
          m0 = -s1 * (sums.total1(t[0]) * over);
        }
        if (A.dtoken != nullptr) {
          dtoken = sums.total1(dtoken);
          if (here && at.lane == 0) {
            if (A.gate_bf16) {
              stg(static_cast<uint16_t*>(A.dtoken) + row, f32_to_bf16_bits(dtoken));
            } else {
              stg(static_cast<float*>(A.dtoken) + row, dtoken);
            }
          }
        }
        // Without a norm yn is the branch, and infinities times m0 = 0 are no part of dz.
        if (!(flags & kJoinNorm1)) {
#pragma unroll
          for (int p = 0; p < P; ++p)
#pragma unroll
            for (int e = 0; e < V; ++e) yn[p][e] = 0.f;
        }
        if (here && A.dy != nullptr) {
#pragma unroll
          for (int p = 0; p < P; ++p) {
            float o[V];
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = __builtin_fmaf(dt[p][e], s1, __builtin_fmaf(yn[p][e], m0, m1));
            at.template store<BB>(row_at<BB>(A.dy, row, A.lddy), p, o);
          }
        }
      }
    }
    if constexpr (JOIN) {
      if (A.pa != nullptr) store_sums(aa, A.pa + piece * (int64_t)A.pitch, A, lane0, part, lds);
      if constexpr (BIAS) {
        if (A.pb != nullptr) store_sums(ab, A.pb + piece * (int64_t)A.pitch, A, lane0, part, lds);
      }
    }
  }
  if (A.flags & kJoinNorm2) {
    if (A.pw != nullptr) store_sums(aw, A.pw + blockIdx.x * (int64_t)A.pitch, A, lane0, part, lds);
    if constexpr (BIAS) {
      if (A.pc != nullptr) store_sums(ac, A.pc + blockIdx.x * (int64_t)A.pitch, A, lane0, part, lds);
    }
  }
}

}  // namespace shp
