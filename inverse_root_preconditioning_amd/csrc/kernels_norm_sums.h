// Gradients of a join's parameters from the partial sums of its backward kernel.
#pragma once

#include "kernels_norm.h"

namespace shp {

// out[c] = sum over s of gate[s / per_group][c] part[s][c] (no gate: 1).
struct SumJob {
  const float* part;
  const void* gate;
  void* out;
  int64_t count;
  int gate_bf16, out_bf16;
};

struct SumArgs {
  SumJob job[4];
  int jobs;
  // the gate's rows, after the jobs: dgate[g][c] = w[c] sum of pa + b[c] sum of pb over the pieces of g
  const float *pa, *pb;
  NormSide after;
  void* dgate;
  int dgate_bf16;
  int64_t groups;
  uint32_t per_group;
  int64_t cols, pitch;
};

__device__ __forceinline__ float param_at(const void* p, int bf16, int64_t i) {
  if (bf16) return __builtin_bit_cast(float, (uint32_t)ldg(static_cast<const uint16_t*>(p) + i) << 16);
  return ldg(static_cast<const float*>(p) + i);
}
__device__ __forceinline__ void store_param(void* p, int bf16, int64_t i, float v) {
  if (bf16) {
    stg(static_cast<uint16_t*>(p) + i, f32_to_bf16_bits(v));
  } else {
    stg(static_cast<float*>(p) + i, v);
  }
}

constexpr int kSumLanes = 64;  // rows of partial sums that a workgroup reads side by side
constexpr int kSumCols = 16;   // columns of a workgroup

// The partial sums are few rows (those of the workgroups that were resident), read from
// the last-level cache by 64 lanes a column: 256 rows of 2048 columns 4 us, three
// such sums together 4.1, most of it the launch and one load's latency.
// kSumCols columns a workgroup, blockIdx.y the job or (after the jobs) the gate's row.
__global__ void __launch_bounds__(kSumCols * kSumLanes) join_sums_kernel(const SumArgs S) {
  __shared__ float lds[kSumLanes][kSumCols];
  const int c = threadIdx.x % kSumCols, part = threadIdx.x / kSumCols;
  const int64_t col = (int64_t)blockIdx.x * kSumCols + c;
  const bool in = col < S.cols;
  float v = 0.f;
  if ((int)blockIdx.y < S.jobs) {
    const SumJob J = S.job[blockIdx.y];
    if (in) {
#pragma unroll 16
      for (int64_t s = part; s < J.count; s += kSumLanes) {
        float g = 1.f;
        if (J.gate != nullptr) g = param_at(J.gate, J.gate_bf16, (s / S.per_group) * S.cols + col);
        v = __builtin_fmaf(g, ldg(J.part + s * S.pitch + col), v);
      }
    }
  } else if (in) {
    const int64_t s0 = (int64_t)(blockIdx.y - S.jobs) * S.per_group;
    const float w = S.after.w != nullptr ? param_at(S.after.w, S.after.w_bf16, col) : 1.f;
    const float b = S.pb != nullptr && S.after.b != nullptr ? param_at(S.after.b, S.after.b_bf16, col) : 0.f;
#pragma unroll 8
    for (uint32_t s = part; s < S.per_group; s += kSumLanes) {
      const int64_t at = (s0 + s) * S.pitch + col;
      v = __builtin_fmaf(w, ldg(S.pa + at), v);
      if (S.pb != nullptr) v = __builtin_fmaf(b, ldg(S.pb + at), v);
    }
  }
  lds[part][c] = v;
  __syncthreads();
  if (part != 0 || !in) return;
  v = 0.f;
#pragma unroll
  for (int i = 0; i < kSumLanes; ++i) v += lds[i][c];
  if ((int)blockIdx.y < S.jobs) {
    store_param(S.job[blockIdx.y].out, S.job[blockIdx.y].out_bf16, col, v);
  } else {
    store_param(S.dgate, S.dgate_bf16, (int64_t)(blockIdx.y - S.jobs) * S.cols + col, v);
  }
}

// The gate's rows where each has few pieces: a column a thread, blockIdx.y the first of the rows that it takes.
__global__ void __launch_bounds__(256) join_gate_kernel(const SumArgs S) {
  const int64_t col = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (col >= S.cols) return;
  const float w = S.after.w != nullptr ? param_at(S.after.w, S.after.w_bf16, col) : 1.f;
  const float b = S.pb != nullptr && S.after.b != nullptr ? param_at(S.after.b, S.after.b_bf16, col) : 0.f;
  for (int64_t g = blockIdx.y; g < S.groups; g += gridDim.y) {
    float v = 0.f;
    for (uint32_t s = 0; s < S.per_group; ++s) {
      const int64_t at = (g * S.per_group + s) * S.pitch + col;
      v = __builtin_fmaf(w, ldg(S.pa + at), v);
      if (S.pb != nullptr) v = __builtin_fmaf(b, ldg(S.pb + at), v);
    }
    store_param(S.dgate, S.dgate_bf16, g * S.cols + col, v);
  }
}

}  // namespace shp
