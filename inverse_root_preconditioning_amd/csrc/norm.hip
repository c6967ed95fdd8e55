// C entry points of norms and joins (gfx950): arguments are checked on the
// host, kernels enqueued on the caller's stream; nothing is allocated and
// nothing synchronises.
#include <algorithm>
#include <cmath>

#include "kernels_norm_sums.h"
#include "norm_launch.h"

using namespace shp;

namespace {

// Rows that a workgroup of the forward kernel takes in turn, where that leaves
// as many as are resident: enough that the parameters' loads do not count
// and a row's loads overlap the row before, few enough that the workgroups end
// together.  Joins of 2^25 bf16 elements with 8-bit copies, us by turns:
// rows of 512:  1: 70, 2: 63, 4: 64;   of 2050 (5 waves)  2: 110, 4: 99, 8: 100;
// of 5120 (10):  5: 78, 8: 83, 9: 71, 10: 76;   of 8192 (16):  1: 97, 4: 68, 8: 65, 12: 80.
// The rule suits up to 8 waves and 16; at 10 its 8 is the slowest of those measured (820 workgroups, whose last ones
// run by themselves).
// Fewer rows, a join and a norm, us with workgroups for one a compute unit and for 16 waves a unit:
// 1001 rows of 1537 fp32 11.7, 6.1 and 9.8, 5.3;  of 700 of 4096 bf16 8.1, 5.2 and 7.3, 4.6;  of 500 of
// 8192 fp32 (16 waves a row, 512 workgroups instead of 256) 12.3, 7.3 and 16.8, 7.5.
int64_t turns(uint32_t waves) { return std::min<int64_t>(std::max<int64_t>(waves - 1, 3), 8); }

template <bool SB, bool BB>
int forward(JoinArgs a, hipStream_t stream) {
  constexpr int V = SB ? 8 : 4;
  const RowLayout layout = row_layout(a.cols, V);
  a.waves = layout.waves;
  a.lanes = a.waves == 1 ? 4 : 1;
  const int64_t rows = (a.rows + a.lanes - 1) / a.lanes, each = turns(a.waves);
  const int64_t resident = 256 * (kMaxWaves / (a.waves * a.lanes));
  const int64_t blocks = std::min(std::max((rows + each - 1) / each, std::min(rows, resident)), kMaxThreads / 1024);
  const dim3 grid((uint32_t)blocks), block(kWave * a.waves * a.lanes);
  const bool whole = a.cols % V == 0;
  return with_pieces<V>(layout.pieces, [&](auto p) {
    constexpr int P = decltype(p)::value;
    if (a.y != nullptr && whole) {
      hipLaunchKernelGGL((join_forward_kernel<SB, BB, P, true, true>), grid, block, 0, stream, a);
    } else if (a.y != nullptr) {
      hipLaunchKernelGGL((join_forward_kernel<SB, BB, P, true, false>), grid, block, 0, stream, a);
    } else if (whole) {
      hipLaunchKernelGGL((join_forward_kernel<SB, BB, P, false, true>), grid, block, 0, stream, a);
    } else {
      hipLaunchKernelGGL((join_forward_kernel<SB, BB, P, false, false>), grid, block, 0, stream, a);
    }
    return check_launch();
  });
}

int valid_norm(const shampoo_norm& n) {
  if (n.kind == SHAMPOO_NORM_NONE) return SHAMPOO_OK;
  if (n.kind != SHAMPOO_NORM_RMS && n.kind != SHAMPOO_NORM_LAYER) return SHAMPOO_EUNSUPPORTED;
  if (!((float)n.eps > 0.f) || !std::isfinite((float)n.eps)) return SHAMPOO_EINVAL;
  if (n.weight != nullptr && !valid_type(n.weight_dtype)) return SHAMPOO_EUNSUPPORTED;
  if (n.bias != nullptr && !valid_type(n.bias_dtype)) return SHAMPOO_EUNSUPPORTED;
  return SHAMPOO_OK;
}

bool has_bias(const shampoo_join& j) { return (j.after.kind != SHAMPOO_NORM_NONE && j.after.bias != nullptr) ||
                                              (j.before.kind != SHAMPOO_NORM_NONE && j.before.bias != nullptr); }

NormSide norm_side(const shampoo_norm& n) {
  NormSide s = {};
  s.kind = (int)n.kind;
  if (n.kind == SHAMPOO_NORM_NONE) return s;
  s.w = n.weight;
  s.b = n.bias;
  s.w_bf16 = n.weight_dtype == SHAMPOO_T_BF16;
  s.b_bf16 = n.bias_dtype == SHAMPOO_T_BF16;
  s.eps = (float)n.eps;
  return s;
}

uint32_t norm_flags(int64_t kind, uint32_t norm, uint32_t mean) {
  return kind == SHAMPOO_NORM_NONE ? 0 : kind == SHAMPOO_NORM_LAYER ? norm | mean : norm;
}

// What both directions check; `empty` where there is nothing to do.
int common(const shampoo_join* j, JoinArgs* a, bool* empty) {
  if (j == nullptr) return SHAMPOO_EINVAL;
  *empty = false;
  if (!valid_type(j->stream_dtype) || !valid_type(j->branch_dtype)) return SHAMPOO_EUNSUPPORTED;
  if (j->stream_dtype == SHAMPOO_T_BF16 && j->branch_dtype == SHAMPOO_T_F32) return SHAMPOO_EUNSUPPORTED;
  int rc = check_sides(j->rows, j->cols);
  if (rc != SHAMPOO_OK) return rc;
  if (j->cols > SHAMPOO_NORM_COLS) return SHAMPOO_EUNSUPPORTED;
  if ((rc = valid_norm(j->after)) != SHAMPOO_OK || (rc = valid_norm(j->before)) != SHAMPOO_OK) return rc;
  if (j->gate_kind < SHAMPOO_GATE_NONE || j->gate_kind > SHAMPOO_GATE_TOKEN) return SHAMPOO_EUNSUPPORTED;
  const bool join = j->branch != nullptr;
  if (!join && (j->after.kind != SHAMPOO_NORM_NONE || j->gate_kind != SHAMPOO_GATE_NONE ||
                j->before.kind == SHAMPOO_NORM_NONE))
    return SHAMPOO_EINVAL;
  if (j->gate_kind != SHAMPOO_GATE_NONE && !valid_type(j->gate_dtype)) return SHAMPOO_EUNSUPPORTED;
  if (j->gate_kind == SHAMPOO_GATE_ROWS && (j->gate_rows < 1 || j->gate_rows > kMaxRows || j->rows % j->gate_rows != 0))
    return SHAMPOO_EINVAL;
  if (join && !std::isfinite((float)j->scale)) return SHAMPOO_EINVAL;
  if (j->rows == 0 || j->cols == 0) {
    *empty = true;
    return SHAMPOO_OK;
  }
  if (j->gate_kind != SHAMPOO_GATE_NONE && j->gate == nullptr) return SHAMPOO_EINVAL;
  *a = JoinArgs{};
  a->rows = j->rows;
  a->cols = (uint32_t)j->cols;
  a->scale = join ? (float)j->scale : 1.f;
  a->r = j->residual;
  a->y = j->branch;
  a->ldr = j->ld_residual;
  a->ldy = j->ld_branch;
  const uint32_t padded = (uint32_t)mx8_padded(j->cols);
  a->kr = Mx8Rows{j->residual_codes, j->residual_scales, padded};
  a->ky = Mx8Rows{j->branch_codes, j->branch_scales, padded};
  if ((a->kr.codes != nullptr || a->kr.scales != nullptr) && !valid_mx8(a->kr.codes, a->kr.scales))
    return SHAMPOO_EINVAL;
  if ((a->ky.codes != nullptr || a->ky.scales != nullptr) && !valid_mx8(a->ky.codes, a->ky.scales))
    return SHAMPOO_EINVAL;
  if (!join && a->ky.codes != nullptr) return SHAMPOO_EINVAL;
  a->after = norm_side(j->after);
  a->before = norm_side(j->before);
  a->gate = j->gate;
  a->gate_bf16 = j->gate_dtype == SHAMPOO_T_BF16;
  a->gate_rows = (uint32_t)(j->gate_kind == SHAMPOO_GATE_ROWS ? j->gate_rows : j->rows);
  a->flags = norm_flags(j->after.kind, kJoinNorm1, kJoinMean1) | norm_flags(j->before.kind, kJoinNorm2, kJoinMean2);
  if (j->gate_kind == SHAMPOO_GATE_ROWS) a->flags |= kJoinRuns;
  if (j->gate_kind == SHAMPOO_GATE_TOKEN) a->flags |= kJoinToken;
  if ((reinterpret_cast<uintptr_t>(j->after_stats) & 7) != 0 || (reinterpret_cast<uintptr_t>(j->before_stats) & 7) != 0)
    return SHAMPOO_EINVAL;
  a->stats1 = j->after_stats;
  a->stats2 = j->before_stats;
  return SHAMPOO_OK;
}

// How the rows go to the backward kernel's workgroups: as many as are resident,
// each within one run of rows that share a gate row, or (short runs) with whole ones.
struct Split {
  int64_t groups, pieces, blocks;
  uint32_t per_group, per_block;
  RowLayout layout;
  uint32_t lanes;
};
Split split_rows(const shampoo_join& j) {
  Split s;
  const bool bf16 = j.stream_dtype == SHAMPOO_T_BF16;
  s.layout = row_layout(j.cols, bf16 ? 8 : 4);
  const BackGrid grid = back_grid(s.layout, bf16 ? 8 : 4);
  s.lanes = grid.lanes;
  const int64_t run = j.gate_kind == SHAMPOO_GATE_ROWS ? j.gate_rows : j.rows;
  const int64_t want = (((j.rows + grid.resident - 1) / grid.resident) + s.lanes - 1) / s.lanes * s.lanes;
  s.groups = j.rows / run;
  s.per_group = (uint32_t)((run + want - 1) / want);
  s.pieces = s.groups * s.per_group;
  s.per_block = (uint32_t)std::max<int64_t>(1, want / run);
  s.blocks = (s.pieces + s.per_block - 1) / s.per_block;
  return s;
}

int64_t pitch_of(int64_t cols) { return (cols + 7) / 8 * 8; }

// Bytes of the partial sums: rows for each workgroup, and for each piece where gradients of what
// multiplies or follows the normed branch are wanted (no g: those of every parameter that there is).
size_t sums_bytes(const shampoo_join& j, const Split& s, const shampoo_join_grads* g) {
  const bool norm = j.after.kind != SHAMPOO_NORM_NONE, weight = norm && j.after.weight != nullptr;
  const bool bias = norm && j.after.bias != nullptr;
  const bool gate = j.gate_kind == SHAMPOO_GATE_ROWS && (g == nullptr || g->d_gate != nullptr);
  const bool scaled = gate || (weight && (g == nullptr || g->d_after_weight != nullptr));
  const bool added = bias && (gate || g == nullptr || g->d_after_bias != nullptr);
  const int64_t rows = s.blocks * (has_bias(j) ? 2 : 1) + s.pieces * ((int)scaled + (int)added);
  return (size_t)rows * (size_t)pitch_of(j.cols) * sizeof(float);
}

}  // namespace

extern "C" {

int shampoo_join_forward(const shampoo_join* join, void* h, int64_t ld_h, void* u, int64_t ld_u, hipStream_t stream) {
  JoinArgs a;
  bool empty;
  const int rc = common(join, &a, &empty);
  if (rc != SHAMPOO_OK) return rc;
  const bool has_y = join->branch != nullptr, has_u = join->before.kind != SHAMPOO_NORM_NONE;
  const int64_t cols = join->cols;
  if (join->ld_residual < cols || (has_y && (join->ld_branch < cols || ld_h < cols)) || (has_u && ld_u < cols))
    return SHAMPOO_EINVAL;
  if (empty) return SHAMPOO_OK;
  if (a.r == nullptr || (has_y && h == nullptr) || (has_u && u == nullptr)) return SHAMPOO_EINVAL;
  if (a.kr.codes != nullptr) a.flags |= kJoinCodesR;
  if (a.ky.codes != nullptr) a.flags |= kJoinCodesY;
  a.h = h;
  a.ldh = ld_h;
  a.u = u;
  a.ldu = ld_u;
  if (join->stream_dtype == SHAMPOO_T_BF16) return forward<true, true>(a, stream);
  return join->branch_dtype == SHAMPOO_T_BF16 ? forward<false, true>(a, stream) : forward<false, false>(a, stream);
}

size_t shampoo_join_backward_workspace_bytes(const shampoo_join* join, const shampoo_join_grads* g) {
  JoinArgs a;
  bool empty;
  if (common(join, &a, &empty) != SHAMPOO_OK || empty) return 0;
  return sums_bytes(*join, split_rows(*join), g);
}

size_t shampoo_join_workspace_bytes(const shampoo_join* join) {
  return shampoo_join_backward_workspace_bytes(join, nullptr);
}

int shampoo_join_backward(const shampoo_join* join, const shampoo_join_grads* g, void* ws, size_t ws_bytes,
                          hipStream_t stream) {
  JoinArgs a;
  bool empty;
  int rc = common(join, &a, &empty);
  if (rc != SHAMPOO_OK) return rc;
  if (g == nullptr) return SHAMPOO_EINVAL;
  const bool has_y = join->branch != nullptr, has1 = join->after.kind != SHAMPOO_NORM_NONE;
  const bool has2 = join->before.kind != SHAMPOO_NORM_NONE && g->d_u != nullptr;
  const bool gated = join->gate_kind != SHAMPOO_GATE_NONE;
  const int64_t cols = join->cols;
  if ((g->d_h != nullptr && g->ld_d_h < cols) || (g->d_u != nullptr && g->ld_d_u < cols) ||
      (g->d_residual != nullptr && g->ld_d_residual < cols) || (g->d_branch != nullptr && g->ld_d_branch < cols))
    return SHAMPOO_EINVAL;
  if (!has_y && (g->d_h != nullptr || g->d_branch != nullptr)) return SHAMPOO_EINVAL;
  if (g->d_u != nullptr && join->before.kind == SHAMPOO_NORM_NONE) return SHAMPOO_EINVAL;
  if ((g->d_after_weight != nullptr && (!has1 || join->after.weight == nullptr)) ||
      (g->d_after_bias != nullptr && (!has1 || join->after.bias == nullptr)) || (g->d_gate != nullptr && !gated) ||
      (g->d_before_weight != nullptr && (!has2 || join->before.weight == nullptr)) ||
      (g->d_before_bias != nullptr && (!has2 || join->before.bias == nullptr)))
    return SHAMPOO_EINVAL;
  if (empty) return SHAMPOO_OK;
  if (g->d_h == nullptr && !has2) return SHAMPOO_EINVAL;
  // what is read: inputs, or their copies
  const bool need_r = has2, need_y = has_y && (has1 || gated || has2);
  const bool keep = a.kr.codes != nullptr || a.ky.codes != nullptr;
  if (keep) {
    if ((need_r && a.kr.codes == nullptr) || (need_y && a.ky.codes == nullptr)) return SHAMPOO_EINVAL;
  } else {
    if (need_r && (a.r == nullptr || join->ld_residual < cols)) return SHAMPOO_EINVAL;
    if (need_y && join->ld_branch < cols) return SHAMPOO_EINVAL;
  }
  if ((has1 && a.stats1 == nullptr) || (has2 && a.stats2 == nullptr)) return SHAMPOO_EINVAL;
  const int64_t gate_rows = join->gate_kind == SHAMPOO_GATE_ROWS ? join->gate_rows : 0;
  const Split s = split_rows(*join);
  if (ws == nullptr || ws_bytes < sums_bytes(*join, s, g)) return SHAMPOO_EWORKSPACE;
  if (!aligned16(ws)) return SHAMPOO_EINVAL;
  if (s.blocks > kMaxThreads / 1024) return SHAMPOO_EUNSUPPORTED;
  a.dh = g->d_h;
  a.lddh = g->ld_d_h;
  a.du = has2 ? g->d_u : nullptr;
  a.lddu = g->ld_d_u;
  a.dr = g->d_residual;
  a.lddr = g->ld_d_residual;
  a.dy = g->d_branch;
  a.lddy = g->ld_d_branch;
  if (!has2) a.flags &= ~(kJoinNorm2 | kJoinMean2);
  if (need_y) a.flags |= kJoinNeedY;
  if (a.dh != nullptr) a.flags |= kJoinDh;
  a.pieces = (uint32_t)s.pieces;
  a.per_group = s.per_group;
  a.per_block = s.per_block;
  a.waves = s.layout.waves;
  a.lanes = s.lanes;
  a.pitch = (uint32_t)pitch_of(cols);
  if (join->gate_kind == SHAMPOO_GATE_TOKEN) {
    a.dtoken = g->d_gate;
  }
  const bool gate_sums = gate_rows > 0 && g->d_gate != nullptr;
  float* part = static_cast<float*>(ws);
  auto place = [&](bool wanted, int64_t rows) {
    float* const at = wanted ? part : nullptr;
    if (wanted) part += rows * a.pitch;
    return at;
  };
  a.pa = place(g->d_after_weight != nullptr || gate_sums, s.pieces);
  a.pw = place(g->d_before_weight != nullptr, s.blocks);
  a.pb = place(g->d_after_bias != nullptr || (gate_sums && a.after.b != nullptr), s.pieces);
  a.pc = place(g->d_before_bias != nullptr, s.blocks);
  const bool bias = has_bias(*join);
  const uint32_t blocks = (uint32_t)s.blocks;
  if (join->stream_dtype == SHAMPOO_T_BF16) {
    rc = join_backward_bf16(a, s.layout.pieces, keep, bias, blocks, stream);
  } else if (join->branch_dtype == SHAMPOO_T_BF16) {
    rc = join_backward_mixed(a, s.layout.pieces, keep, bias, blocks, stream);
  } else {
    rc = join_backward_f32(a, s.layout.pieces, keep, bias, blocks, stream);
  }
  if (rc != SHAMPOO_OK) return rc;
  SumArgs m = {};
  auto job = [&](const float* from, int64_t count, bool gate, void* out, bool bf16) {
    if (out == nullptr) return;
    SumJob& J = m.job[m.jobs++];
    J.part = from;
    J.count = count;
    J.gate = gate ? a.gate : nullptr;
    J.gate_bf16 = a.gate_bf16;
    J.out = out;
    J.out_bf16 = bf16;
  };
  job(a.pw, s.blocks, false, g->d_before_weight, a.before.w_bf16);
  job(a.pc, s.blocks, false, g->d_before_bias, a.before.b_bf16);
  job(a.pa, s.pieces, gate_rows > 0, g->d_after_weight, a.after.w_bf16);
  job(a.pb, s.pieces, gate_rows > 0, g->d_after_bias, a.after.b_bf16);
  m.per_group = s.per_group;
  m.cols = cols;
  m.pitch = a.pitch;
  int64_t rows_y = m.jobs;
  if (gate_sums) {
    m.pa = a.pa;
    m.pb = a.after.b != nullptr ? a.pb : nullptr;
    m.after = a.after;
    m.dgate = g->d_gate;
    m.dgate_bf16 = a.gate_bf16;
    m.groups = s.groups;
    // Rows with some pieces each are summed like the jobs, beside them; else by a thread an element.
    if (s.per_group > 4 && s.groups <= 1024) {
      rows_y += s.groups;
    } else {
      hipLaunchKernelGGL(join_gate_kernel,
                         dim3((uint32_t)((cols + 255) / 256), (uint32_t)std::min<int64_t>(s.groups, 4096)), dim3(256), 0,
                         stream, m);
      if ((rc = check_launch()) != SHAMPOO_OK) return rc;
    }
  }
  if (rows_y == 0) return SHAMPOO_OK;
  hipLaunchKernelGGL(join_sums_kernel, dim3((uint32_t)((cols + kSumCols - 1) / kSumCols), (uint32_t)rows_y),
                     dim3(kSumCols * kSumLanes), 0,
                     stream, m);
  return check_launch();
}

}  // extern "C"
