// C entry points of the MX8 conversion and the activations (gfx950): arguments
// are checked on the host, kernels enqueued on the caller's stream; nothing is
// allocated and nothing synchronises.
#include "host.h"
#include "kernels_act.h"

using namespace shp;

namespace {

// Shape and grid of a pass with `passes` rows a thread; 0 workgroups: more than a launch takes.
uint32_t shape_of(int64_t rows, int64_t padded, bool bf16, int passes, RowShape* shape) {
  int64_t col_blocks;
  row_shape(padded, bf16 ? 8 : 4, &shape->lanes_log2, &col_blocks);
  const int64_t per_block = (int64_t)passes * (256 >> shape->lanes_log2);
  const int64_t blocks = col_blocks * ((rows + per_block - 1) / per_block);
  shape->col_blocks = (uint32_t)col_blocks;
  return blocks > kMaxThreads / 256 ? 0 : (uint32_t)blocks;
}

Mx8Rows mx8_rows(const uint8_t* codes, const uint8_t* scales, int64_t cols) {
  return Mx8Rows{const_cast<uint8_t*>(codes), const_cast<uint8_t*>(scales),
                 (uint32_t)mx8_padded(cols)};
}

template <bool BACK, bool BF16, int ACT, bool GATED, bool KEEP>
int launch_act(const ActArgs& a, uint32_t blocks, hipStream_t stream) {
  if constexpr (BACK) {
    hipLaunchKernelGGL((act_backward_kernel<BF16, ACT, GATED, KEEP>), dim3(blocks), dim3(256), 0, stream, a);
  } else {
    hipLaunchKernelGGL((act_forward_kernel<BF16, ACT, GATED, KEEP>), dim3(blocks), dim3(256), 0, stream, a);
  }
  return check_launch();
}

template <bool BACK, bool BF16, int ACT>
int launch_act(const ActArgs& a, bool gated, bool keep, uint32_t blocks, hipStream_t stream) {
  if (gated) return keep ? launch_act<BACK, BF16, ACT, true, true>(a, blocks, stream)
                         : launch_act<BACK, BF16, ACT, true, false>(a, blocks, stream);
  return keep ? launch_act<BACK, BF16, ACT, false, true>(a, blocks, stream)
              : launch_act<BACK, BF16, ACT, false, false>(a, blocks, stream);
}

template <bool BACK, bool BF16>
int launch_act(int act, const ActArgs& a, bool gated, bool keep, uint32_t blocks, hipStream_t stream) {
  switch (act) {
    case SHAMPOO_ACT_SILU: return launch_act<BACK, BF16, SHAMPOO_ACT_SILU>(a, gated, keep, blocks, stream);
    case SHAMPOO_ACT_GELU: return launch_act<BACK, BF16, SHAMPOO_ACT_GELU>(a, gated, keep, blocks, stream);
    case SHAMPOO_ACT_GELU_TANH: return launch_act<BACK, BF16, SHAMPOO_ACT_GELU_TANH>(a, gated, keep, blocks, stream);
    case SHAMPOO_ACT_RELU: return launch_act<BACK, BF16, SHAMPOO_ACT_RELU>(a, gated, keep, blocks, stream);
    default: return launch_act<BACK, BF16, SHAMPOO_ACT_RELU2>(a, gated, keep, blocks, stream);
  }
}

bool valid_act(int act) { return act >= SHAMPOO_ACT_SILU && act <= SHAMPOO_ACT_RELU2; }

}  // namespace

extern "C" {

int shampoo_mx8_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                         uint8_t* scales, hipStream_t stream) {
  if (!valid_type(dtype)) return SHAMPOO_EUNSUPPORTED;
  const int rc = check_sides(rows, cols);
  if (rc != SHAMPOO_OK) return rc;
  if (ld < cols) return SHAMPOO_EINVAL;
  if (rows == 0 || cols == 0) return SHAMPOO_OK;
  if (x == nullptr || !valid_mx8(codes, scales)) return SHAMPOO_EINVAL;
  Mx8Args a = {};
  a.x = x;
  a.rows = rows;
  a.cols = (uint32_t)cols;
  a.ld = ld;
  a.m = mx8_rows(codes, scales, cols);
  const bool bf16 = dtype == SHAMPOO_T_BF16;
  const uint32_t blocks = shape_of(rows, a.m.padded, bf16, kMx8Passes, &a.shape);
  if (blocks == 0) return SHAMPOO_EUNSUPPORTED;
  if (bf16) {
    hipLaunchKernelGGL(mx8_quantize_kernel<true>, dim3(blocks), dim3(256), 0, stream, a);
  } else {
    hipLaunchKernelGGL(mx8_quantize_kernel<false>, dim3(blocks), dim3(256), 0, stream, a);
  }
  return check_launch();
}

int shampoo_mx8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out,
                           int dtype, int64_t ld, hipStream_t stream) {
  if (!valid_type(dtype)) return SHAMPOO_EUNSUPPORTED;
  const int rc = check_sides(rows, cols);
  if (rc != SHAMPOO_OK) return rc;
  if (ld < cols) return SHAMPOO_EINVAL;
  if (rows == 0 || cols == 0) return SHAMPOO_OK;
  if (!valid_mx8(codes, scales) || out == nullptr) return SHAMPOO_EINVAL;
  Mx8Args a = {};
  a.out = out;
  a.rows = rows;
  a.cols = (uint32_t)cols;
  a.ld = ld;
  a.m = mx8_rows(codes, scales, cols);
  const bool bf16 = dtype == SHAMPOO_T_BF16;
  const uint32_t blocks = shape_of(rows, cols, bf16, kMx8Passes, &a.shape);
  if (blocks == 0) return SHAMPOO_EUNSUPPORTED;
  if (bf16) {
    hipLaunchKernelGGL(mx8_dequantize_kernel<true>, dim3(blocks), dim3(256), 0, stream, a);
  } else {
    hipLaunchKernelGGL(mx8_dequantize_kernel<false>, dim3(blocks), dim3(256), 0, stream, a);
  }
  return check_launch();
}

int shampoo_activation(int act, const void* a, int64_t lda, const void* b, int64_t ldb, int64_t rows, int64_t cols,
                       int dtype, void* y, int64_t ldy, uint8_t* a_codes, uint8_t* a_scales, uint8_t* b_codes,
                       uint8_t* b_scales, hipStream_t stream) {
  if (!valid_type(dtype) || !valid_act(act)) return SHAMPOO_EUNSUPPORTED;
  const int rc = check_sides(rows, cols);
  if (rc != SHAMPOO_OK) return rc;
  const bool gated = b != nullptr, keep = a_codes != nullptr;
  if (lda < cols || ldy < cols || (gated && ldb < cols)) return SHAMPOO_EINVAL;
  if (rows == 0 || cols == 0) return SHAMPOO_OK;
  if (a == nullptr || y == nullptr) return SHAMPOO_EINVAL;
  if (keep ? !valid_mx8(a_codes, a_scales) : a_scales != nullptr) return SHAMPOO_EINVAL;
  if (keep && gated ? !valid_mx8(b_codes, b_scales) : (b_codes != nullptr || b_scales != nullptr)) return SHAMPOO_EINVAL;
  ActArgs p = {};
  p.a = a;
  p.b = b;
  p.y = y;
  p.lda = lda;
  p.ldb = ldb;
  p.ldy = ldy;
  p.rows = rows;
  p.cols = (uint32_t)cols;
  p.ka = mx8_rows(a_codes, a_scales, cols);
  p.kb = mx8_rows(b_codes, b_scales, cols);
  const bool bf16 = dtype == SHAMPOO_T_BF16;
  const uint32_t blocks = shape_of(rows, mx8_padded(cols), bf16, kActPasses, &p.shape);
  if (blocks == 0) return SHAMPOO_EUNSUPPORTED;
  return bf16 ? launch_act<false, true>(act, p, gated, keep, blocks, stream)
              : launch_act<false, false>(act, p, gated, keep, blocks, stream);
}

int shampoo_activation_backward(int act, const void* dy, int64_t lddy, const void* a, int64_t lda, const void* b,
                                int64_t ldb, const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes,
                                const uint8_t* b_scales, int gated, int64_t rows, int64_t cols, int dtype, void* da,
                                int64_t ldda, void* db, int64_t lddb, hipStream_t stream) {
  if (!valid_type(dtype) || !valid_act(act)) return SHAMPOO_EUNSUPPORTED;
  const int rc = check_sides(rows, cols);
  if (rc != SHAMPOO_OK) return rc;
  const bool keep = a_codes != nullptr;
  if (lddy < cols || (da != nullptr && ldda < cols) || (db != nullptr && lddb < cols)) return SHAMPOO_EINVAL;
  if (!keep && (lda < cols || (gated && ldb < cols))) return SHAMPOO_EINVAL;
  if (!gated && db != nullptr) return SHAMPOO_EINVAL;
  if (rows == 0 || cols == 0 || (da == nullptr && db == nullptr)) return SHAMPOO_OK;
  if (dy == nullptr) return SHAMPOO_EINVAL;
  if (keep ? !valid_mx8(a_codes, a_scales) || (gated && !valid_mx8(b_codes, b_scales))
           : a == nullptr || (gated && b == nullptr))
    return SHAMPOO_EINVAL;
  ActArgs p = {};
  p.a = a;
  p.b = b;
  p.dy = dy;
  p.da = da;
  p.db = db;
  p.lda = lda;
  p.ldb = ldb;
  p.lddy = lddy;
  p.ldda = ldda;
  p.lddb = lddb;
  p.rows = rows;
  p.cols = (uint32_t)cols;
  p.ka = mx8_rows(a_codes, a_scales, cols);
  p.kb = mx8_rows(b_codes, b_scales, cols);
  const bool bf16 = dtype == SHAMPOO_T_BF16;
  const uint32_t blocks = shape_of(rows, cols, bf16, kActPasses, &p.shape);
  if (blocks == 0) return SHAMPOO_EUNSUPPORTED;
  return bf16 ? launch_act<true, true>(act, p, gated != 0, keep, blocks, stream)
              : launch_act<true, false>(act, p, gated != 0, keep, blocks, stream);
}

}  // extern "C"
