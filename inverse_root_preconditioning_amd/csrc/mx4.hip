// C entry points of the MX4 quantisation and products (gfx950): arguments are
// checked on the host, kernels enqueued on the caller's stream; nothing is
// allocated and nothing synchronises.
#include <algorithm>
#include <cmath>

#include "kernels_mx4.h"

using namespace shp;

namespace {

// A launch has fewer than 2^32 threads along x, 256 of them in a workgroup.
constexpr int64_t kMaxGrid = 0xffffffff / 256;
constexpr int64_t kMaxSide = (int64_t)1 << 31;  // rows and columns of a matrix
constexpr int64_t kMaxK = (int64_t)1 << 24;     // columns a product sums over (32-bit offsets within a tile)

int check_launch() { return hipGetLastError() == hipSuccess ? SHAMPOO_OK : SHAMPOO_EHIP; }

bool valid_type(int t) { return t == SHAMPOO_T_F32 || t == SHAMPOO_T_BF16; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

int check_sides(int64_t a, int64_t b, int64_t c) {
  if (a < 0 || b < 0 || c < 0) return SHAMPOO_EINVAL;
  if (a > kMaxSide || b > kMaxSide || c > kMaxSide) return SHAMPOO_EUNSUPPORTED;
  return SHAMPOO_OK;
}

bool valid_mx4(const uint8_t* codes, const uint8_t* scales) {
  return codes != nullptr && scales != nullptr && aligned16(codes) && aligned16(scales);
}

// Whether an [M][a] and an [M][b] matrix with rows lda and ldb elements of
// `size` bytes apart may share memory.  Of one row distance (two stretches of
// one matrix's columns) that is told exactly, else by the ends alone.
bool may_overlap(const void* pa, int64_t a, int64_t lda, const void* pb, int64_t b, int64_t ldb, int64_t M,
                 int64_t size) {
  typedef __int128 wide;
  const wide a0 = (wide) reinterpret_cast<uintptr_t>(pa), b0 = (wide) reinterpret_cast<uintptr_t>(pb);
  const wide wa = (wide)a * size, wb = (wide)b * size, row = (wide)lda * size;
  if (a0 + (M - 1) * row + wa <= b0 || b0 + (M - 1) * ((wide)ldb * size) + wb <= a0) return false;
  if (M == 1 || lda != ldb) return true;
  const wide between = ((b0 - a0) % row + row) % row;  // from a row of the first to the next row of the second
  return between < wa || between + wb > row;
}

// Lanes (a power of two, 16 to 256) that take a row of pieces of `elems`, and how
// many such stretches a row has.
void row_shape(int64_t padded, int64_t elems, int* lanes_log2, int64_t* col_blocks) {
  int k = 4;
  while (k < 8 && (elems << k) < padded) ++k;
  *lanes_log2 = k;
  *col_blocks = (padded + (elems << k) - 1) / (elems << k);
}

// Columns (and rows with ROWS) with V elements a lane.
template <bool BF16, int V, bool ROWS>
int quantize_cols(Mx4QuantArgs a, hipStream_t stream) {
  const int64_t width = kWave * V, col_blocks = ((ROWS ? a.padded_cols : a.cols) + width - 1) / width;
  const int64_t blocks = col_blocks * (a.padded_rows / 128);
  if (blocks > kMaxGrid) return SHAMPOO_EUNSUPPORTED;
  a.col_blocks = (uint32_t)col_blocks;
  hipLaunchKernelGGL((mx4_quantize_cols_kernel<BF16, V, ROWS>), dim3((uint32_t)blocks), dim3(256), 0, stream, a);
  return check_launch();
}

template <bool BF16>
int quantize_rows(Mx4QuantArgs a, hipStream_t stream) {
  int64_t col_blocks;
  row_shape(a.padded_cols, 8, &a.lanes_log2, &col_blocks);
  const int64_t per_block = 4 * (256 >> a.lanes_log2), row_blocks = (a.rows + per_block - 1) / per_block;
  if (col_blocks * row_blocks > kMaxGrid) return SHAMPOO_EUNSUPPORTED;
  a.col_blocks = (uint32_t)col_blocks;
  hipLaunchKernelGGL(mx4_quantize_rows_kernel<BF16>, dim3((uint32_t)(col_blocks * row_blocks)), dim3(256), 0, stream,
                     a);
  return check_launch();
}

// Columns take 16 bytes of a row a lane, or two elements where that would leave
// compute units without a workgroup: there a wave's own work is the time.
// Both orientations of 1000 x 1003 bf16: 16.5 us with 16 bytes, 10.5 (the
// host's time) with two elements; of 8192 x 2048: 12.6 and 13.4 us.
constexpr int64_t kSmallQuantBlocks = 256;

template <bool BF16>
int quantize_type(const Mx4QuantArgs& a, hipStream_t stream) {
  constexpr int V = BF16 ? 8 : 4;
  if (a.codes_t == nullptr) return quantize_rows<BF16>(a, stream);
  const bool few = (a.padded_rows / 128) * ((a.cols + kWave * V - 1) / (kWave * V)) < kSmallQuantBlocks;
  if (a.codes != nullptr) return few ? quantize_cols<BF16, 2, true>(a, stream) : quantize_cols<BF16, V, true>(a, stream);
  return few ? quantize_cols<BF16, 2, false>(a, stream) : quantize_cols<BF16, V, false>(a, stream);
}

int quantize(Mx4QuantArgs a, bool bf16, hipStream_t stream) {
  a.padded_cols = mx4_padded(a.cols);
  a.padded_rows = mx4_padded(a.rows);
  return bf16 ? quantize_type<true>(a, stream) : quantize_type<false>(a, stream);
}

template <int T>
int product_tiles(Mx4ProductArgs a, int splits, hipStream_t stream) {
  const int64_t tm = (a.M + 64 * T - 1) / (64 * T), tn = (a.N + 64 * T - 1) / (64 * T);
  if (tm * tn > kMaxGrid) return SHAMPOO_EUNSUPPORTED;
  a.tiles_m = (uint32_t)tm;
  a.tiles_n = (uint32_t)tn;
  const bool beta = a.beta != 0.f;
  // one workgroup a compute unit, going from tile to tile, where it can
  const bool stream_tiles = mx4_streams(T, beta) && a.padded % 1024 == 0;
  const dim3 grid((uint32_t)(stream_tiles ? std::min<int64_t>(tm * tn, 256) : tm * tn), (uint32_t)splits), block(256);
  if (a.bf16 && beta) {
    hipLaunchKernelGGL((mx4_product_kernel<T, true, true>), grid, block, 0, stream, a);
  } else if (a.bf16) {
    hipLaunchKernelGGL((mx4_product_kernel<T, true, false>), grid, block, 0, stream, a);
  } else if (beta) {
    hipLaunchKernelGGL((mx4_product_kernel<T, false, true>), grid, block, 0, stream, a);
  } else {
    hipLaunchKernelGGL((mx4_product_kernel<T, false, false>), grid, block, 0, stream, a);
  }
  return check_launch();
}

constexpr int64_t kFewRows = 16;  // most rows of A that the weight-streaming form takes

// Whether that form also quantises A.
bool few_quantise(int64_t M, int64_t K) { return M <= kFewRows && M * mx4_padded(K) <= kMx4FewElems; }

template <int AM, int NT, int BATCH>
int few_rows_launch(const Mx4FewArgs& a, hipStream_t stream) {
  const int64_t blocks = (a.p.N + 16 * NT - 1) / (16 * NT);
  if (blocks > kMaxGrid) return SHAMPOO_EUNSUPPORTED;
  hipLaunchKernelGGL((mx4_few_rows_kernel<AM, NT, BATCH>), dim3((uint32_t)blocks), dim3(256), 0, stream, a);
  return check_launch();
}

// 32 rows of B a workgroup where that still leaves one for every compute unit
// and A has more than a row or two to read for each of them; batches of 4
// steps unless that would leave waves without any.
template <int AM>
int few_rows(const Mx4FewArgs& a, hipStream_t stream) {
  const bool wide = a.p.M > 2 && a.p.N >= 32 * 256;
  if (a.p.padded >= 4 * 4 * 128) return wide ? few_rows_launch<AM, 2, 4>(a, stream) : few_rows_launch<AM, 1, 4>(a, stream);
  if (a.p.padded >= 4 * 2 * 128) return wide ? few_rows_launch<AM, 2, 2>(a, stream) : few_rows_launch<AM, 1, 2>(a, stream);
  return wide ? few_rows_launch<AM, 2, 1>(a, stream) : few_rows_launch<AM, 1, 1>(a, stream);
}

int64_t tiles_of(int64_t M, int64_t N, int64_t edge) { return ((M + edge - 1) / edge) * ((N + edge - 1) / edge); }

// Splits of the columns for a product on 64 x 64 tiles, and the 1024-column
// blocks of each: as many as fill the 256 compute units, where the columns
// saved (1.3 us a block) pay for adding up the parts (2.5 us).
int split_columns(int64_t M, int64_t N, int64_t K, int* blocks_each) {
  const int64_t blocks = (K + 1023) / 1024, tiles = tiles_of(M, N, 64);
  *blocks_each = (int)blocks;
  if (M <= kFewRows || blocks < 4 || tiles > 128) return 1;
  const int64_t want = std::min<int64_t>(blocks, 256 / tiles);
  *blocks_each = (int)((blocks + want - 1) / want);
  return (int)((blocks + *blocks_each - 1) / *blocks_each);
}

// Tile edge: the largest of 256, 128 and 64 whose grid still occupies most of
// the 256 compute units.
int product(Mx4ProductArgs a, int64_t K, void* ws, hipStream_t stream) {
  if (a.M <= kFewRows) {
    Mx4FewArgs f = {};
    f.p = a;
    return few_rows<MX4_A_MX4>(f, stream);
  }
  const int splits = split_columns(a.M, a.N, K, &a.split_blocks);
  if (splits > 1) {
    Mx4SumArgs s;
    s.p = a;
    s.parts = static_cast<const float*>(ws);
    s.splits = splits;
    a.c = ws;
    a.ldc = a.N;
    a.alpha = 1.f;
    a.beta = 0.f;
    a.bf16 = 0;
    const int rc = product_tiles<1>(a, splits, stream);
    if (rc != SHAMPOO_OK) return rc;
    hipLaunchKernelGGL(mx4_sum_kernel, dim3((uint32_t)((a.M * a.N + 255) / 256)), dim3(256), 0, stream, s);
    return check_launch();
  }
  if (tiles_of(a.M, a.N, 256) >= 192) return product_tiles<4>(a, 1, stream);
  if (tiles_of(a.M, a.N, 128) >= 192) return product_tiles<2>(a, 1, stream);
  return product_tiles<1>(a, 1, stream);
}

}  // namespace

extern "C" {

int shampoo_mx4_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                         uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t, hipStream_t stream) {
  if (!valid_type(dtype)) return SHAMPOO_EUNSUPPORTED;
  const int rc = check_sides(rows, cols, 0);
  if (rc != SHAMPOO_OK) return rc;
  if (ld < cols) return SHAMPOO_EINVAL;
  if ((codes == nullptr) != (scales == nullptr) || (codes_t == nullptr) != (scales_t == nullptr))
    return SHAMPOO_EINVAL;
  if (rows == 0 || cols == 0) return SHAMPOO_OK;
  if (x == nullptr || (codes == nullptr && codes_t == nullptr)) return SHAMPOO_EINVAL;
  if ((codes != nullptr && !valid_mx4(codes, scales)) || (codes_t != nullptr && !valid_mx4(codes_t, scales_t)))
    return SHAMPOO_EINVAL;
  Mx4QuantArgs a = {};
  a.x = x;
  a.rows = rows;
  a.cols = cols;
  a.ld = ld;
  a.codes = codes;
  a.scales = scales;
  a.codes_t = codes_t;
  a.scales_t = scales_t;
  return quantize(a, dtype == SHAMPOO_T_BF16, stream);
}

int shampoo_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out,
                           int dtype, int64_t ld, hipStream_t stream) {
  if (!valid_type(dtype)) return SHAMPOO_EUNSUPPORTED;
  const int rc = check_sides(rows, cols, 0);
  if (rc != SHAMPOO_OK) return rc;
  if (ld < cols) return SHAMPOO_EINVAL;
  if (rows == 0 || cols == 0) return SHAMPOO_OK;
  if (!valid_mx4(codes, scales) || out == nullptr) return SHAMPOO_EINVAL;
  Mx4DequantArgs a;
  a.codes = codes;
  a.scales = scales;
  a.rows = rows;
  a.cols = cols;
  a.padded = mx4_padded(cols);
  a.ld = ld;
  a.out = out;
  int64_t col_blocks;
  row_shape(a.padded, dtype == SHAMPOO_T_BF16 ? 8 : 4, &a.lanes_log2, &col_blocks);
  const int64_t per_block = 4 * (256 >> a.lanes_log2), row_blocks = (rows + per_block - 1) / per_block;
  if (col_blocks * row_blocks > kMaxGrid) return SHAMPOO_EUNSUPPORTED;
  a.col_blocks = (uint32_t)col_blocks;
  const dim3 grid((uint32_t)(col_blocks * row_blocks)), block(256);
  if (dtype == SHAMPOO_T_BF16) {
    hipLaunchKernelGGL(mx4_dequantize_kernel<true>, grid, block, 0, stream, a);
  } else {
    hipLaunchKernelGGL(mx4_dequantize_kernel<false>, grid, block, 0, stream, a);
  }
  return check_launch();
}

size_t shampoo_mx4_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (check_sides(M, N, K) != SHAMPOO_OK || M == 0 || N == 0 || K > kMaxK) return 0;
  int each;
  const int splits = split_columns(M, N, K, &each);
  return splits > 1 ? align_up((size_t)splits * M * N * sizeof(float)) : 0;
}

int shampoo_mx4_product(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes,
                        const uint8_t* b_scales, int64_t M, int64_t N, int64_t K, float alpha, float beta, void* c,
                        int dtype, int64_t ldc, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!valid_type(dtype)) return SHAMPOO_EUNSUPPORTED;
  const int rc = check_sides(M, N, K);
  if (rc != SHAMPOO_OK) return rc;
  if (K > kMaxK) return SHAMPOO_EUNSUPPORTED;
  if (ldc < N || !std::isfinite(alpha) || !std::isfinite(beta)) return SHAMPOO_EINVAL;
  if (M == 0 || N == 0) return SHAMPOO_OK;
  if (c == nullptr || (K > 0 && (!valid_mx4(a_codes, a_scales) || !valid_mx4(b_codes, b_scales))))
    return SHAMPOO_EINVAL;
  const size_t need = shampoo_mx4_workspace_bytes(M, N, K);
  if (need > 0 && (ws == nullptr || ws_bytes < need)) return SHAMPOO_EWORKSPACE;
  if (need > 0 && !aligned16(ws)) return SHAMPOO_EINVAL;
  Mx4ProductArgs a = {};
  a.a = a_codes;
  a.as = a_scales;
  a.b = b_codes;
  a.bs = b_scales;
  a.M = M;
  a.N = N;
  a.padded = mx4_padded(K);
  a.c = c;
  a.ldc = ldc;
  a.alpha = alpha;
  a.beta = beta;
  a.bf16 = dtype == SHAMPOO_T_BF16;
  return product(a, K, ws, stream);
}

size_t shampoo_mx4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (check_sides(M, N, K) != SHAMPOO_OK) return 0;
  if (few_quantise(M, K)) return 0;
  const size_t elems = (size_t)M * (size_t)mx4_padded(K);
  return align_up(elems / 2) + align_up(elems / kMx4Group) + shampoo_mx4_workspace_bytes(M, N, K);
}

int shampoo_mx4_linear(const void* x, int64_t ldx, const uint8_t* w_codes, const uint8_t* w_scales, int64_t M,
                       int64_t N, int64_t K, void* y, int64_t ldy, int dtype, void* ws, size_t ws_bytes,
                       hipStream_t stream) {
  if (!valid_type(dtype)) return SHAMPOO_EUNSUPPORTED;
  int rc = check_sides(M, N, K);
  if (rc != SHAMPOO_OK) return rc;
  if (K > kMaxK) return SHAMPOO_EUNSUPPORTED;
  if (ldx < K || ldy < N) return SHAMPOO_EINVAL;
  if (M == 0 || N == 0) return SHAMPOO_OK;
  if (y == nullptr || (K > 0 && (x == nullptr || !valid_mx4(w_codes, w_scales)))) return SHAMPOO_EINVAL;
  const size_t need = shampoo_mx4_linear_workspace_bytes(M, N, K);
  if (need > 0 && (ws == nullptr || ws_bytes < need)) return SHAMPOO_EWORKSPACE;
  if (!aligned16(ws)) return SHAMPOO_EINVAL;
  // With few rows every workgroup reads X for itself while others write Y.
  if (K > 0 && may_overlap(x, K, ldx, y, N, ldy, M, dtype == SHAMPOO_T_BF16 ? 2 : 4)) return SHAMPOO_EINVAL;
  if (few_quantise(M, K)) {
    Mx4FewArgs f = {};
    f.p.b = w_codes;
    f.p.bs = w_scales;
    f.p.M = M;
    f.p.N = N;
    f.p.padded = mx4_padded(K);
    f.p.c = y;
    f.p.ldc = ldy;
    f.p.alpha = 1.f;
    f.p.bf16 = dtype == SHAMPOO_T_BF16;
    f.x = x;
    f.ldx = ldx;
    f.K = K;
    return dtype == SHAMPOO_T_BF16 ? few_rows<MX4_A_BF16>(f, stream) : few_rows<MX4_A_F32>(f, stream);
  }
  const size_t elems = (size_t)M * (size_t)mx4_padded(K);
  uint8_t* codes = static_cast<uint8_t*>(ws);
  uint8_t* scales = codes + align_up(elems / 2);
  uint8_t* rest = scales + align_up(elems / kMx4Group);
  if (K > 0) rc = shampoo_mx4_quantize(x, dtype, M, K, ldx, codes, scales, nullptr, nullptr, stream);
  if (rc != SHAMPOO_OK) return rc;
  return shampoo_mx4_product(codes, scales, w_codes, w_scales, M, N, K, 1.f, 0.f, y, dtype, ldy, rest,
                             ws_bytes - (size_t)(rest - codes), stream);
}

}  // extern "C"
