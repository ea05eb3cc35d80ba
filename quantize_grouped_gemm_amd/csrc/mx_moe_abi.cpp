// C ABI of the routed-experts operators and the FP8 products with blocks of
// 128 (declared and documented in include/mxmoe.h): argument validation on the
// host, device check, and launch on the caller's stream. Nothing here reads
// device memory or synchronizes.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/mxmoe.h"
#include "mx_abi_common.h"
#include "mx_moe.h"

using namespace mxabi;

namespace {

constexpr int64_t kMaxIndex = (1ll << 31) - (1 << 16);   // rows, slots and capacities are int32 on the device
constexpr int64_t kMaxTiles = 1ll << 22;                 // workgroups of 512 threads in a grid of 2^32 threads, halved
constexpr int64_t kMaxTokens = 1ll << 23;                // a workgroup of 256 threads each at most, 2^32 threads a grid
constexpr int64_t kMaxRows = 1ll << 25;                  // 126 rows of column-wise codes pass 32-bit offsets beyond
constexpr int64_t kMaxCols = 1ll << 20;
constexpr int64_t kMaxStride = 1ll << 26;

int64_t up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

mx_status check_logits(const char* fn, const void* x, mx_dtype dt, int64_t ld, int64_t rows, int32_t experts,
                       mx_score score, int32_t top, float scale) {
  MX_REQUIRE(dt == MX_BF16 || dt == MX_F32, MX_ERR_ARG, "%s: bad dtype", fn);
  MX_REQUIRE(score == MX_SOFTMAX || score == MX_SIGMOID, MX_ERR_ARG, "%s: bad score", fn);
  MX_REQUIRE(rows >= 0 && rows <= kMaxTokens, MX_ERR_SHAPE, "%s: rows (%lld) must be in [0, 2^23]", fn, (long long)rows);
  MX_REQUIRE(experts >= 1 && experts <= mxk::kMaxExperts, MX_ERR_SHAPE, "%s: experts (%d) must be in [1, %d]", fn, experts,
             mxk::kMaxExperts);
  MX_REQUIRE(top >= 1 && top <= std::min(experts, mxk::kMaxTopExperts), MX_ERR_SHAPE,
             "%s: top (%d) must be in [1, min(%d, experts)]", fn, top, mxk::kMaxTopExperts);
  MX_REQUIRE(ld >= experts && ld <= (1ll << 40), MX_ERR_ALIGN, "%s: ld (%lld) must be >= experts", fn, (long long)ld);
  MX_REQUIRE(std::isfinite(scale), MX_ERR_ARG, "%s: scale must be finite", fn);
  if (rows == 0) return MX_OK;
  MX_REQUIRE(x, MX_ERR_NULL, "%s: x is NULL", fn);
  MX_REQUIRE((reinterpret_cast<uintptr_t>(x) & (dt == MX_F32 ? 3u : 1u)) == 0, MX_ERR_ALIGN,
             "%s: x is not aligned to its element", fn);
  return MX_OK;
}

mx_status check_rows(const char* fn, const char* name, const void* p, int64_t ld, int64_t cols) {
  MX_REQUIRE(p, MX_ERR_NULL, "%s: %s is NULL", fn, name);
  MX_REQUIRE(al16(p) && ld >= cols && ld % 8 == 0, MX_ERR_ALIGN,
             "%s: %s must be 16-byte aligned with a row stride (%lld) >= the row length and a multiple of 8", fn, name,
             (long long)ld);
  MX_REQUIRE(ld <= kMaxStride, MX_ERR_SHAPE, "%s: %s row stride (%lld) above 2^26", fn, name, (long long)ld);
  return MX_OK;
}

mx_status check_pair(const char* fn, const char* name, const void* q, const void* s, bool optional, bool f32) {
  if (optional && !q && !s) return MX_OK;
  MX_REQUIRE(q && s, MX_ERR_NULL, "%s: %s codes/scales NULL", fn, name);
  MX_REQUIRE(al16(q), MX_ERR_ALIGN, "%s: %s codes must be 16-byte aligned", fn, name);
  MX_REQUIRE(!f32 || al4(s), MX_ERR_ALIGN, "%s: %s scales must be 4-byte aligned", fn, name);
  return MX_OK;
}

mx_status check_mode(const char* fn, mx_b128_mode mode) {
  MX_REQUIRE(mode == MX_B128_F32 || mode == MX_B128_RCEIL, MX_ERR_ARG, "%s: bad scale mode %d", fn, (int)mode);
  return MX_OK;
}

mx_status check_extent(const char* fn, int64_t rows, int64_t cols, int64_t step) {
  MX_REQUIRE(rows >= 0 && rows <= kMaxRows, MX_ERR_SHAPE, "%s: rows (%lld) must be in [0, 2^25]", fn, (long long)rows);
  MX_REQUIRE(cols > 0 && cols <= kMaxCols && cols % step == 0, MX_ERR_SHAPE,
             "%s: the row length (%lld) must be a positive multiple of %lld, at most 2^20", fn, (long long)cols,
             (long long)step);
  // the row-wise kernel takes 16 rows and 128 columns a workgroup
  MX_REQUIRE(up(rows, 128) / 128 * (up(cols, 128) / 128) <= kMaxTiles / 8, MX_ERR_SHAPE, "%s: too many tiles for one launch",
             fn);
  return MX_OK;
}

mx_status check_gather(const char* fn, int64_t x_rows, const int32_t* src, int32_t top, const float* weights) {
  MX_REQUIRE(x_rows >= 0 && x_rows < kMaxIndex, MX_ERR_SHAPE, "%s: x_rows (%lld) out of range", fn, (long long)x_rows);
  MX_REQUIRE(src, MX_ERR_NULL, "%s: src is NULL", fn);
  MX_REQUIRE(top >= 1, MX_ERR_SHAPE, "%s: top (%d) must be >= 1", fn, top);
  MX_REQUIRE(al4(src) && al4(weights), MX_ERR_ALIGN, "%s: src/weights must be 4-byte aligned", fn);
  return MX_OK;
}

// Buffer offsets inside a tile are 32 bits: 256 rows of `ld` codes, and one
// operand's scales.
mx_status check_operand(const char* fn, const char* name, const void* q, const void* s, int64_t ld, int64_t scales) {
  MX_CHECK(check_pair(fn, name, q, s, false, true));
  MX_REQUIRE(ld * 256 < (1ll << 31) && scales * 4 < (1ll << 31), MX_ERR_SHAPE, "%s: %s is too large (row %lld, %lld scales)",
             fn, name, (long long)ld, (long long)scales);
  return MX_OK;
}

mx_status check_groups(const char* fn, const int32_t* offs, int32_t E, int64_t cap) {
  MX_REQUIRE(E >= 1 && E <= mxk::kMaxExperts, MX_ERR_SHAPE, "%s: E (%d) must be in [1, %d]", fn, E, mxk::kMaxExperts);
  MX_REQUIRE(cap >= 0 && cap < kMaxIndex, MX_ERR_SHAPE, "%s: cap (%lld) out of range", fn, (long long)cap);
  MX_REQUIRE(offs, MX_ERR_NULL, "%s: offs is NULL", fn);
  MX_REQUIRE(al4(offs), MX_ERR_ALIGN, "%s: offs must be 4-byte aligned", fn);
  return MX_OK;
}

// Workgroups of a product's launch.
mx_status check_grid(const char* fn, int64_t workgroups) {
  MX_REQUIRE(workgroups < kMaxTiles, MX_ERR_SHAPE, "%s: too many tiles for one launch", fn);
  return MX_OK;
}

}  // namespace

extern "C" {

mx_status mx_route(const void* x, mx_dtype x_dtype, int64_t ld, int64_t rows, int32_t experts, const float* bias,
                   mx_score score, int32_t groups, int32_t top_groups, mx_group_score group_score, int32_t top, int renorm,
                   float scale, float* weights, int32_t* idx, void* stream) {
  const char* fn = "mx_route";
  MX_CHECK(check_logits(fn, x, x_dtype, ld, rows, experts, score, top, scale));
  MX_REQUIRE(groups >= 1 && groups <= mxk::kMaxExpertGroups && experts % groups == 0, MX_ERR_SHAPE,
             "%s: groups (%d) must be in [1, %d] and divide the experts", fn, groups, mxk::kMaxExpertGroups);
  MX_REQUIRE(top_groups >= 1 && top_groups <= groups, MX_ERR_SHAPE, "%s: top_groups (%d) must be in [1, groups]", fn,
             top_groups);
  MX_REQUIRE(group_score == MX_GROUP_MAX || group_score == MX_GROUP_TOP2, MX_ERR_ARG, "%s: bad group score", fn);
  if (rows == 0) return MX_OK;
  MX_REQUIRE(weights && idx, MX_ERR_NULL, "%s: weights/idx NULL", fn);
  MX_REQUIRE(al4(weights) && al4(idx) && al4(bias), MX_ERR_ALIGN, "%s: weights/idx/bias must be 4-byte aligned", fn);
  MX_DEVICE();
  mxk::RouteArgs a{};
  a.x = x; a.ld = ld; a.rows = rows; a.bias = bias;
  a.experts = experts; a.groups = groups; a.top_groups = top_groups; a.top = top;
  a.f32 = x_dtype == MX_F32; a.sigmoid = score == MX_SIGMOID; a.two = group_score == MX_GROUP_TOP2; a.renorm = renorm != 0;
  a.scale = scale; a.weights = weights; a.idx = idx;
  return launched(mxk::launch_route(a, as_stream(stream)), fn);
}

mx_status mx_route_bwd(const void* x, mx_dtype x_dtype, int64_t ld, int64_t rows, int32_t experts, mx_score score,
                       const int32_t* idx, int32_t top, int renorm, float scale, const float* dweights, void* dlogits,
                       void* stream) {
  const char* fn = "mx_route_bwd";
  MX_CHECK(check_logits(fn, x, x_dtype, ld, rows, experts, score, top, scale));
  if (rows == 0) return MX_OK;
  MX_REQUIRE(idx && dweights && dlogits, MX_ERR_NULL, "%s: idx/dweights/dlogits NULL", fn);
  MX_REQUIRE(al4(idx) && al4(dweights) && al4(dlogits), MX_ERR_ALIGN, "%s: idx/dweights/dlogits must be 4-byte aligned", fn);
  MX_DEVICE();
  mxk::RouteArgs a{};
  a.x = x; a.ld = ld; a.rows = rows; a.experts = experts; a.groups = a.top_groups = 1; a.top = top;
  a.f32 = x_dtype == MX_F32; a.sigmoid = score == MX_SIGMOID; a.renorm = renorm != 0;
  a.scale = scale; a.idx = const_cast<int32_t*>(idx); a.dweights = dweights; a.dx = dlogits;
  return launched(mxk::launch_route_bwd(a, as_stream(stream)), fn);
}

int64_t mx_dispatch_work(int64_t slots, int32_t experts) {
  return slots < 0 || experts < 0 ? 0 : mxk::dispatch_work(slots, experts);
}

mx_status mx_dispatch(const int32_t* idx, int64_t slots, int32_t experts, int32_t multiple, int64_t cap, int32_t* sizes,
                      int32_t* offs, int32_t* src, int32_t* pos, int32_t* work, void* stream) {
  const char* fn = "mx_dispatch";
  MX_REQUIRE(experts >= 1 && experts <= mxk::kMaxExperts, MX_ERR_SHAPE, "%s: experts (%d) must be in [1, %d]", fn, experts,
             mxk::kMaxExperts);
  MX_REQUIRE(multiple >= 1 && multiple <= 1024, MX_ERR_SHAPE, "%s: multiple (%d) must be in [1, 1024]", fn, multiple);
  MX_REQUIRE(slots >= 0 && slots < kMaxIndex && cap < kMaxIndex, MX_ERR_SHAPE, "%s: slots (%lld), cap (%lld) out of range",
             fn, (long long)slots, (long long)cap);
  const int64_t need = slots + std::min<int64_t>(experts, slots) * (multiple - 1);
  MX_REQUIRE(cap >= need, MX_ERR_SHAPE, "%s: cap (%lld) must be at least %lld", fn, (long long)cap, (long long)need);
  MX_REQUIRE(sizes && offs && (src || cap == 0) && ((idx && pos) || slots == 0), MX_ERR_NULL,
             "%s: idx/sizes/offs/src/pos NULL", fn);
  MX_REQUIRE(work || mxk::dispatch_work(slots, experts) == 0, MX_ERR_NULL, "%s: work is NULL", fn);
  MX_REQUIRE(al4(idx) && al4(sizes) && al4(offs) && al4(src) && al4(pos) && al4(work), MX_ERR_ALIGN,
             "%s: arrays must be 4-byte aligned", fn);
  MX_DEVICE();
  return launched(mxk::launch_dispatch(mxk::DispatchArgs{idx, slots, cap, experts, multiple, sizes, offs, src, pos, work},
                                       as_stream(stream)), fn);
}

mx_status mx_gather_quantize(const void* x, int64_t ld, int64_t x_rows, int64_t cols, const int32_t* src, int32_t top,
                             const float* weights, int64_t rows, mx_scale_mode mode, mx_scale_layout layout, uint8_t* q_row,
                             uint8_t* s_row, uint8_t* q_col, uint8_t* s_col, void* stream) {
  const char* fn = "mx_gather_quantize";
  MX_REQUIRE(mode == MX_RCEIL || mode == MX_FLOOR, MX_ERR_ARG, "%s: bad scale mode %d", fn, (int)mode);
  MX_REQUIRE(layout == MX_SCALES_PLAIN || layout == MX_SCALES_K128, MX_ERR_ARG, "%s: bad scale layout", fn);
  const int64_t step = layout == MX_SCALES_K128 ? 128 : 32;
  MX_CHECK(check_extent(fn, rows, cols, step));
  if (rows == 0) return MX_OK;
  MX_CHECK(check_gather(fn, x_rows, src, top, weights));
  if (x_rows) MX_CHECK(check_rows(fn, "x", x, ld, cols));
  MX_CHECK(check_pair(fn, "row-wise", q_row, s_row, false, layout == MX_SCALES_K128));
  MX_CHECK(check_pair(fn, "column-wise", q_col, s_col, true, layout == MX_SCALES_K128));
  MX_DEVICE();
  mxk::RowsQuantArgs a{};
  a.x = static_cast<const uint16_t*>(x); a.ld = ld; a.x_rows = x_rows; a.src = src; a.weights = weights; a.top = top;
  a.rows = rows; a.cols = cols; a.rows_pad = up(rows, step); a.rceil = mode == MX_RCEIL; a.k128 = layout == MX_SCALES_K128;
  a.q_row = q_row; a.s_row = s_row; a.q_col = q_col; a.s_col = s_col;
  return launched(mxk::launch_gather_mx(a, as_stream(stream)), fn);
}

mx_status mx_b128_gather_quantize(const void* x, int64_t ld, int64_t x_rows, int64_t cols, const int32_t* src, int32_t top,
                                  const float* weights, int64_t rows, mx_b128_mode mode, uint8_t* q_row, float* s_row,
                                  uint8_t* q_col, float* s_col, void* stream) {
  const char* fn = "mx_b128_gather_quantize";
  MX_CHECK(check_mode(fn, mode));
  MX_CHECK(check_extent(fn, rows, cols, 128));
  if (rows == 0) return MX_OK;
  MX_CHECK(check_gather(fn, x_rows, src, top, weights));
  if (x_rows) MX_CHECK(check_rows(fn, "x", x, ld, cols));
  MX_CHECK(check_pair(fn, "row-wise", q_row, s_row, false, true));
  MX_CHECK(check_pair(fn, "column-wise", q_col, s_col, true, true));
  MX_DEVICE();
  mxk::RowsQuantArgs a{};
  a.x = static_cast<const uint16_t*>(x); a.ld = ld; a.x_rows = x_rows; a.src = src; a.weights = weights; a.top = top;
  a.rows = rows; a.cols = cols; a.rows_pad = up(rows, 128); a.rceil = mode == MX_B128_RCEIL; a.k128 = true;
  a.q_row = q_row; a.s_row = s_row; a.q_col = q_col; a.s_col = s_col;
  return launched(mxk::launch_b128_quant(a, as_stream(stream)), fn);
}

mx_status mx_combine(const void* y, int64_t ld_y, int64_t y_rows, const int32_t* pos, const float* weights, const void* r,
                     int64_t ld_r, int64_t rows, int32_t top, int64_t cols, void* out, void* stream) {
  const char* fn = "mx_combine";
  MX_CHECK(check_extent(fn, rows, cols, 8));
  MX_REQUIRE(rows <= kMaxTokens, MX_ERR_SHAPE, "%s: rows (%lld) must be in [0, 2^23]", fn, (long long)rows);
  MX_REQUIRE(top >= 1 && top <= 1024, MX_ERR_SHAPE, "%s: top (%d) must be in [1, 1024]", fn, top);
  MX_REQUIRE(y_rows >= 0 && y_rows < kMaxIndex, MX_ERR_SHAPE, "%s: y_rows (%lld) out of range", fn, (long long)y_rows);
  if (rows == 0) return MX_OK;
  if (y_rows) MX_CHECK(check_rows(fn, "y", y, ld_y, cols));
  if (r) MX_CHECK(check_rows(fn, "r", r, ld_r, cols));
  MX_REQUIRE(pos && out, MX_ERR_NULL, "%s: pos/out NULL", fn);
  MX_REQUIRE(al4(pos) && al4(weights) && al16(out), MX_ERR_ALIGN,
             "%s: pos/weights must be 4-byte and out 16-byte aligned", fn);
  MX_DEVICE();
  mxk::CombineArgs a{};
  a.y = static_cast<const uint16_t*>(y); a.ld_y = ld_y; a.y_rows = y_rows; a.pos = pos; a.weights = weights;
  a.r = static_cast<const uint16_t*>(r); a.ld_r = ld_r; a.rows = rows; a.top = top; a.cols = cols;
  a.out = static_cast<uint16_t*>(out);
  return launched(mxk::launch_combine(a, as_stream(stream)), fn);
}

mx_status mx_combine_bwd(const void* dout, int64_t ld_dout, const void* y, int64_t ld_y, int64_t y_rows, const int32_t* pos,
                         int64_t rows, int32_t top, int64_t cols, float* dweights, void* stream) {
  const char* fn = "mx_combine_bwd";
  MX_CHECK(check_extent(fn, rows, cols, 8));
  MX_REQUIRE(rows <= kMaxTokens, MX_ERR_SHAPE, "%s: rows (%lld) must be in [0, 2^23]", fn, (long long)rows);
  MX_REQUIRE(top >= 1 && top <= 1024, MX_ERR_SHAPE, "%s: top (%d) must be in [1, 1024]", fn, top);
  MX_REQUIRE(y_rows >= 0 && y_rows < kMaxIndex, MX_ERR_SHAPE, "%s: y_rows (%lld) out of range", fn, (long long)y_rows);
  if (rows == 0) return MX_OK;
  MX_CHECK(check_rows(fn, "dout", dout, ld_dout, cols));
  if (y_rows) MX_CHECK(check_rows(fn, "y", y, ld_y, cols));
  MX_REQUIRE(pos && dweights, MX_ERR_NULL, "%s: pos/dweights NULL", fn);
  MX_REQUIRE(al4(pos) && al4(dweights), MX_ERR_ALIGN, "%s: pos/dweights must be 4-byte aligned", fn);
  MX_DEVICE();
  mxk::CombineArgs a{};
  a.y = static_cast<const uint16_t*>(y); a.ld_y = ld_y; a.y_rows = y_rows; a.pos = pos;
  a.dout = static_cast<const uint16_t*>(dout); a.ld_dout = ld_dout; a.rows = rows; a.top = top; a.cols = cols;
  a.dweights = dweights;
  return launched(mxk::launch_combine_bwd(a, as_stream(stream)), fn);
}

mx_status mx_b128_quantize(const void* x, int64_t ld, int64_t rows, int64_t cols, mx_b128_mode mode, uint8_t* q_row,
                           float* s_row, uint8_t* q_col, float* s_col, void* stream) {
  const char* fn = "mx_b128_quantize";
  MX_CHECK(check_mode(fn, mode));
  MX_CHECK(check_extent(fn, rows, cols, 128));
  if (rows == 0) return MX_OK;
  MX_CHECK(check_rows(fn, "x", x, ld, cols));
  MX_REQUIRE(q_row || q_col, MX_ERR_NULL, "%s: no output", fn);
  MX_CHECK(check_pair(fn, "row-wise", q_row, s_row, true, true));
  MX_CHECK(check_pair(fn, "column-wise", q_col, s_col, true, true));
  MX_DEVICE();
  mxk::RowsQuantArgs a{};
  a.x = static_cast<const uint16_t*>(x); a.ld = ld; a.x_rows = rows; a.top = 1;
  a.rows = rows; a.cols = cols; a.rows_pad = up(rows, 128); a.rceil = mode == MX_B128_RCEIL; a.k128 = true;
  a.q_row = q_row; a.s_row = s_row; a.q_col = q_col; a.s_col = s_col;
  return launched(mxk::launch_b128_quant(a, as_stream(stream)), fn);
}

mx_status mx_b128_quantize_weight(const void* w, int64_t batch, int64_t rows, int64_t cols, mx_b128_mode mode, uint8_t* q,
                                  float* s, uint8_t* q_t, float* s_t, void* stream) {
  const char* fn = "mx_b128_quantize_weight";
  MX_CHECK(check_mode(fn, mode));
  MX_REQUIRE(batch >= 0 && rows >= 0 && cols > 0 && rows <= (1ll << 24) && cols <= (1ll << 24) && rows % 16 == 0 &&
                 cols % 16 == 0, MX_ERR_SHAPE, "%s: rows (%lld) and cols (%lld) must be multiples of 16, at most 2^24", fn,
             (long long)rows, (long long)cols);
  const int64_t tiles = ((rows + 127) / 128) * ((cols + 127) / 128);
  MX_REQUIRE(batch <= kMaxTiles && tiles <= kMaxTiles && batch * tiles <= kMaxTiles, MX_ERR_SHAPE,
             "%s: too many tiles for one launch", fn);
  if (batch == 0 || rows == 0) return MX_OK;
  MX_REQUIRE(w, MX_ERR_NULL, "%s: w is NULL", fn);
  MX_REQUIRE(al16(w), MX_ERR_ALIGN, "%s: w must be 16-byte aligned", fn);
  MX_CHECK(check_pair(fn, "row-wise", q, s, false, true));
  MX_CHECK(check_pair(fn, "transposed", q_t, s_t, true, true));
  MX_DEVICE();
  return launched(mxk::launch_b128_weight(
                      mxk::B128WeightArgs{static_cast<const uint16_t*>(w), batch, rows, cols, mode == MX_B128_RCEIL, q, q_t, s,
                                          s_t}, as_stream(stream)), fn);
}

mx_status mx_b128_mm(const uint8_t* qa, const float* sa, const uint8_t* qb, const float* sb, int block_b, int64_t M,
                     int64_t N, int64_t K, mx_dtype out_dtype, void* out, int64_t ldo, void* stream) {
  const char* fn = "mx_b128_mm";
  MX_REQUIRE(out_dtype == MX_BF16 || out_dtype == MX_F32, MX_ERR_ARG, "%s: bad output dtype", fn);
  MX_REQUIRE(M >= 0 && M < kMaxIndex && N >= 0 && N < kMaxIndex && N % 8 == 0 && K >= 0 && K % 128 == 0, MX_ERR_SHAPE,
             "%s: M (%lld), N (%lld, a multiple of 8), K (%lld, a multiple of 128)", fn, (long long)M, (long long)N,
             (long long)K);
  if (M == 0 || N == 0) return MX_OK;
  mxk::B128GemmArgs a{};
  a.qa = qa; a.qb = qb; a.sa = sa; a.sb = sb; a.M = M; a.N = N; a.K = K; a.ldo = ldo;
  a.block_b = block_b != 0; a.out_f32 = out_dtype == MX_F32; a.out = out;
  MX_CHECK(check_grid(fn, mxk::b128_mm_grid(a)));
  if (K) {
    MX_CHECK(check_operand(fn, "A", qa, sa, K, K / 128 * M));
    MX_CHECK(check_operand(fn, "B", qb, sb, K, K / 128 * (block_b ? (N + 127) / 128 : N)));
  }
  MX_REQUIRE(out, MX_ERR_NULL, "%s: out is NULL", fn);
  MX_REQUIRE(al16(out) && ldo >= N && ldo % (out_dtype == MX_F32 ? 4 : 8) == 0, MX_ERR_ALIGN,
             "%s: output rows must be 16-byte aligned and ldo (%lld) >= N", fn, (long long)ldo);
  MX_DEVICE();
  return launched(mxk::launch_b128_mm(a, as_stream(stream)), fn);
}

mx_status mx_b128_grouped_mm(const uint8_t* qa, const float* sa, const uint8_t* qw, const float* sw, const int32_t* offs,
                             int32_t E, int64_t cap, int64_t N, int64_t K, void* out, int32_t* dev_err, void* stream) {
  const char* fn = "mx_b128_grouped_mm";
  MX_CHECK(check_groups(fn, offs, E, cap));
  MX_REQUIRE(N >= 0 && N % 8 == 0 && N < kMaxIndex && K > 0 && K % 128 == 0, MX_ERR_SHAPE,
             "%s: N (%lld) must be a multiple of 8, K (%lld) a positive multiple of 128", fn, (long long)N, (long long)K);
  if (cap == 0 || N == 0) return MX_OK;
  mxk::B128GemmArgs a{};
  a.qa = qa; a.qb = qw; a.sa = sa; a.sb = sw; a.M = cap; a.N = N; a.K = K; a.ldo = N;
  a.block_b = true; a.out = out; a.offs = offs; a.E = E; a.dev_err = dev_err;
  MX_CHECK(check_grid(fn, mxk::b128_grouped_grid(a)));
  MX_CHECK(check_operand(fn, "A", qa, sa, K, K / 128 * cap));
  MX_CHECK(check_operand(fn, "B", qw, sw, K, K / 128 * ((N + 127) / 128)));
  MX_REQUIRE(out, MX_ERR_NULL, "%s: out is NULL", fn);
  MX_REQUIRE(al16(out) && al4(dev_err), MX_ERR_ALIGN, "%s: out must be 16-byte and dev_err 4-byte aligned", fn);
  MX_DEVICE();
  return launched(mxk::launch_b128_grouped(a, as_stream(stream)), fn);
}

mx_status mx_b128_grouped_mm_wgrad(const uint8_t* qg, const float* sg, const uint8_t* qx, const float* sx,
                                   const int32_t* offs, int32_t E, int64_t cap, int64_t N, int64_t K, mx_dtype out_dtype,
                                   void* out, int32_t* dev_err, void* stream) {
  const char* fn = "mx_b128_grouped_mm_wgrad";
  MX_REQUIRE(out_dtype == MX_BF16 || out_dtype == MX_F32, MX_ERR_ARG, "%s: bad output dtype", fn);
  MX_CHECK(check_groups(fn, offs, E, cap));
  MX_REQUIRE(cap % 128 == 0, MX_ERR_SHAPE, "%s: cap (%lld) must be a multiple of 128", fn, (long long)cap);
  MX_REQUIRE(N >= 0 && N < kMaxIndex && K >= 0 && K % 8 == 0 && K < kMaxIndex, MX_ERR_SHAPE,
             "%s: N (%lld), K (%lld, a multiple of 8)", fn, (long long)N, (long long)K);
  if (N == 0 || K == 0) return MX_OK;
  mxk::B128GemmArgs a{};
  a.qa = qg; a.qb = qx; a.sa = sg; a.sb = sx; a.M = N; a.N = K; a.K = cap; a.ldo = K;
  a.out_f32 = out_dtype == MX_F32; a.out = out; a.offs = offs; a.E = E; a.dev_err = dev_err;
  MX_CHECK(check_grid(fn, mxk::b128_wgrad_grid(a)));
  if (cap) {
    MX_CHECK(check_operand(fn, "G", qg, sg, cap, cap / 128 * N));
    MX_CHECK(check_operand(fn, "X", qx, sx, cap, cap / 128 * K));
  }
  MX_REQUIRE(out, MX_ERR_NULL, "%s: out is NULL", fn);
  MX_REQUIRE(al16(out) && al4(dev_err), MX_ERR_ALIGN, "%s: out must be 16-byte and dev_err 4-byte aligned", fn);
  MX_DEVICE();
  return launched(mxk::launch_b128_wgrad(a, as_stream(stream)), fn);
}

}  // extern "C"
