// C ABI of the layer-boundary operators (declared and documented in
// include/mxlm.h): argument validation on the host, device check, and launch
// on the caller's stream. Nothing here reads device memory or synchronizes.

#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/mxlm.h"
#include "mx_abi_common.h"
#include "mx_lm.h"

using namespace mxabi;

namespace {

constexpr int64_t kMaxRows = (int64_t)65535 * 128;   // one grid row per 128 tokens

// The tile kernels address the 32 rows between two of a thread's chunks with
// 32-bit byte offsets: 31 strides of 2^27 bytes stay below 2^32, so 2^26
// elements of bf16 and 2^25 of float32.
constexpr int64_t kMaxStride = 1ll << 26;

// One workgroup of 512 threads per 128 x 128 tile; a grid holds 2^32 threads.
constexpr int64_t kMaxTiles = 1ll << 21;

bool tiles_fit(int64_t rows, int64_t cols) { return (rows + 127) / 128 * ((cols + 127) / 128) <= kMaxTiles; }

bool al8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
int64_t step_of(mx_scale_layout layout) { return layout == MX_SCALES_K128 ? 128 : 32; }
int64_t round_up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

mx_status check_format(const char* fn, mx_scale_mode mode, mx_scale_layout layout) {
  MX_REQUIRE(mode == MX_RCEIL || mode == MX_FLOOR, MX_ERR_ARG, "%s: bad scale mode %d", fn, (int)mode);
  MX_REQUIRE(layout == MX_SCALES_PLAIN || layout == MX_SCALES_K128, MX_ERR_ARG, "%s: bad scale layout", fn);
  return MX_OK;
}

mx_status check_extent(const char* fn, int64_t rows, int64_t cols, mx_scale_layout layout, int64_t max_cols) {
  const int64_t m = step_of(layout);
  MX_REQUIRE(rows >= 0 && rows <= kMaxRows, MX_ERR_SHAPE, "%s: rows (%lld) must be in [0, %lld]", fn,
             (long long)rows, (long long)kMaxRows);
  MX_REQUIRE(cols > 0 && cols <= max_cols && cols % m == 0, MX_ERR_SHAPE,
             "%s: the row length (%lld) must be a positive multiple of %lld, at most %lld", fn, (long long)cols,
             (long long)m, (long long)max_cols);
  MX_REQUIRE(tiles_fit(rows, cols), MX_ERR_SHAPE, "%s: too many tiles for one launch", fn);
  return MX_OK;
}

// A codes + scales pair: both or (if optional) neither.
mx_status check_pair(const char* fn, const char* name, const uint8_t* q, const uint8_t* s, mx_scale_layout layout,
                     bool optional) {
  if (optional && !q && !s) return MX_OK;
  MX_REQUIRE(q && s, MX_ERR_NULL, "%s: %s codes/scales NULL", fn, name);
  MX_REQUIRE(al16(q), MX_ERR_ALIGN, "%s: %s codes must be 16-byte aligned", fn, name);
  MX_REQUIRE(layout == MX_SCALES_PLAIN || al4(s), MX_ERR_ALIGN, "%s: %s scales must be 4-byte aligned", fn, name);
  return MX_OK;
}

mx_status check_rows(const char* fn, const char* name, const void* p, int64_t ld, int64_t cols) {
  MX_REQUIRE(p, MX_ERR_NULL, "%s: %s is NULL", fn, name);
  MX_REQUIRE(al16(p) && ld >= cols && ld % 8 == 0, MX_ERR_ALIGN,
             "%s: %s must be 16-byte aligned with a row stride (%lld) >= the row length and a multiple of 8", fn,
             name, (long long)ld);
  MX_REQUIRE(ld <= kMaxStride, MX_ERR_SHAPE, "%s: %s row stride (%lld) above 2^26", fn, name, (long long)ld);
  return MX_OK;
}

mx_status check_logits(const char* fn, const void* x, mx_dtype dt, int64_t ld, int64_t rows, int64_t vocab,
                       float scale) {
  MX_REQUIRE(dt == MX_BF16 || dt == MX_F32, MX_ERR_ARG, "%s: bad dtype", fn);
  MX_REQUIRE(rows >= 0 && rows <= kMaxRows, MX_ERR_SHAPE, "%s: rows (%lld) must be in [0, %lld]", fn,
             (long long)rows, (long long)kMaxRows);
  MX_REQUIRE(vocab >= 1 && vocab < (1ll << 31) - (1 << 16), MX_ERR_SHAPE,
             "%s: vocab (%lld) must be in [1, 2^31 - 2^16)", fn, (long long)vocab);
  MX_REQUIRE(ld >= vocab, MX_ERR_ALIGN, "%s: ld (%lld) must be >= vocab", fn, (long long)ld);
  MX_REQUIRE(scale >= 1e-6f && scale <= 1e6f, MX_ERR_ARG, "%s: scale must be in [1e-6, 1e6]", fn);
  if (rows == 0) return MX_OK;
  MX_REQUIRE(x, MX_ERR_NULL, "%s: x is NULL", fn);
  MX_REQUIRE((reinterpret_cast<uintptr_t>(x) & (dt == MX_F32 ? 3u : 1u)) == 0, MX_ERR_ALIGN,
             "%s: x is not aligned to its element", fn);
  return MX_OK;
}

}  // namespace

extern "C" {

mx_status mx_add_rmsnorm_quant(const void* x, int64_t ld_x, const void* r, int64_t ld_r, const float* w,
                               int64_t rows, int64_t cols, float eps, mx_scale_mode mode, mx_scale_layout layout,
                               void* sum, float* rstd, uint8_t* q_row, uint8_t* s_row, uint8_t* q_col,
                               uint8_t* s_col, uint8_t* q_ck, uint8_t* s_ck, void* stream) {
  const char* fn = "mx_add_rmsnorm_quant";
  MX_CHECK(check_format(fn, mode, layout));
  MX_CHECK(check_extent(fn, rows, cols, layout, mxk::kNormMaxCols));
  MX_REQUIRE(eps >= 0 && std::isfinite(eps), MX_ERR_ARG, "%s: eps must be finite and >= 0", fn);
  if (rows == 0) return MX_OK;
  MX_CHECK(check_rows(fn, "x", x, ld_x, cols));
  MX_REQUIRE((r != nullptr) == (sum != nullptr), MX_ERR_NULL, "%s: r and sum go together", fn);
  if (r) {
    MX_CHECK(check_rows(fn, "r", r, ld_r, cols));
    MX_REQUIRE(al16(sum), MX_ERR_ALIGN, "%s: sum must be 16-byte aligned", fn);
  }
  MX_REQUIRE(w && rstd, MX_ERR_NULL, "%s: w/rstd NULL", fn);
  MX_REQUIRE(al16(w) && al4(rstd), MX_ERR_ALIGN, "%s: w must be 16-byte and rstd 4-byte aligned", fn);
  MX_CHECK(check_pair(fn, "row-wise", q_row, s_row, layout, false));
  MX_CHECK(check_pair(fn, "column-wise", q_col, s_col, layout, true));
  MX_CHECK(check_pair(fn, "checkpoint", q_ck, s_ck, layout, true));
  MX_DEVICE();
  mxk::NormFwdArgs a{};
  a.x = static_cast<const uint16_t*>(x); a.r = static_cast<const uint16_t*>(r);
  a.w = w; a.ld_x = ld_x; a.ld_r = ld_r;
  a.rows = rows; a.cols = cols; a.rows_pad = round_up(rows, step_of(layout));
  a.eps = eps; a.rceil = mode == MX_RCEIL; a.k128 = layout == MX_SCALES_K128;
  a.sum = static_cast<uint16_t*>(sum); a.rstd = rstd;
  a.q_row = q_row; a.s_row = s_row; a.q_col = q_col; a.s_col = s_col; a.q_ck = q_ck; a.s_ck = s_ck;
  return launched(mxk::launch_norm_fwd(a, as_stream(stream)), fn);
}

int64_t mx_add_rmsnorm_bwd_work(int64_t rows, int64_t cols) {
  return rows <= 0 || cols <= 0 ? 0 : mxk::norm_bwd_work(rows, cols);
}

mx_status mx_add_rmsnorm_bwd(const void* dy, int64_t ld_dy, const float* w, const float* rstd, const void* x,
                             int64_t ld_x, const uint8_t* q_ck, const uint8_t* s_ck, const void* dsum,
                             int64_t ld_dsum, int64_t rows, int64_t cols, mx_scale_mode mode,
                             mx_scale_layout layout, void* dx, float* dw, uint8_t* q_row, uint8_t* s_row,
                             uint8_t* q_col, uint8_t* s_col, float* work, void* stream) {
  const char* fn = "mx_add_rmsnorm_bwd";
  MX_CHECK(check_format(fn, mode, layout));
  MX_CHECK(check_extent(fn, rows, cols, layout, mxk::kNormMaxCols));
  MX_REQUIRE(dw, MX_ERR_NULL, "%s: dw is NULL", fn);
  MX_REQUIRE(al16(dw), MX_ERR_ALIGN, "%s: dw must be 16-byte aligned", fn);
  if (rows > 0) {
    MX_CHECK(check_rows(fn, "dy", dy, ld_dy, cols));
    MX_REQUIRE((x != nullptr) != (q_ck != nullptr), MX_ERR_NULL, "%s: give exactly one of x and the checkpoint", fn);
    if (x) MX_CHECK(check_rows(fn, "x", x, ld_x, cols));
    else MX_CHECK(check_pair(fn, "checkpoint", q_ck, s_ck, layout, false));
    if (dsum) MX_CHECK(check_rows(fn, "dsum", dsum, ld_dsum, cols));
    MX_REQUIRE(w && rstd && dx && work, MX_ERR_NULL, "%s: w/rstd/dx/work NULL", fn);
    MX_REQUIRE(al16(w) && al4(rstd) && al16(dx) && al16(work), MX_ERR_ALIGN,
               "%s: w/dx/work must be 16-byte and rstd 4-byte aligned", fn);
    MX_CHECK(check_pair(fn, "row-wise", q_row, s_row, layout, true));
    MX_CHECK(check_pair(fn, "column-wise", q_col, s_col, layout, true));
  }
  MX_DEVICE();
  mxk::NormBwdArgs a{};
  a.dy = static_cast<const uint16_t*>(dy); a.x = static_cast<const uint16_t*>(x);
  a.dsum = static_cast<const uint16_t*>(dsum); a.w = w; a.rstd = rstd; a.q_ck = q_ck; a.s_ck = s_ck;
  a.ld_dy = ld_dy; a.ld_x = ld_x; a.ld_dsum = ld_dsum;
  a.rows = rows; a.cols = cols; a.rows_pad = round_up(rows, step_of(layout));
  a.rceil = mode == MX_RCEIL; a.k128 = layout == MX_SCALES_K128;
  a.dx = static_cast<uint16_t*>(dx); a.dw = dw;
  a.q_row = q_row; a.s_row = s_row; a.q_col = q_col; a.s_col = s_col; a.work = work;
  return launched(mxk::launch_norm_bwd(a, as_stream(stream)), fn);
}

static mx_status check_swiglu_ck(const char* fn, int64_t rows, int64_t hidden, mx_scale_mode mode,
                                 mx_scale_layout layout, const uint8_t* q_row, const uint8_t* s_row,
                                 const uint8_t* q_col, const uint8_t* s_col, const uint8_t* q_ck,
                                 const uint8_t* s_ck) {
  MX_CHECK(check_format(fn, mode, layout));
  MX_CHECK(check_extent(fn, rows, hidden, layout, kMaxStride / 2));
  if (rows == 0) return MX_OK;
  MX_CHECK(check_pair(fn, "row-wise", q_row, s_row, layout, false));
  MX_CHECK(check_pair(fn, "column-wise", q_col, s_col, layout, false));
  return check_pair(fn, "checkpoint", q_ck, s_ck, layout, false);
}

mx_status mx_swiglu_ckpt_fwd(const void* a, const void* b, int64_t ld_ab, int64_t rows, int64_t hidden,
                             mx_scale_mode mode, mx_scale_layout layout, uint8_t* q_row, uint8_t* s_row,
                             uint8_t* q_col, uint8_t* s_col, uint8_t* q_ck, uint8_t* s_ck, void* stream) {
  const char* fn = "mx_swiglu_ckpt_fwd";
  MX_CHECK(check_swiglu_ck(fn, rows, hidden, mode, layout, q_row, s_row, q_col, s_col, q_ck, s_ck));
  if (rows == 0) return MX_OK;
  MX_CHECK(check_rows(fn, "a", a, ld_ab, hidden));
  MX_CHECK(check_rows(fn, "b", b, ld_ab, hidden));
  MX_DEVICE();
  mxk::SwigluCkArgs k{};
  k.a = static_cast<const uint16_t*>(a); k.b = static_cast<const uint16_t*>(b); k.ld_ab = ld_ab;
  k.rows = rows; k.hidden = hidden; k.rows_pad = round_up(rows, step_of(layout));
  k.rceil = mode == MX_RCEIL; k.k128 = layout == MX_SCALES_K128;
  k.q_row = q_row; k.s_row = s_row; k.q_col = q_col; k.s_col = s_col; k.q_ck = q_ck; k.s_ck = s_ck;
  return launched(mxk::launch_swiglu_ck_fwd(k, as_stream(stream)), fn);
}

mx_status mx_swiglu_ckpt_bwd(const void* dh, int64_t ld_dh, const uint8_t* q_ck, const uint8_t* s_ck, int64_t rows,
                             int64_t hidden, mx_scale_mode mode, mx_scale_layout layout, uint8_t* q_row,
                             uint8_t* s_row, uint8_t* q_col, uint8_t* s_col, void* stream) {
  const char* fn = "mx_swiglu_ckpt_bwd";
  MX_CHECK(check_swiglu_ck(fn, rows, hidden, mode, layout, q_row, s_row, q_col, s_col, q_ck, s_ck));
  if (rows == 0) return MX_OK;
  MX_CHECK(check_rows(fn, "dh", dh, ld_dh, hidden));
  MX_DEVICE();
  mxk::SwigluCkArgs k{};
  k.dh = static_cast<const uint16_t*>(dh); k.ld_dh = ld_dh;
  k.rows = rows; k.hidden = hidden; k.rows_pad = round_up(rows, step_of(layout));
  k.rceil = mode == MX_RCEIL; k.k128 = layout == MX_SCALES_K128;
  k.q_row = q_row; k.s_row = s_row; k.q_col = q_col; k.s_col = s_col;
  k.q_ck = const_cast<uint8_t*>(q_ck); k.s_ck = const_cast<uint8_t*>(s_ck);
  return launched(mxk::launch_swiglu_ck_bwd(k, as_stream(stream)), fn);
}

int64_t mx_token_logprobs_work(int64_t rows, int64_t vocab, int32_t top) {
  return rows <= 0 || vocab <= 0 || top < 0 ? 0 : mxk::logprob_work(rows, vocab, top);
}

mx_status mx_token_logprobs(const void* x, mx_dtype x_dtype, int64_t ld, int64_t rows, int64_t vocab,
                            const int64_t* targets, int64_t ignore_index, float scale, int32_t top, float* logp,
                            float* entropy, float* stats, float* top_logp, int32_t* top_idx, void* work,
                            int32_t* dev_err, void* stream) {
  const char* fn = "mx_token_logprobs";
  MX_CHECK(check_logits(fn, x, x_dtype, ld, rows, vocab, scale));
  MX_REQUIRE(top >= 0 && top <= mxk::kMaxTop && top <= vocab, MX_ERR_SHAPE, "%s: top (%d) must be in [0, min(%d, vocab)]",
             fn, top, mxk::kMaxTop);
  if (rows == 0) return MX_OK;
  MX_REQUIRE(targets && logp && entropy && stats, MX_ERR_NULL, "%s: targets/logp/entropy/stats NULL", fn);
  MX_REQUIRE(al8(targets) && al4(logp) && al4(entropy) && al8(stats), MX_ERR_ALIGN,
             "%s: targets/stats must be 8-byte and logp/entropy 4-byte aligned", fn);
  if (top) {
    MX_REQUIRE(top_logp && top_idx, MX_ERR_NULL, "%s: top_logp/top_idx NULL", fn);
    MX_REQUIRE(al4(top_logp) && al4(top_idx), MX_ERR_ALIGN, "%s: top_logp/top_idx must be 4-byte aligned", fn);
  }
  MX_REQUIRE(al4(dev_err), MX_ERR_ALIGN, "%s: dev_err must be 4-byte aligned", fn);
  if (mxk::logprob_work(rows, vocab, top) > 0) {
    MX_REQUIRE(work, MX_ERR_NULL, "%s: work is NULL", fn);
    MX_REQUIRE(al16(work), MX_ERR_ALIGN, "%s: work must be 16-byte aligned", fn);
  }
  MX_DEVICE();
  mxk::LogprobArgs a{};
  a.x = x; a.f32 = x_dtype == MX_F32; a.ld = ld; a.rows = rows; a.vocab = vocab;
  a.targets = targets; a.ignore_index = ignore_index; a.scale = scale; a.dev_err = dev_err;
  a.top = top; a.logp = logp; a.entropy = entropy; a.stats_out = stats; a.top_logp = top_logp; a.top_idx = top_idx;
  a.work = work;
  return launched(mxk::launch_logprob_fwd(a, as_stream(stream)), fn);
}

mx_status mx_token_logprobs_bwd(const void* x, mx_dtype x_dtype, int64_t ld, int64_t rows, int64_t vocab,
                                const int64_t* targets, int64_t ignore_index, const float* stats,
                                const float* entropy, const float* dlogp, const float* dent, float scale,
                                mx_scale_mode mode, mx_scale_layout layout, uint8_t* q_row, uint8_t* s_row,
                                uint8_t* q_col, uint8_t* s_col, int32_t* dev_err, void* stream) {
  const char* fn = "mx_token_logprobs_bwd";
  MX_CHECK(check_format(fn, mode, layout));
  MX_CHECK(check_logits(fn, x, x_dtype, ld, rows, vocab, scale));
  const int64_t max_ld = x_dtype == MX_F32 ? kMaxStride / 2 : kMaxStride;
  MX_REQUIRE(vocab <= max_ld - 128 && ld <= max_ld, MX_ERR_SHAPE, "%s: vocab (%lld) or ld (%lld) above %lld", fn,
             (long long)vocab, (long long)ld, (long long)max_ld);
  MX_REQUIRE(tiles_fit(rows, vocab), MX_ERR_SHAPE, "%s: too many tiles for one launch", fn);
  if (rows == 0) return MX_OK;
  MX_REQUIRE(targets && stats && entropy, MX_ERR_NULL, "%s: targets/stats/entropy NULL", fn);
  MX_REQUIRE(al8(targets) && al8(stats) && al4(entropy) && al4(dlogp) && al4(dent) && al4(dev_err), MX_ERR_ALIGN,
             "%s: targets/stats must be 8-byte and entropy/dlogp/dent/dev_err 4-byte aligned", fn);
  MX_CHECK(check_pair(fn, "row-wise", q_row, s_row, layout, false));
  MX_CHECK(check_pair(fn, "column-wise", q_col, s_col, layout, false));
  MX_DEVICE();
  mxk::LogprobArgs a{};
  a.x = x; a.f32 = x_dtype == MX_F32; a.ld = ld; a.rows = rows; a.vocab = vocab;
  a.targets = targets; a.ignore_index = ignore_index; a.scale = scale; a.dev_err = dev_err;
  a.stats = stats; a.ent_in = entropy; a.dlogp = dlogp; a.dent = dent;
  a.vocab_pad = round_up(vocab, step_of(layout)); a.rows_pad = round_up(rows, step_of(layout));
  a.rceil = mode == MX_RCEIL; a.k128 = layout == MX_SCALES_K128;
  a.q_row = q_row; a.s_row = s_row; a.q_col = q_col; a.s_col = s_col;
  return launched(mxk::launch_logprob_bwd(a, as_stream(stream)), fn);
}

}  // extern "C"
