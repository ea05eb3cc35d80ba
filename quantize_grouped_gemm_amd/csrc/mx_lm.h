// Argument blocks and launchers of the layer-boundary operators (internal;
// the public interface is include/mxlm.h). Shapes are validated by the caller
// (mx_lm_abi.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxk {

struct NormFwdArgs {
  const uint16_t *x, *r;
  const float* w;
  int64_t ld_x, ld_r, rows, cols, rows_pad;
  float eps;
  bool rceil, k128;
  uint16_t* sum;
  float* rstd;
  uint8_t *q_row, *s_row, *q_col, *s_col, *q_ck, *s_ck;
};

struct NormBwdArgs {
  const uint16_t *dy, *x, *dsum;
  const float *w, *rstd;
  const uint8_t *q_ck, *s_ck;
  int64_t ld_dy, ld_x, ld_dsum, rows, cols, rows_pad;
  bool rceil, k128;
  uint16_t* dx;
  float* dw;
  uint8_t *q_row, *s_row, *q_col, *s_col;
  float* work;
};

struct SwigluCkArgs {
  const uint16_t *a, *b;     // forward
  int64_t ld_ab;
  const uint16_t* dh;        // backward
  int64_t ld_dh;
  int64_t rows, hidden, rows_pad;
  bool rceil, k128;
  uint8_t *q_row, *s_row, *q_col, *s_col, *q_ck, *s_ck;
  bool bands;                // order of the tiles, set by the launcher
};

struct LogprobArgs {
  const void* x;
  bool f32;
  int64_t ld, rows, vocab;
  const int64_t* targets;
  int64_t ignore_index;
  float scale;
  int32_t* dev_err;
  // forward
  int32_t top;
  float *logp, *entropy, *stats_out, *top_logp;
  int32_t* top_idx;
  void* work;
  // backward
  const float *stats, *ent_in, *dlogp, *dent;
  int64_t vocab_pad, rows_pad;
  bool rceil, k128;
  uint8_t *q_row, *s_row, *q_col, *s_col;
  bool bands;                // order of the tiles, set by the launcher
};

// A launch costs the host 2.8 us with up to 112 bytes of kernel arguments and 3.4
// with more, of the 4 to 10 us that a small call takes: kernels get their blocks
// packed (sizes in 32 bits, what follows from others left out) and widen them,
// and none reads the grid's or the workgroup's size, which would add 256 bytes.
constexpr size_t kArgBytes = 112;

constexpr int64_t kNormMaxCols = 16384;
constexpr int32_t kMaxTop = 64;

hipError_t launch_norm_fwd(const NormFwdArgs& a, hipStream_t s);
int64_t norm_bwd_work(int64_t rows, int64_t cols);   // float32 elements
hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t s);
hipError_t launch_swiglu_ck_fwd(const SwigluCkArgs& a, hipStream_t s);
hipError_t launch_swiglu_ck_bwd(const SwigluCkArgs& a, hipStream_t s);
int64_t logprob_work(int64_t rows, int64_t vocab, int32_t top);   // bytes
hipError_t launch_logprob_fwd(const LogprobArgs& a, hipStream_t s);
hipError_t launch_logprob_bwd(const LogprobArgs& a, hipStream_t s);

}  // namespace mxk
