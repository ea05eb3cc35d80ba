// Argument blocks and launchers of the routed-experts operators and the FP8
// products with blocks of 128 (internal; the public interface is
// include/mxmoe.h). Shapes are validated by the caller (mx_moe_abi.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxk {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopExperts = 16;    // experts a token goes to
constexpr int kMaxExpertGroups = 16;

struct RouteArgs {
  const void* x;
  int64_t ld, rows;
  const float* bias;
  int32_t experts, groups, top_groups, top;
  bool f32, sigmoid, two, renorm;     // two: a group counts by its two largest values
  float scale;
  float* weights;
  int32_t* idx;          // forward: output; backward: input
  const float* dweights; // backward
  void* dx;
};
hipError_t launch_route(const RouteArgs& a, hipStream_t s);
hipError_t launch_route_bwd(const RouteArgs& a, hipStream_t s);

struct DispatchArgs {
  const int32_t* idx;
  int64_t slots, cap;
  int32_t experts, multiple;
  int32_t *sizes, *offs, *src, *pos, *work;
};
int64_t dispatch_work(int64_t slots, int64_t experts);
hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t s);

struct CombineArgs {
  const uint16_t *y, *r, *dout;
  const int32_t* pos;
  const float* weights;
  int64_t ld_y, ld_r, ld_dout, rows, cols, y_rows;
  int32_t top;
  uint16_t* out;
  float* dweights;
};
hipError_t launch_combine(const CombineArgs& a, hipStream_t s);
hipError_t launch_combine_bwd(const CombineArgs& a, hipStream_t s);

// Rows of a bf16 matrix, taken as they are (src NULL) or through a row map,
// scaled by a weight each or not, and quantized.
struct RowsQuantArgs {
  const uint16_t* x;
  int64_t ld, x_rows;
  const int32_t* src;      // [rows] slot of each output row, or NULL
  const float* weights;    // by slot, or NULL
  int32_t top;             // slots per row of x
  int64_t rows, cols, rows_pad;
  bool rceil, k128;
  uint8_t *q_row, *q_col;
  void *s_row, *s_col;     // E8M0 bytes (MXFP8) or float32 (blocks of 128)
};
hipError_t launch_gather_mx(const RowsQuantArgs& a, hipStream_t s);
hipError_t launch_b128_quant(const RowsQuantArgs& a, hipStream_t s);

struct B128WeightArgs {
  const uint16_t* w;
  int64_t batch, rows, cols;
  bool rceil;
  uint8_t *q, *q_t;
  float *s, *s_t;
};
hipError_t launch_b128_weight(const B128WeightArgs& a, hipStream_t s);

struct B128GemmArgs {
  const uint8_t *qa, *qb;     // [M, K]; [N, K] or per expert [N, K]; weight gradient: [M, K total], [N, K total]
  const float *sa, *sb;
  int64_t M, N, K;            // grouped: M = capacity; weight gradient: K = capacity
  int64_t ldo;
  bool block_b;               // sb one scale for 128 x 128 (else 1 x 128)
  bool out_f32;
  void* out;
  const int32_t* offs;        // grouped: [E]
  int32_t E;
  int32_t* dev_err;
};
// Workgroups (of at most 512 threads) that the launches below take.
int64_t b128_mm_grid(const B128GemmArgs& a);
int64_t b128_grouped_grid(const B128GemmArgs& a);
int64_t b128_wgrad_grid(const B128GemmArgs& a);
hipError_t launch_b128_mm(const B128GemmArgs& a, hipStream_t s);
hipError_t launch_b128_grouped(const B128GemmArgs& a, hipStream_t s);
hipError_t launch_b128_wgrad(const B128GemmArgs& a, hipStream_t s);

}  // namespace mxk
