// Row-wise pieces shared by the kernels that hold whole rows in registers: a
// group of WAVES waves owns a row, and lane l of the group's wave w holds its
// chunks i of 8 consecutive bf16 values at columns 8 (64 w + l + 64 WAVES i).
// The 4 lanes of a quad then hold one 32-value block and 16 lanes one
// 128-column step, as in mx_tile.h.
#pragma once

#include "mx_device.h"
#include "mx_tile.h"

namespace mxk {

// Quantizes one chunk of row `row` at column `col` (a multiple of 8) and
// stores its codes and its block's or step's scales. All lanes must reach
// this function; `ok` (uniform over each quad) guards the stores.
__device__ __forceinline__ void chunk_rowq(uint4 v, bool ok, bool rceil, const TileOut& o, int64_t row, int col) {
  const uint32_t sb = scale_byte(quad_max(absmax8_bits(v)), rceil);
  const uint2 codes = e4m3_chunk(v, sb, !rceil);
  if (o.k128) {
    const uint32_t packed = or_row_quarters(sb << (8 * ((col >> 5) & 3)));
    if (ok) {
      *reinterpret_cast<uint2*>(o.q + row * o.ld + col) = codes;
      if ((col & 127) == 0) *reinterpret_cast<uint32_t*>(o.s + ((int64_t)(col >> 7) * o.srows + row) * 4) = packed;
    }
  } else if (ok) {
    *reinterpret_cast<uint2*>(o.q + row * o.ld + col) = codes;
    if ((col & 31) == 0) o.s[row * (o.ld / kBlock) + (col >> 5)] = (uint8_t)sb;
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

// Sum over the WAVES waves of this thread's group; every thread of the
// workgroup must call it. `buf`: one float per wave, free again at the next
// barrier.
template <int WAVES>
__device__ __forceinline__ float group_sum(float v, float* buf) {
  v = wave_sum(v);
  if constexpr (WAVES > 1) {
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) buf[w] = v;
    __syncthreads();
    const int g = w / WAVES * WAVES;
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) v += buf[g + i];
  }
  return v;
}

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ void load8f(const float* p, float (&f)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// y = bf16((s * rstd) * w) of 8 values; one expression for every kernel that
// forms y, so the row-wise and column-wise codes come from the same bits.
__device__ __forceinline__ uint4 norm_chunk(uint4 s, float rstd, const float (&w)[8]) {
  float f[8];
  unpack8(s, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = (f[i] * rstd) * w[i];
  return pack8(f);
}

}  // namespace mxk
