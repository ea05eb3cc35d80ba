// Row-wise pieces of the kernels that hold whole rows in registers: thread t
// of the threads that own a row holds its chunks i of 8 consecutive bf16
// values at columns 8 (t + threads * i). The 4 lanes of a quad then hold one
// 32-value block and 16 lanes one 128-column step, as in mx_tile.h.
#pragma once

#include "mx_device.h"
#include "mx_lm_device.h"
#include "mx_tile.h"

namespace mxk {

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

// y = bf16(s rstd w) of 8 values, in float32 with one rounding before bf16's:
// with rstd = h + l, h its upper 8 significant bits, s h and s l are exact
// (s has 8 bits), so fma(s h, w, (s l) w) is off by half an ulp. Two rounded
// products are off by up to one and a half, which moves about three times as
// many values across a bf16 rounding border. Every kernel that forms y uses
// this function, so the row-wise and column-wise codes come from the same
// bits.
__device__ __forceinline__ uint4 norm_chunk(uint4 s, float rstd, const float (&w)[8]) {
  const float h = __uint_as_float(__float_as_uint(rstd) & 0xFFFF0000u);
  const float l = rstd - h;
  float f[8];
  unpack8(s, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = fmaf(f[i] * h, w[i], (f[i] * l) * w[i]);
  return pack8(f);
}

}  // namespace mxk
