// Loads, stores and conversions that only the layer-boundary kernels use (those
// shared with the GEMMs and the quantizer are in mx_device.h).
#pragma once

#include "mx_device.h"

namespace mxk {

// load_stream16 (mx_device.h) for 8 bytes, and for stores of lines that the kernels right behind
// do not read (or that are too many for the 256 MB Infinity Cache to hold until
// they do): such lines leave the cache to the others.
__device__ __forceinline__ uint2 load_stream8(const void* p) {
  typedef unsigned v2u __attribute__((ext_vector_type(2)));
  const v2u q = __builtin_nontemporal_load(reinterpret_cast<const v2u*>(p));
  return make_uint2(q.x, q.y);
}

__device__ __forceinline__ void store_stream8(void* p, uint2 v) {
  typedef unsigned v2u __attribute__((ext_vector_type(2)));
  __builtin_nontemporal_store((v2u){v.x, v.y}, reinterpret_cast<v2u*>(p));
}

__device__ __forceinline__ void store_stream16(void* p, uint4 v) {
  typedef unsigned v4u __attribute__((ext_vector_type(4)));
  __builtin_nontemporal_store((v4u){v.x, v.y, v.z, v.w}, reinterpret_cast<v4u*>(p));
}

// 2^(b - 127) as a float32, NaN for b = 0xFF.
__device__ __forceinline__ float e8m0_f32(uint32_t b) {
  return b == 0xFFu ? __uint_as_float(0x7FC00000u) : scale_f32(b);
}

// Values of 8 E4M3 codes (little-endian) under scale byte sb, by gfx950's
// v_cvt_scalef32_pk_f32_fp8. Measured on the device it equals value times scale
// in float32 for all 256 codes under all 256 scale bytes: exact down to the
// smallest subnormals, infinity on overflow, NaN for a NaN code or scale.
__device__ __forceinline__ void e4m3_chunk_values(uint2 q, uint32_t sb, float (&f)[8]) {
  const float sc = e8m0_f32(sb);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w = i ? q.y : q.x;
    const mx_f32x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, sc, false);
    const mx_f32x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, sc, true);
    f[4 * i] = lo.x;
    f[4 * i + 1] = lo.y;
    f[4 * i + 2] = hi.x;
    f[4 * i + 3] = hi.y;
  }
}

}  // namespace mxk
