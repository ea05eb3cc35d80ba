// MX quantization of a 128 x 128 bf16 tile by 512 threads, specialised on the
// format (scale rounding, scale layout) and on whether the tile is whole. Same
// LDS swizzle and results as mx_tile.h; thread t holds 4 chunks of 8 values,
// chunk j at tile row (t >> 4) + 32 j, columns 8 (t & 15) .. + 7. LDS holds
// four tiles a CU, and with 8 waves a tile (64 VGPRs) every SIMD has 8 waves
// to issue from where 4-wave tiles leave it 4. The kernels that use it are
// close to their VALU issue rate, and here a dual quantization takes about
// half the instructions of mx_tile.h:
//   * mode and layout are template arguments, and a whole tile's loads and
//     stores carry no per-chunk bounds;
//   * addresses are a uniform 64-bit base plus a 32-bit lane offset;
//   * the block maximum stays in the upper half of a dword through its
//     exchange, where the scale byte is an add, a shift and a saturating
//     subtraction;
//   * NaN and infinity are looked for once per pass and wave; the general
//     code runs only where one is found;
//   * scale bytes are gathered in LDS and leave as whole dwords.
#pragma once

#include "mx_device.h"
#include "mx_row.h"
#include "mx_tile.h"

namespace mxk {

template <bool RCEIL, bool K128>
struct Fmt {
  static constexpr bool rceil = RCEIL, k128 = K128;
};

// n rounded up to the layout's block step.
template <class F>
__device__ __forceinline__ int64_t padded(int64_t n) {
  constexpr int64_t step = F::k128 ? 128 : kBlock;
  return (n + step - 1) / step * step;
}

constexpr int kFmtThreads = 512;
constexpr int kChunks = kTR * kTC / 8 / kFmtThreads;   // 4 per thread
constexpr int kRowStep = kFmtThreads / 16;              // rows between a thread's chunks

// The id-th of n in an order where each XCD (the workgroups of equal id mod 8)
// walks its own contiguous eighth, forwards or from its end.
__device__ __forceinline__ uint32_t band_id(uint32_t id, uint32_t n, bool reverse) {
  const uint32_t xcd = id & 7, i = id >> 3, len = n / 8 + (xcd < n % 8);
  return xcd * (n / 8) + min(xcd, n % 8) + (reverse ? len - 1 - i : i);
}

struct TilePos {
  int64_t r0, c0;
};

// Tile `id` of nx x ny in row order, or with `bands` in bands of that order:
// the eight XCDs then work on different rows at any time.
__device__ __forceinline__ TilePos tile_pos(uint32_t id, uint32_t nx, uint32_t ny, bool bands) {
  if (bands) id = band_id(id, nx * ny, false);
  const uint32_t y = id / nx;
  return TilePos{(int64_t)y * kTR, (int64_t)(id - y * nx) * kTC};
}

// LDS of one tile: the bf16 values and the scale bytes of both directions
// (one dword = four blocks per row or column).
struct TileLds {
  uint4 v[kTR * kTC / 8];
  uint32_t s_row[kTR], s_col[kTC];
};

// max |v| of a chunk's 8 values as bf16 bits in the upper half (the lower half
// holds another one's and does not affect the comparison).
__device__ __forceinline__ uint32_t absmax8_hi(uint4 v) {
  const mx_us2 a = __builtin_elementwise_max(__builtin_bit_cast(mx_us2, v.x & 0x7FFF7FFFu),
                                             __builtin_bit_cast(mx_us2, v.y & 0x7FFF7FFFu));
  const mx_us2 b = __builtin_elementwise_max(__builtin_bit_cast(mx_us2, v.z & 0x7FFF7FFFu),
                                             __builtin_bit_cast(mx_us2, v.w & 0x7FFF7FFFu));
  const uint32_t m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(a, b));
  return max(m, m << 16);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}

// max over the 4 lanes of a quad.
__device__ __forceinline__ uint32_t quad_max_hi(uint32_t m) {
  m = max(m, dpp<0xB1>(m));
  return max(m, dpp<0x4E>(m));
}

// Scale byte of a finite block maximum in the upper half of m: the exponent
// field, one more if RCEIL and the mantissa field exceeds 0x60 (adding 0x1F
// carries exactly then), minus 8, not below 0.
template <bool RCEIL>
__device__ __forceinline__ uint32_t scale_byte_hi(uint32_t m) {
  return __builtin_elementwise_sub_sat((m + (RCEIL ? 0x1F0000u : 0u)) >> 23, 8u);
}

// 2^(b - 127) for b < 255.
__device__ __forceinline__ float scale_of(uint32_t b) { return __uint_as_float(max(b << 23, 0x00400000u)); }

constexpr uint32_t kNonFiniteHi = 0x7F800000u;

// bf16 bits of 448 * 2^E for a FLOOR scale byte, in both halves.
__device__ __forceinline__ uint32_t floor_limit2(uint32_t sb) {
  const uint32_t lim = (sb << 7) + ((8u << 7) | 0x60u);
  return lim | (lim << 16);
}

// cvt4 without a defined starting value (both halves are written; the empty
// asm stands for a register of any content, a zero would cost a move).
__device__ __forceinline__ uint32_t cvt4u(uint32_t w0, uint32_t w1, float scale) {
  mx_v2s r;
  asm volatile("" : "=v"(r));
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(mx_v2bf, w0), scale, false);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(mx_v2bf, w1), scale, true);
  return __builtin_bit_cast(uint32_t, r);
}

// Codes of a chunk under a finite block's scale byte.
template <bool RCEIL>
__device__ __forceinline__ uint2 chunk_codes(uint4 v, uint32_t sb) {
  if constexpr (!RCEIL) {
    const uint32_t lim2 = floor_limit2(sb);
    v = make_uint4(clamp_pair(v.x, lim2), clamp_pair(v.y, lim2), clamp_pair(v.z, lim2), clamp_pair(v.w, lim2));
  }
  const float sc = scale_of(sb);
  return make_uint2(cvt4u(v.x, v.y, sc), cvt4u(v.z, v.w, sc));
}

// The thread's chunks of the bf16 tile whose (0,0) is `base` (uniform), row
// stride ld <= 2^26 (31 rows of 2^27 bytes fit the lanes' 32-bit offsets); zeros
// outside the valid region.
template <bool FULL>
__device__ __forceinline__ void fmt_load(uint4 (&v)[kChunks], const uint16_t* base, int64_t ld, int rows_valid,
                                         int cols_valid) {
  if constexpr (FULL) {
    const uint32_t t = threadIdx.x;
    const uint32_t off = ((t >> 4) * (uint32_t)ld + (t & 15) * 8) * 2;
#pragma unroll
    for (int j = 0; j < kChunks; ++j)
      v[j] = load_stream16(reinterpret_cast<const char*>(base + (int64_t)(kRowStep * j) * ld) + off);
  } else {
    const int t = threadIdx.x;
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int row = (t >> 4) + kRowStep * j;
      v[j] = row < rows_valid && (t & 15) * 8 < cols_valid ? load_stream16(base + row * ld + (t & 15) * 8)
                                                           : make_uint4(0, 0, 0, 0);
    }
  }
}

// Codes of 8 (16) values, non-temporal with STREAM.
template <bool STREAM>
__device__ __forceinline__ void store_codes(uint8_t* p, uint2 v) {
  if constexpr (STREAM) store_stream8(p, v);
  else *reinterpret_cast<uint2*>(p) = v;
}

template <bool STREAM>
__device__ __forceinline__ void store_codes(uint8_t* p, uint4 v) {
  if constexpr (STREAM) store_stream16(p, v);
  else *reinterpret_cast<uint4*>(p) = v;
}

// Row-wise codes of the tile from the threads' chunks; scale bytes to s_row.
// All threads must reach this function.
template <class F, bool FULL, bool STREAM>
__device__ __forceinline__ void fmt_rowq(const uint4 (&v)[kChunks], int rows_valid, int cols_valid,
                                         const TileOut& o, int64_t r0, int64_t c0, uint32_t* s_row) {
  const uint32_t t = threadIdx.x, cc = t & 15, tr = t >> 4;
  uint8_t* base = o.q + r0 * o.ld + c0;
  const uint32_t off = tr * (uint32_t)o.ld + cc * 8;
  uint32_t sb[kChunks], all = 0;
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    sb[j] = quad_max_hi(absmax8_hi(v[j]));
    all = max(all, sb[j]);
  }
  const bool special = __any(all >= kNonFiniteHi);
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    uint2 codes;
    if (!special) {
      sb[j] = scale_byte_hi<F::rceil>(sb[j]);
      codes = chunk_codes<F::rceil>(v[j], sb[j]);
    } else {
      sb[j] = scale_byte(sb[j] >> 16, F::rceil);
      codes = e4m3_chunk(v[j], sb[j], !F::rceil);
    }
    if (FULL || ((int)tr + kRowStep * j < rows_valid && (int)cc * 8 < cols_valid))
      store_codes<STREAM>(base + (int64_t)(kRowStep * j) * o.ld + off, codes);
  }
  if ((t & 3) == 0) {
    uint8_t* s = reinterpret_cast<uint8_t*>(s_row) + tr * 4 + (cc >> 2);
#pragma unroll
    for (int j = 0; j < kChunks; ++j) s[4 * kRowStep * j] = (uint8_t)sb[j];
  }
}

// Chunk j of row r = tr + 32 j goes to slot lds_unit(r, cc): as tr >> 4 is 0 or
// 1, the swizzle's 2 ((r >> 4) & 7) is 2 (tr >> 4) + 4 j, and the slot is chunk
// 0's with 4 j XORed into its unit.
__device__ __forceinline__ void fmt_to_lds(const uint4 (&v)[kChunks], TileLds& l) {
  const uint32_t t = threadIdx.x, tr = t >> 4;
  const uint32_t slot = lds_unit(tr, t & 15);
#pragma unroll
  for (int j = 0; j < kChunks; ++j) l.v[(slot ^ (4 * j)) + 16 * kRowStep * j] = v[j];
}

// Column-wise codes from the LDS copy: lane l of wave w takes rows 16 q .. 16 q
// + 15, q = l & 7, of the columns 2 cp and 2 cp + 1, cp = 8 w + (l >> 3), so the
// 8 lanes of a column pair cover 128 codes of two output rows; scale bytes to
// s_col. rows_valid counts the rows that are written, zero rows
// included.
template <class F, bool FULL, bool STREAM>
__device__ __forceinline__ void fmt_colq(TileLds& l, int rows_valid, int cols_valid, const TileOut& o, int64_t r0,
                                         int64_t c0) {
  const uint32_t* lds = reinterpret_cast<const uint32_t*>(l.v);
  const uint32_t lane = threadIdx.x & 63, w = threadIdx.x >> 6, q = lane & 7;
  uint8_t* base = o.q + c0 * o.ld + r0;
  const uint32_t cp = 8 * w + (lane >> 3);
  uint32_t v[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) v[r] = lds[lds_unit(16 * q + r, cp >> 2) * 4 + (cp & 3)];
  mx_us2 m = __builtin_bit_cast(mx_us2, v[0] & 0x7FFF7FFFu);
#pragma unroll
  for (int r = 1; r < 16; ++r) m = __builtin_elementwise_max(m, __builtin_bit_cast(mx_us2, v[r] & 0x7FFF7FFFu));
  m = __builtin_elementwise_max(m, __builtin_bit_cast(mx_us2, dpp<0xB1>(__builtin_bit_cast(uint32_t, m))));
  const uint32_t m1 = __builtin_bit_cast(uint32_t, m), m0 = m1 << 16;
  uint32_t sb0, sb1, c0w[4], c1w[4];
  const bool special = __any(max(m0, m1) >= kNonFiniteHi);
  if (!special) {
    sb0 = scale_byte_hi<F::rceil>(m0);
    sb1 = scale_byte_hi<F::rceil>(m1);
  } else {
    sb0 = scale_byte(m0 >> 16, F::rceil);
    sb1 = scale_byte(m1 >> 16, F::rceil);
  }
  if constexpr (!F::rceil) {
    const uint32_t lim2 = special ? sat_bits(sb0) | (sat_bits(sb1) << 16)
                                  : __builtin_amdgcn_perm(floor_limit2(sb1), floor_limit2(sb0), 0x07060100u);
#pragma unroll
    for (int r = 0; r < 16; ++r) v[r] = clamp_pair(v[r], lim2);
  }
  const float sc0 = scale_of(sb0), sc1 = scale_of(sb1);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t* x = &v[4 * k];
    c0w[k] = cvt4u(__builtin_amdgcn_perm(x[1], x[0], 0x05040100u), __builtin_amdgcn_perm(x[3], x[2], 0x05040100u), sc0);
    c1w[k] = cvt4u(__builtin_amdgcn_perm(x[1], x[0], 0x07060302u), __builtin_amdgcn_perm(x[3], x[2], 0x07060302u), sc1);
  }
  if (special) {   // blocks with scale 0xFF: 0x7F with each element's sign
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t a = 0x7F7F7F7Fu, b = 0x7F7F7F7Fu;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a |= ((v[4 * k + i] >> 15) & 1u) << (8 * i + 7);
        b |= ((v[4 * k + i] >> 31) & 1u) << (8 * i + 7);
      }
      if (sb0 == 0xFFu) c0w[k] = a;
      if (sb1 == 0xFFu) c1w[k] = b;
    }
  }
  if (FULL || ((int)(2 * cp) < cols_valid && (int)(16 * q) < rows_valid)) {
    const uint32_t off = 2 * cp * (uint32_t)o.ld + 16 * q;
    store_codes<STREAM>(base + off, make_uint4(c0w[0], c0w[1], c0w[2], c0w[3]));
    store_codes<STREAM>(base + o.ld + off, make_uint4(c1w[0], c1w[1], c1w[2], c1w[3]));
  }
  if ((lane & 1) == 0) {
    uint8_t* sp = reinterpret_cast<uint8_t*>(l.s_col) + 8 * cp + (q >> 1);
    sp[0] = (uint8_t)sb0;
    sp[4] = (uint8_t)sb1;
  }
}

// Stores the gathered scale bytes of `lines` tile rows (or columns) i = 0 ..:
// output row r0 + i, blocks (c0 / 32) .. as far as `extent` reaches. One
// thread a line, `i` its index.
template <class F>
__device__ __forceinline__ void fmt_scales(const uint32_t* s, int i, int lines, int extent, const TileOut& o, int64_t r0,
                                           int64_t c0) {
  if (i >= lines) return;
  const uint32_t w = s[i];
  if constexpr (F::k128) {
    *reinterpret_cast<uint32_t*>(o.s + ((c0 >> 7) * o.srows + r0 + i) * 4) = w;
  } else {
    uint8_t* p = o.s + (r0 + i) * (o.ld / kBlock) + (c0 >> 5);
#pragma unroll
    for (int b = 0; b < 4; ++b)
      if (32 * b < extent) p[b] = (uint8_t)(w >> (8 * b));
  }
}

// Both directions of the tile in v (column-wise with rows_pad >= rows_valid
// rows, the extra ones zeros). Holds barriers; ends with one if `more` work
// on the same LDS follows. RS, CS: row-wise, column-wise codes non-temporal.
template <class F, bool FULL, bool RS, bool CS>
__device__ __forceinline__ void fmt_dual(const uint4 (&v)[kChunks], TileLds& l, int rows_valid, int rows_pad,
                                         int cols_valid, const TileOut& orow, const TileOut& ocol, int64_t r0,
                                         int64_t crow, bool more) {
  fmt_rowq<F, FULL, RS>(v, rows_valid, cols_valid, orow, r0, crow, l.s_row);
  fmt_to_lds(v, l);
  __syncthreads();
  fmt_colq<F, FULL, CS>(l, rows_pad, cols_valid, ocol, r0, crow);
  __syncthreads();
  const int t = threadIdx.x;
  if (t < kTR) fmt_scales<F>(l.s_row, t, rows_valid, cols_valid, orow, r0, crow);
  else if (t < kTR + kTC) fmt_scales<F>(l.s_col, t - kTR, cols_valid, rows_pad, ocol, crow, r0);
  if (more) __syncthreads();
}

// Quantizes one chunk of row `row` at column `col` (a multiple of 8) and
// stores its codes and its block's or step's scales. All lanes must reach
// this function; `ok` (uniform over each quad) guards the stores.
template <class F, bool STREAM>
__device__ __forceinline__ void fmt_chunk(uint4 v, bool ok, const TileOut& o, int64_t row, uint32_t col) {
  const uint32_t m = quad_max_hi(absmax8_hi(v));
  uint32_t sb;
  uint2 codes;
  if (!__any(m >= kNonFiniteHi)) {
    sb = scale_byte_hi<F::rceil>(m);
    codes = chunk_codes<F::rceil>(v, sb);
  } else {
    sb = scale_byte(m >> 16, F::rceil);
    codes = e4m3_chunk(v, sb, !F::rceil);
  }
  if constexpr (F::k128) {
    uint32_t packed = sb << (8 * ((col >> 5) & 3));
    packed |= dpp<0x124>(packed);
    packed |= dpp<0x128>(packed);
    if (ok) {
      store_codes<STREAM>(o.q + row * o.ld + col, codes);
      if ((col & 127) == 0) *reinterpret_cast<uint32_t*>(o.s + ((int64_t)(col >> 7) * o.srows + row) * 4) = packed;
    }
  } else if (ok) {
    store_codes<STREAM>(o.q + row * o.ld + col, codes);
    if ((col & 31) == 0) o.s[row * (o.ld / kBlock) + (col >> 5)] = (uint8_t)sb;
  }
}

// Calls f(Fmt<..>{}) for the runtime mode and layout.
template <class Fn>
inline void with_fmt(bool rceil, bool k128, Fn f) {
  if (rceil) {
    if (k128) f(Fmt<true, true>{});
    else f(Fmt<true, false>{});
  } else {
    if (k128) f(Fmt<false, true>{});
    else f(Fmt<false, false>{});
  }
}

}  // namespace mxk
