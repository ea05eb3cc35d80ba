// FP8 quantization with one float32 scale for a block of 128: 1 x 128 along
// the rows and along the columns (activations and gradients), 128 x 128
// (weights); and rows gathered on the way, in this format and in MXFP8.
//
//   s = float32(max(amax, 2^-100) / 448), or the power of two at or above it
//   code = E4M3(float32(v / s)), both roundings to nearest even
// A block that holds a NaN or infinity gets scale NaN and codes 0x7F with each
// element's sign. The quotient is the correctly rounded one: about one value in
// 500 of bf16 data lies exactly between two codes of v * 448 / amax, and there
// a product with a rounded reciprocal would take either. The block's reciprocal
// is therefore held in two parts, 1/s = h + l to some 2^-46, and v/s is fma(v, h, v l),
// two instructions. (Exactly halfway quotients come out exact; no others are close
// enough to a border: every pair of mantissas of amax and v gives the division's code.)
// h lies below 1/s, so l >= 0 and -0 stays -0. Under a power of two the
// conversion instruction divides by itself.
//
// Tiles of 128 x 128 by 512 threads as in mx_fmt.h; every input is read once and
// both directions leave from the chip. Bound by HBM where nothing is weighted: 32
// weights of 4096 x 7168 both ways 695 us (5.4 TB/s), 1000 x 4096 activations both ways
// 5.4 us (latency). Weighted rows under float32 scales take some 20 vector
// instructions a value and are bound by those: 6144 x 5120 both ways 22.5 us.

#include "mx_device.h"
#include "mx_fmt.h"
#include "mx_moe.h"
#include "mx_row.h"

namespace mxk {

typedef short mx_s2 __attribute__((ext_vector_type(2)));

constexpr float kTinyMax = 0x1p-100f;

struct BlockScale {
  float s, h, l;   // scale and its reciprocal h + l (float32 scales only)
  bool bad;        // a NaN or infinity in the block
};

// Scale of a block whose largest magnitude has the bf16 bits `amax`. The quotient
// by 448 is corrected by its remainder (128 mantissas of amax, all of them tested
// against the division); h is the hardware's reciprocal (off by at most one step), two steps down.
template <bool POW2>
__device__ __forceinline__ BlockScale block_scale(uint32_t amax) {
  constexpr float kInv = 1.0f / 448.0f;
  const float m = __uint_as_float(max(amax << 16, __float_as_uint(kTinyMax)));
  const float q = m * kInv;
  float s = fmaf(fmaf(-q, 448.0f, m), kInv, q);
  BlockScale b;
  b.bad = amax >= 0x7F80u;
  if constexpr (POW2) {
    s = __uint_as_float((__float_as_uint(s) + 0x7FFFFFu) & 0x7F800000u);
    b.h = b.l = 0.0f;
  } else {
    b.h = __uint_as_float(__float_as_uint(__builtin_amdgcn_rcpf(s)) - 2);
    b.l = fmaf(-s, b.h, 1.0f) * b.h;
  }
  b.s = b.bad ? __uint_as_float(0x7FC00000u) : s;
  return b;
}

__device__ __forceinline__ float quotient(float v, const BlockScale& b) {
  return fmaf(v, b.h, v * b.l);
}

// Codes of 4 values, little-endian.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  int r;
  asm volatile("" : "=v"(r));     // both halves are written
  r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, r, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

// 0x7F with the signs of 4 bf16 values (two dwords).
__device__ __forceinline__ uint32_t nan_codes(uint32_t w0, uint32_t w1) {
  return 0x7F7F7F7Fu | ((w0 >> 8) & 0x80u) | ((w0 >> 16) & 0x8000u) | ((w1 << 8) & 0x800000u) | (w1 & 0x80000000u);
}

// Codes of a chunk. All lanes must reach this function.
template <bool POW2>
__device__ __forceinline__ uint2 block_codes(uint4 v, const BlockScale& b) {
  uint2 c;
  if constexpr (POW2) {
    c = make_uint2(cvt4u(v.x, v.y, b.s), cvt4u(v.z, v.w, b.s));
  } else {
    float f[8];
    unpack8(v, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = quotient(f[i], b);
    c = make_uint2(codes4(f[0], f[1], f[2], f[3]), codes4(f[4], f[5], f[6], f[7]));
  }
  if (__any(b.bad) && b.bad) c = make_uint2(nan_codes(v.x, v.y), nan_codes(v.z, v.w));
  return c;
}

// bf16 of w v rounded once. The float32 product p is off by e = w v - p, which
// matters only where p lies on a border of bf16, its lower half 0x8000: one product in
// 65536, and the least of 16 signed bits, looked for with packed minima. e is formed in
// float64, which holds the product; in float32 it would vanish where p is subnormal.
__device__ __forceinline__ uint4 weigh(uint4 v, float w) {
  float f[8], p[8];
  unpack8(v, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) p[i] = w * f[i];
  mx_s2 m{0, 0};
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint32_t low = __builtin_amdgcn_perm(__float_as_uint(p[i + 1]), __float_as_uint(p[i]), 0x05040100u);
    m = __builtin_elementwise_min(m, __builtin_bit_cast(mx_s2, low));
  }
  if (min(m.x, m.y) == INT16_MIN) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t b = __float_as_uint(p[i]);
      const double e = fma((double)w, (double)f[i], -(double)p[i]);
      if ((b & 0xFFFFu) == 0x8000u && e != 0.0) b += (e > 0.0) == (p[i] > 0.0f) ? 1u : ~0u;
      p[i] = __uint_as_float(b);
    }
  }
  return pack8(p);
}

// The source of output row r: NULL if there is none (its values are zeros).
template <bool MAP>
__device__ __forceinline__ const uint16_t* row_source(const RowsQuantArgs& a, FastDiv top, int64_t r, float& w) {
  w = 1.0f;
  if (r >= a.rows) return nullptr;
  if constexpr (!MAP) return a.x + r * a.ld;
  const int32_t slot = a.src[r];
  if (slot < 0) return nullptr;
  const int64_t row = fdiv((uint32_t)slot, top);
  if (row >= a.x_rows) return nullptr;
  if (a.weights) w = a.weights[slot];
  return a.x + row * a.ld;
}

// Workgroup id -> block of columns bx and band of rows by, columns first.
__device__ __forceinline__ void grid_pos(uint32_t nx, int64_t& bx, int64_t& by) {
  const uint32_t y = blockIdx.x / nx;
  by = y;
  bx = blockIdx.x - y * nx;
}

// The tiles of gathered rows go through column by column, an eighth of them an
// XCD: a token's row is read once for each of its experts, and the 256 bytes of
// it that a column of tiles needs (2 MB of 8192 tokens) stay in the XCD's L2
// meanwhile. us of 8192 x 7168 to 8 of 32 experts in MXFP8 both ways, columns one
// by one / two / seven together / rows first: 199, 205, 268, 281 with the tokens' rows
// in the Infinity Cache, 272, 290, 294, 315 from HBM.
template <bool MAP>
__device__ __forceinline__ void tile_pos_of(uint32_t nx, uint32_t ny, int64_t& bx, int64_t& by) {
  if constexpr (!MAP) return grid_pos(nx, bx, by);
  const uint32_t id = band_id(blockIdx.x, nx * ny, false), x = id / ny;
  bx = x;
  by = id - x * ny;
}

// The thread's 4 chunks of the tile at (r0, c0); false if none of its rows has a source.
template <bool MAP>
__device__ __forceinline__ bool load_rows(uint4 (&v)[kChunks], const RowsQuantArgs& a, FastDiv top, int64_t r0, int64_t c0,
                                          int cols_valid) {
  const int t = threadIdx.x;
  const uint16_t* p[kChunks];
  float w[kChunks];
#pragma unroll
  for (int j = 0; j < kChunks; ++j) p[j] = row_source<MAP>(a, top, r0 + (t >> 4) + kRowStep * j, w[j]);
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    // rows that a map repeats are read again by other workgroups: those stay in the caches
    const uint16_t* q = p[j] + c0 + 8 * (t & 15);
    v[j] = p[j] && 8 * (t & 15) < cols_valid ? (MAP ? *reinterpret_cast<const uint4*>(q) : load_stream16(q))
                                             : make_uint4(0, 0, 0, 0);
  }
  if (MAP && a.weights) {
#pragma unroll
    for (int j = 0; j < kChunks; ++j) v[j] = weigh(v[j], w[j]);
  }
  return p[0] || p[1] || p[2] || p[3];
}

// A whole tile of zeros (rows behind the last group): its codes both ways.
template <bool STREAM>
__device__ __forceinline__ void zero_codes(const RowsQuantArgs& a, int64_t r0, int64_t c0) {
  const int t = threadIdx.x;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int line = (t >> 3) + 64 * j;      // 8 lanes a line of 128 codes
    store_codes<STREAM>(a.q_row + (r0 + line) * a.cols + c0 + 16 * (t & 7), make_uint4(0, 0, 0, 0));
    store_codes<STREAM>(a.q_col + (c0 + line) * a.rows_pad + r0 + 16 * (t & 7), make_uint4(0, 0, 0, 0));
  }
}

// max |v| bits over 16 lanes of two chunks at once: each keeps a half of the
// dword that goes through the exchanges.
__device__ __forceinline__ void row16_max_pair(uint4 a, uint4 b, uint32_t& ma, uint32_t& mb) {
  auto part = [](uint4 v) {
    const mx_us2 lo = __builtin_elementwise_max(__builtin_bit_cast(mx_us2, v.x & 0x7FFF7FFFu),
                                                __builtin_bit_cast(mx_us2, v.y & 0x7FFF7FFFu));
    const mx_us2 hi = __builtin_elementwise_max(__builtin_bit_cast(mx_us2, v.z & 0x7FFF7FFFu),
                                                __builtin_bit_cast(mx_us2, v.w & 0x7FFF7FFFu));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(lo, hi));
  };
  const uint32_t x = part(a), y = part(b);
  mx_us2 m = __builtin_elementwise_max(__builtin_bit_cast(mx_us2, __builtin_amdgcn_perm(y, x, 0x05040100u)),
                                       __builtin_bit_cast(mx_us2, __builtin_amdgcn_perm(y, x, 0x07060302u)));
  m = __builtin_elementwise_max(m, __builtin_bit_cast(mx_us2, dpp<0xB1>(__builtin_bit_cast(uint32_t, m))));
  m = __builtin_elementwise_max(m, __builtin_bit_cast(mx_us2, dpp<0x4E>(__builtin_bit_cast(uint32_t, m))));
  m = __builtin_elementwise_max(m, __builtin_bit_cast(mx_us2, dpp<0x141>(__builtin_bit_cast(uint32_t, m))));
  m = __builtin_elementwise_max(m, __builtin_bit_cast(mx_us2, dpp<0x140>(__builtin_bit_cast(uint32_t, m))));
  ma = m.x;
  mb = m.y;
}

// Row-wise only: 16 lanes a row and block, 16 rows a workgroup, so that few
// rows spread over many workgroups.
template <bool MAP, bool POW2, bool STREAM>
__global__ __launch_bounds__(256) void k_b128_rows(RowsQuantArgs a, FastDiv top) {
  const int cc = threadIdx.x & 15;
  int64_t bx, by;
  tile_pos_of<MAP>((uint32_t)(a.cols / 128), (uint32_t)((a.rows + 15) / 16), bx, by);
  const int64_t r = by * 16 + (threadIdx.x >> 4), c = bx * 128 + 8 * cc;
  float w;
  const uint16_t* p = row_source<MAP>(a, top, r, w);
  uint4 v = make_uint4(0, 0, 0, 0);
  if (p) v = MAP ? *reinterpret_cast<const uint4*>(p + c) : load_stream16(p + c);
  if (MAP && a.weights) v = weigh(v, w);
  const BlockScale b = block_scale<POW2>(row16_max(absmax8_bits(v)));
  const uint2 q = block_codes<POW2>(v, b);
  if (r >= a.rows) return;
  store_codes<STREAM>(a.q_row + r * a.cols + c, q);
  if (cc == 0) reinterpret_cast<float*>(a.s_row)[bx * a.rows + r] = b.s;
}

template <bool MAP, bool POW2, bool STREAM>
__global__ __launch_bounds__(kFmtThreads) void k_b128_tile(RowsQuantArgs a, FastDiv top) {
  __shared__ TileLds l;
  const int t = threadIdx.x;
  int64_t bx, by;
  tile_pos_of<MAP>((uint32_t)(a.cols / kTC), (uint32_t)(a.rows_pad / kTR), bx, by);
  const int64_t r0 = by * kTR, c0 = bx * kTC;
  uint4 v[kChunks];
  const bool some = load_rows<MAP>(v, a, top, r0, c0, kTC);
  if (MAP && r0 + kTR <= a.rows && !__syncthreads_or(some)) {
    zero_codes<STREAM>(a, r0, c0);
    const float z = block_scale<POW2>(0).s;
    if (t < kTR) reinterpret_cast<float*>(a.s_row)[bx * a.rows + r0 + t] = z;
    else if (t < kTR + kTC) reinterpret_cast<float*>(a.s_col)[by * a.cols + c0 + t - kTR] = z;
    return;
  }
  if (a.q_row) {
    uint32_t m[kChunks];
#pragma unroll
    for (int j = 0; j < kChunks; j += 2) row16_max_pair(v[j], v[j + 1], m[j], m[j + 1]);
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int64_t r = r0 + (t >> 4) + kRowStep * j;
      const BlockScale b = block_scale<POW2>(m[j]);
      const uint2 q = block_codes<POW2>(v[j], b);
      if (r < a.rows) {
        store_codes<STREAM>(a.q_row + r * a.cols + c0 + 8 * (t & 15), q);
        if ((t & 15) == 0) reinterpret_cast<float*>(a.s_row)[bx * a.rows + r] = b.s;
      }
    }
  }
  fmt_to_lds(v, l);
  __syncthreads();
  // column pair cp, rows 16 q .. 16 q + 15 (as in fmt_colq); 8 lanes hold a pair's 128 rows
  const uint32_t* lds = reinterpret_cast<const uint32_t*>(l.v);
  const uint32_t lane = t & 63, q = lane & 7, cp = 8 * (t >> 6) + (lane >> 3);
  uint32_t x[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) x[r] = lds[lds_unit(16 * q + r, cp >> 2) * 4 + (cp & 3)];
  mx_us2 m = __builtin_bit_cast(mx_us2, x[0] & 0x7FFF7FFFu);
#pragma unroll
  for (int r = 1; r < 16; ++r) m = __builtin_elementwise_max(m, __builtin_bit_cast(mx_us2, x[r] & 0x7FFF7FFFu));
  m = __builtin_elementwise_max(m, __builtin_bit_cast(mx_us2, dpp<0xB1>(__builtin_bit_cast(uint32_t, m))));
  m = __builtin_elementwise_max(m, __builtin_bit_cast(mx_us2, dpp<0x4E>(__builtin_bit_cast(uint32_t, m))));
  m = __builtin_elementwise_max(m, __builtin_bit_cast(mx_us2, dpp<0x141>(__builtin_bit_cast(uint32_t, m))));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const BlockScale b = block_scale<POW2>(h ? m.y : m.x);
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t* w = &x[4 * k];
      if constexpr (POW2) {
        const uint32_t sel = h ? 0x07060302u : 0x05040100u;
        c[k] = cvt4u(__builtin_amdgcn_perm(w[1], w[0], sel), __builtin_amdgcn_perm(w[3], w[2], sel), b.s);
      } else {
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = quotient(h ? bf16_hi(w[i]) : bf16_lo(w[i]), b);
        c[k] = codes4(f[0], f[1], f[2], f[3]);
      }
    }
    if (b.bad) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        c[k] = 0x7F7F7F7Fu;
#pragma unroll
        for (int i = 0; i < 4; ++i) c[k] |= ((x[4 * k + i] >> (h ? 31 : 15)) & 1u) << (8 * i + 7);
      }
    }
    const int64_t col = c0 + 2 * cp + h;
    store_codes<STREAM>(a.q_col + col * a.rows_pad + r0 + 16 * q, make_uint4(c[0], c[1], c[2], c[3]));
    if (q == 0) reinterpret_cast<float*>(a.s_col)[by * a.cols + col] = b.s;
  }
}

// The 4 x 4 bytes of four dwords transposed.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
  const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
  w[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
  w[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
  w[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
  w[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

// Weights: one scale a 128 x 128 tile, so the transposed copy holds the same
// codes, moved through LDS as bytes (row pitch 33 dwords: the 16 lanes that
// read 8 rows each start 8 banks apart).
constexpr int kBytePitch = 33;

template <bool POW2, bool STREAM>
__global__ __launch_bounds__(kFmtThreads) void k_b128_weight(B128WeightArgs a, uint32_t tiles_r) {
  __shared__ uint32_t bytes[kTR * kBytePitch];
  __shared__ uint32_t wave_max[kFmtThreads / 64];
  const int t = threadIdx.x, cc = t & 15;
  int64_t bx, by;
  grid_pos((uint32_t)((a.cols + kTC - 1) / kTC), bx, by);
  const int64_t e = (uint32_t)by / tiles_r, tr = by - e * tiles_r;
  const int64_t r0 = tr * kTR, c0 = bx * kTC;
  const int rows_valid = (int)min<int64_t>(kTR, a.rows - r0), cols_valid = (int)min<int64_t>(kTC, a.cols - c0);
  const uint16_t* w = a.w + (e * a.rows + r0) * a.cols + c0;
  uint4 v[kChunks];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    const int row = (t >> 4) + kRowStep * j;
    v[j] = row < rows_valid && 8 * cc < cols_valid ? load_stream16(w + row * a.cols + 8 * cc) : make_uint4(0, 0, 0, 0);
    m = max(m, absmax8_bits(v[j]));
  }
  m = row16_max(m);
  m = max(m, (uint32_t)__shfl_xor((int)m, 16));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32));
  if ((t & 63) == 0) wave_max[t >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kFmtThreads / 64; ++i) m = max(m, wave_max[i]);
  const BlockScale b = block_scale<POW2>(m);
  uint8_t* q = a.q + (e * a.rows + r0) * a.cols + c0;
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    const int row = (t >> 4) + kRowStep * j;
    const uint2 c = block_codes<POW2>(v[j], b);
    if (row < rows_valid && 8 * cc < cols_valid) store_codes<STREAM>(q + row * a.cols + 8 * cc, c);
    bytes[row * kBytePitch + 2 * cc] = c.x;
    bytes[row * kBytePitch + 2 * cc + 1] = c.y;
  }
  const int64_t sr = tiles_r, sc = (a.cols + kTC - 1) / kTC;
  if (t == 0) {
    a.s[(e * sc + bx) * sr + tr] = b.s;
    if (a.q_t) a.s_t[(e * sr + tr) * sc + bx] = b.s;
  }
  if (!a.q_t) return;
  __syncthreads();
  // lane: rows 8 p .. 8 p + 7 (p = t & 15) of columns 4 cq .. 4 cq + 3: 16 lanes write a column's 128 codes
  const int p = t & 15, cq = t >> 4;
  uint32_t x[2][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[h][i] = bytes[(8 * p + 4 * h + i) * kBytePitch + cq];
    transpose4(x[h]);
  }
  if (8 * p >= rows_valid || 4 * cq >= cols_valid) return;
  uint8_t* qt = a.q_t + (e * a.cols + c0 + 4 * cq) * a.rows + r0 + 8 * p;
#pragma unroll
  for (int i = 0; i < 4; ++i) store_codes<STREAM>(qt + i * a.rows, make_uint2(x[0][i], x[1][i]));
}

// Gathered rows in MXFP8 (the tile quantizer of mx_fmt.h).
template <class F, bool DUAL, bool STREAM>
__global__ __launch_bounds__(kFmtThreads) void k_gather_mx(RowsQuantArgs a, FastDiv top) {
  __shared__ TileLds l;
  int64_t bx, by;
  tile_pos_of<true>((uint32_t)((a.cols + kTC - 1) / kTC), (uint32_t)((a.rows_pad + kTR - 1) / kTR), bx, by);
  const int64_t r0 = by * kTR, c0 = bx * kTC;
  const int rows_valid = (int)min<int64_t>(kTR, a.rows - r0), cols_valid = (int)min<int64_t>(kTC, a.cols - c0);
  const int rows_pad = (int)min<int64_t>(kTR, a.rows_pad - r0);
  const TileOut orow{a.q_row, reinterpret_cast<uint8_t*>(a.s_row), a.cols, a.rows, F::k128};
  const TileOut ocol{a.q_col, reinterpret_cast<uint8_t*>(a.s_col), a.rows_pad, a.cols, F::k128};
  uint4 v[kChunks];
  const bool some = load_rows<true>(v, a, top, r0, c0, cols_valid);
  if constexpr (DUAL) {
    if (rows_valid == kTR && cols_valid == kTC && !__syncthreads_or(some)) {
      zero_codes<STREAM>(a, r0, c0);
      if (threadIdx.x < kTR) l.s_row[threadIdx.x] = l.s_col[threadIdx.x] = 0;
      if (threadIdx.x < kTR) fmt_scales<F>(l.s_row, threadIdx.x, kTR, kTC, orow, r0, c0);
      if (threadIdx.x < kTR) fmt_scales<F>(l.s_col, threadIdx.x, kTC, kTR, ocol, c0, r0);
    } else if (rows_valid == kTR && cols_valid == kTC)
      fmt_dual<F, true, STREAM, STREAM>(v, l, kTR, kTR, kTC, orow, ocol, r0, c0, false);
    else
      fmt_dual<F, false, STREAM, STREAM>(v, l, rows_valid, rows_pad, cols_valid, orow, ocol, r0, c0, false);
  } else {
    fmt_rowq<F, false, STREAM>(v, rows_valid, cols_valid, orow, r0, c0, l.s_row);
    __syncthreads();
    if (threadIdx.x < kTR) fmt_scales<F>(l.s_row, threadIdx.x, rows_valid, cols_valid, orow, r0, c0);
  }
}

// Codes beyond what the 256 MB Infinity Cache can hold until a product reads them
// go past it: 8192 x 7168 to 8 of 32 experts both ways 287 -> 204 us (one direction
// alone past it 280), row-wise only 198 -> 130, 16384 x 2048 to 4 of 16 row-wise
// 61 -> 42. Fewer codes stay in it for the product.
static bool stream_codes(int64_t rows, int64_t cols) { return rows * cols > (100ll << 20); }

hipError_t launch_gather_mx(const RowsQuantArgs& a, hipStream_t s) {
  if (a.rows_pad == 0) return hipSuccess;
  const dim3 grid((unsigned)(((a.cols + kTC - 1) / kTC) * ((a.rows_pad + kTR - 1) / kTR)));
  const FastDiv top = make_fastdiv((uint32_t)a.top);
  with_fmt(a.rceil, a.k128, [&](auto f) {
    using Fm = decltype(f);
    auto go = [&](auto dual) {
      if (stream_codes(a.rows, a.cols)) hipLaunchKernelGGL((k_gather_mx<Fm, dual, true>), grid, dim3(kFmtThreads), 0, s, a, top);
      else hipLaunchKernelGGL((k_gather_mx<Fm, dual, false>), grid, dim3(kFmtThreads), 0, s, a, top);
    };
    if (a.q_col) go(std::true_type{});
    else go(std::false_type{});
  });
  return hipGetLastError();
}

hipError_t launch_b128_quant(const RowsQuantArgs& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const FastDiv top = make_fastdiv((uint32_t)a.top);
  auto go = [&](auto map, auto pow2) {
    if (a.q_col) {
      const dim3 grid((unsigned)((a.cols / kTC) * (a.rows_pad / kTR)));
      if (stream_codes(a.rows, a.cols)) hipLaunchKernelGGL((k_b128_tile<map, pow2, true>), grid, dim3(kFmtThreads), 0, s, a, top);
      else hipLaunchKernelGGL((k_b128_tile<map, pow2, false>), grid, dim3(kFmtThreads), 0, s, a, top);
    } else {
      const dim3 grid((unsigned)((a.cols / kTC) * ((a.rows + 15) / 16)));
      if (stream_codes(a.rows, a.cols)) hipLaunchKernelGGL((k_b128_rows<map, pow2, true>), grid, dim3(256), 0, s, a, top);
      else hipLaunchKernelGGL((k_b128_rows<map, pow2, false>), grid, dim3(256), 0, s, a, top);
    }
  };
  using T = std::true_type;
  using F = std::false_type;
  if (a.src) {
    if (a.rceil) go(T{}, T{});
    else go(T{}, F{});
  } else {
    if (a.rceil) go(F{}, T{});
    else go(F{}, F{});
  }
  return hipGetLastError();
}

hipError_t launch_b128_weight(const B128WeightArgs& a, hipStream_t s) {
  if (a.batch == 0 || a.rows == 0) return hipSuccess;
  const uint32_t tiles_r = (uint32_t)((a.rows + kTR - 1) / kTR);
  const dim3 grid((unsigned)(((a.cols + kTC - 1) / kTC) * a.batch * tiles_r));
  auto go = [&](auto pow2) {
    if (stream_codes(a.batch * a.rows, a.cols))
      hipLaunchKernelGGL((k_b128_weight<pow2, true>), grid, dim3(kFmtThreads), 0, s, a, tiles_r);
    else
      hipLaunchKernelGGL((k_b128_weight<pow2, false>), grid, dim3(kFmtThreads), 0, s, a, tiles_r);
  };
  if (a.rceil) go(std::true_type{});
  else go(std::false_type{});
  return hipGetLastError();
}

}  // namespace mxk
