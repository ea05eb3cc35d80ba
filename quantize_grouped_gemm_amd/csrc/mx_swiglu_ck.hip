// SwiGLU between two MXFP8 GEMMs with its input kept for the backward in
// 8 bits, for any number of rows:
//   k_swiglu_ck_fwd   h = silu(a) b quantized both ways, [a | b] quantized
//                     along its rows (the checkpoint)
//   k_swiglu_ck_bwd   a, b from the checkpoint; [dA | dB] quantized both ways
//
// One 128 x 128 tile of h per workgroup in the tile scheme of mx_tile.h and mx_fmt.h: each
// input is read once into registers, everything else happens on chip. Rows
// past the last one enter as zeros, so the column-wise blocks that they fill
// up quantize to zeros.
//
// Both are bound by HBM. Stores: the checkpoint is read in the backward pass
// only and goes past the caches (8192 x 14336 forward 197 -> 167..186 us); of
// the backward's two outputs, 480 MB at that size, the Infinity Cache can hold
// one, so the row-wise one goes past it, and so do the checkpoint's codes,
// read for the last time (197 -> 172 us; both outputs past it 188).

#include "mx_device.h"
#include "mx_fmt.h"
#include "mx_lm.h"
#include "mx_row.h"
#include "mx_swiglu.h"
#include "mx_tile.h"

namespace mxk {

struct SwigluPack {
  const uint16_t *a, *b;     // a: dh in the backward
  uint8_t *q_row, *s_row, *q_col, *s_col, *q_ck, *s_ck;
  int32_t ld, rows, hidden, bands;

  template <class F>
  __device__ SwigluCkArgs wide() const {
    SwigluCkArgs w{};
    w.a = a; w.b = b; w.ld_ab = ld; w.dh = a; w.ld_dh = ld;
    w.rows = rows; w.hidden = hidden; w.rows_pad = padded<F>(rows);
    w.q_row = q_row; w.s_row = s_row; w.q_col = q_col; w.s_col = s_col; w.q_ck = q_ck; w.s_ck = s_ck;
    w.bands = bands;
    return w;
  }
};
static_assert(sizeof(SwigluPack) <= kArgBytes);

template <class F, bool FULL>
__device__ __forceinline__ void swiglu_ck_fwd_tile(const SwigluCkArgs& a, TileLds& l, uint32_t (&s_ck)[2][kTR], int64_t r0,
                                                   int64_t c0, int rows_valid, int rows_pad, int cols_valid) {
  uint4 v[kChunks], w[kChunks];
  fmt_load<FULL>(v, a.a + r0 * a.ld_ab + c0, a.ld_ab, rows_valid, cols_valid);
  fmt_load<FULL>(w, a.b + r0 * a.ld_ab + c0, a.ld_ab, rows_valid, cols_valid);
  const TileOut ock{a.q_ck, a.s_ck, 2 * a.hidden, a.rows, F::k128};
  fmt_rowq<F, FULL, true>(v, rows_valid, cols_valid, ock, r0, c0, s_ck[0]);
  fmt_rowq<F, FULL, true>(w, rows_valid, cols_valid, ock, r0, a.hidden + c0, s_ck[1]);
#pragma unroll
  for (int j = 0; j < kChunks; ++j)
    v[j] = make_uint4(swiglu_pair(v[j].x, w[j].x), swiglu_pair(v[j].y, w[j].y),
                      swiglu_pair(v[j].z, w[j].z), swiglu_pair(v[j].w, w[j].w));
  fmt_dual<F, FULL, false, false>(v, l, rows_valid, rows_pad, cols_valid, TileOut{a.q_row, a.s_row, a.hidden, a.rows, F::k128},
                    TileOut{a.q_col, a.s_col, a.rows_pad, a.hidden, F::k128}, r0, c0, false);
  const int t = threadIdx.x & (kTR - 1), half = (int)threadIdx.x / kTR - 2;   // the threads that fmt_dual leaves idle
  if (half >= 0) fmt_scales<F>(s_ck[half], t, rows_valid, cols_valid, ock, r0, half * a.hidden + c0);
}

template <class F>
__global__ __launch_bounds__(kFmtThreads) void k_swiglu_ck_fwd(SwigluPack pack) {
  __shared__ TileLds l;
  __shared__ uint32_t s_ck[2][kTR];
  const SwigluCkArgs a = pack.wide<F>();
  const TilePos at = tile_pos(blockIdx.x, (uint32_t)((a.hidden + kTC - 1) / kTC), (uint32_t)((a.rows_pad + kTR - 1) / kTR),
                              false);
  const int64_t r0 = at.r0, c0 = at.c0;
  const int rows_valid = (int)min<int64_t>(kTR, a.rows - r0);
  const int rows_pad = (int)min<int64_t>(kTR, a.rows_pad - r0);
  const int cols_valid = (int)min<int64_t>(kTC, a.hidden - c0);
  if (rows_valid == kTR && cols_valid == kTC)
    swiglu_ck_fwd_tile<F, true>(a, l, s_ck, r0, c0, kTR, kTR, kTC);
  else
    swiglu_ck_fwd_tile<F, false>(a, l, s_ck, r0, c0, rows_valid, rows_pad, cols_valid);
}

// Codes and scale bytes of the thread's chunks of a tile whose (0,0) is row
// r0, column c0 of the checkpoint [rows, ld]. Chunks outside the valid region
// read its last row or column in their place (loads without a branch: with
// one, the compiler carried the widened float32 values of all chunks through
// it, 256 VGPRs); the caller drops what comes of them.
template <class F, bool FULL>
__device__ __forceinline__ void tile_load_codes(uint2 (&q)[kChunks], uint32_t (&sb)[kChunks], const uint8_t* qp,
                                                const uint8_t* sp, int64_t ld, int64_t rows, int64_t r0, int64_t c0,
                                                int rows_valid, int cols_valid) {
  const uint32_t t = threadIdx.x;
  const uint32_t c = FULL ? (t & 15) * 8 : (uint32_t)min((int)(t & 15) * 8, cols_valid - 8);
  const uint8_t* qbase = qp + r0 * ld + c0;
  const uint8_t* sbase = sp + (F::k128 ? ((c0 >> 7) * rows + r0) * 4 : r0 * (ld / kBlock) + (c0 >> 5));
  const uint32_t sld = F::k128 ? 4u : (uint32_t)(ld / kBlock);
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    const uint32_t r = FULL ? (t >> 4) + kRowStep * j : (uint32_t)min((int)(t >> 4) + kRowStep * j, rows_valid - 1);
    if constexpr (FULL) {
      q[j] = load_stream8(qbase + (int64_t)(kRowStep * j) * ld + ((t >> 4) * (uint32_t)ld + c));
      sb[j] = sbase[(int64_t)(kRowStep * j) * sld + ((t >> 4) * sld + (c >> 5))];
    } else {
      q[j] = load_stream8(qbase + r * ld + c);
      sb[j] = sbase[(int64_t)r * sld + (c >> 5)];
    }
  }
}

template <class F, bool FULL>
__device__ __forceinline__ void swiglu_ck_bwd_tile(const SwigluCkArgs& a, TileLds& l, int64_t r0, int64_t c0,
                                                   int rows_valid, int rows_pad, int cols_valid) {
  const int64_t H2 = 2 * a.hidden;
  uint4 da[kChunks], db[kChunks];
  {
    uint2 qa[kChunks], qb[kChunks];
    uint32_t sa[kChunks], sb[kChunks];
    fmt_load<FULL>(da, a.dh + r0 * a.ld_dh + c0, a.ld_dh, rows_valid, cols_valid);
    tile_load_codes<F, FULL>(qa, sa, a.q_ck, a.s_ck, H2, a.rows, r0, c0, rows_valid, cols_valid);
    tile_load_codes<F, FULL>(qb, sb, a.q_ck, a.s_ck, H2, a.rows, r0, a.hidden + c0, rows_valid, cols_valid);
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      // one chunk's 32 float32 values at a time: left to itself the compiler
      // widens all eight chunks first
      asm volatile("" : "+v"(qa[j].x), "+v"(qa[j].y), "+v"(qb[j].x), "+v"(qb[j].y));
      float fa[8], fb[8], ga[8], gb[8];
      e4m3_chunk_values(qa[j], sa[j], fa);
      e4m3_chunk_values(qb[j], sb[j], fb);
      const uint32_t wd[4] = {da[j].x, da[j].y, da[j].z, da[j].w};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        swiglu_grad_f32(i & 1 ? bf16_hi(wd[i >> 1]) : bf16_lo(wd[i >> 1]), fa[i], fb[i], ga[i], gb[i]);
      const bool ok = FULL || ((int)(threadIdx.x >> 4) + kRowStep * j < rows_valid && (int)(threadIdx.x & 15) * 8 < cols_valid);
      da[j] = ok ? pack8(ga) : make_uint4(0, 0, 0, 0);
      db[j] = ok ? pack8(gb) : make_uint4(0, 0, 0, 0);
      asm volatile("" : "+v"(da[j].x), "+v"(da[j].y), "+v"(da[j].z), "+v"(da[j].w), "+v"(db[j].x), "+v"(db[j].y),
                        "+v"(db[j].z), "+v"(db[j].w));
    }
  }
  const TileOut orow{a.q_row, a.s_row, H2, a.rows, F::k128};
  const TileOut ocol{a.q_col, a.s_col, a.rows_pad, H2, F::k128};
  fmt_dual<F, FULL, true, false>(da, l, rows_valid, rows_pad, cols_valid, orow, ocol, r0, c0, true);
  fmt_dual<F, FULL, true, false>(db, l, rows_valid, rows_pad, cols_valid, orow, ocol, r0, a.hidden + c0, false);
}

template <class F>
__global__ __launch_bounds__(kFmtThreads) void k_swiglu_ck_bwd(SwigluPack pack) {
  __shared__ TileLds l;
  const SwigluCkArgs a = pack.wide<F>();
  const TilePos at = tile_pos(blockIdx.x, (uint32_t)((a.hidden + kTC - 1) / kTC), (uint32_t)((a.rows_pad + kTR - 1) / kTR),
                              a.bands);
  const int64_t r0 = at.r0, c0 = at.c0;
  const int rows_valid = (int)min<int64_t>(kTR, a.rows - r0);
  const int rows_pad = (int)min<int64_t>(kTR, a.rows_pad - r0);
  const int cols_valid = (int)min<int64_t>(kTC, a.hidden - c0);
  if (rows_valid == kTR && cols_valid == kTC)
    swiglu_ck_bwd_tile<F, true>(a, l, r0, c0, kTR, kTR, kTC);
  else
    swiglu_ck_bwd_tile<F, false>(a, l, r0, c0, rows_valid, rows_pad, cols_valid);
}

static SwigluPack pack(const SwigluCkArgs& a, const uint16_t* in, int64_t ld, bool bands) {
  return SwigluPack{in, a.b, a.q_row, a.s_row, a.q_col, a.s_col, a.q_ck, a.s_ck, (int32_t)ld, (int32_t)a.rows,
                    (int32_t)a.hidden, bands};
}

static dim3 tile_grid(const SwigluCkArgs& a) {
  return dim3((unsigned)((a.hidden + kTC - 1) / kTC * ((a.rows_pad + kTR - 1) / kTR)));
}

hipError_t launch_swiglu_ck_fwd(const SwigluCkArgs& a, hipStream_t s) {
  const SwigluPack p = pack(a, a.a, a.ld_ab, false);
  with_fmt(a.rceil, a.k128, [&](auto f) {
    hipLaunchKernelGGL(k_swiglu_ck_fwd<decltype(f)>, tile_grid(a), dim3(kFmtThreads), 0, s, p);
  });
  return hipGetLastError();
}

// Bands (tile_pos) in the backward of many tiles of long rows: 8192 x 9216 135 -> 124
// us, 8192 x 14336 206 -> 191, 16384 x 6912 191 -> 182, 4096 x 28672 214 -> 192
// (8192 x 11008 148 -> 150, 12288 x 8192 172 -> 176). Fewer tiles or shorter rows are
// slower in bands (4096 x 8192 55 -> 59, 8192 x 8192 110 -> 117, 32768 x 2560 142 ->
// 157), and so is the forward (8192 x 8192 97 -> 104, 8192 x 14336 189.5 -> 192.3,
// 16384 x 6912 184 -> 183).
static bool grad_bands(const SwigluCkArgs& a) { return tile_grid(a).x > 4096 && a.hidden > 4096; }

hipError_t launch_swiglu_ck_bwd(const SwigluCkArgs& a, hipStream_t s) {
  const SwigluPack p = pack(a, a.dh, a.ld_dh, grad_bands(a));
  with_fmt(a.rceil, a.k128, [&](auto f) {
    hipLaunchKernelGGL(k_swiglu_ck_bwd<decltype(f)>, tile_grid(a), dim3(kFmtThreads), 0, s, p);
  });
  return hipGetLastError();
}

}  // namespace mxk
