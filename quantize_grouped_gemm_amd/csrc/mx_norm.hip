// Residual addition + RMS norm + MX quantization, and its gradient:
//   k_norm_row    s = x + r, rstd, row-wise codes of y and of s (checkpoint)
//   k_norm_bwd    dx, its row-wise codes, partial sums of dw
//   k_norm_dw     joins the partial sums of dw
//   k_norm_col    column-wise codes of y (recomputed from s and rstd) or dx
//
// Row-wise work needs the whole row's statistic before its first output, and
// column-wise blocks span 32 rows, so the two directions are two launches:
// the row kernels hold whole rows in registers (mx_row.h), the column kernel
// reads s or dx back in 128 x 128 tiles (mx_tile.h).

#include "mx_device.h"
#include "mx_fmt.h"
#include "mx_lm.h"
#include "mx_row.h"
#include "mx_tile.h"

namespace mxk {

// 256 threads = 4 / WAVES rows per workgroup, NCH chunks per lane.
template <int WAVES, int NCH>
__global__ __launch_bounds__(256) void k_norm_row(NormFwdArgs a) {
  __shared__ float buf[4];
  const int lane = threadIdx.x & (64 * WAVES - 1);
  const int64_t row = (int64_t)blockIdx.x * (4 / WAVES) + threadIdx.x / (64 * WAVES);
  const bool live = row < a.rows;
  uint4 v[NCH];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int col = 8 * (lane + 64 * WAVES * i);
    const bool ok = live && col < a.cols;
    v[i] = ok ? load_stream16(a.x + row * a.ld_x + col) : make_uint4(0, 0, 0, 0);
    float f[8];
    unpack8(v[i], f);
    if (a.r) {
      const uint4 u = ok ? load_stream16(a.r + row * a.ld_r + col) : make_uint4(0, 0, 0, 0);
      float g[8];
      unpack8(u, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] += g[k];
      v[i] = pack8(f);
      if (ok) *reinterpret_cast<uint4*>(a.sum + row * a.cols + col) = v[i];
      unpack8(v[i], f);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fmaf(f[k], f[k], ss);
  }
  ss = group_sum<WAVES>(ss, buf);
  const float rstd = 1.0f / sqrtf(ss / (float)a.cols + a.eps);
  if (live && lane == 0) a.rstd[row] = rstd;
  const TileOut orow{a.q_row, a.s_row, a.cols, a.rows, a.k128};
  const TileOut ock{a.q_ck, a.s_ck, a.cols, a.rows, a.k128};
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int col = 8 * (lane + 64 * WAVES * i);
    const bool ok = live && col < a.cols;
    if (a.q_ck) chunk_rowq(v[i], ok, a.rceil, ock, row, col);
    float w[8] = {};
    if (ok) load8f(a.w + col, w);
    chunk_rowq(norm_chunk(v[i], rstd, w), ok, a.rceil, orow, row, col);
  }
}

// Rows per partial sum of dw.
constexpr int64_t kDwRows = 16;

static int64_t dw_parts(int64_t rows) { return (rows + kDwRows - 1) / kDwRows; }

template <int WAVES, int NCH, bool CK>
__global__ __launch_bounds__(256) void k_norm_bwd(NormBwdArgs a) {
  __shared__ float buf[2][4];
  const int lane = threadIdx.x & (64 * WAVES - 1);
  const int64_t part = (int64_t)blockIdx.x * (4 / WAVES) + threadIdx.x / (64 * WAVES);
  float dw[NCH][8] = {};
  const float inv_n = 1.0f / (float)a.cols;
  const TileOut orow{a.q_row, a.s_row, a.cols, a.rows, a.k128};
  for (int rr = 0; rr < kDwRows; ++rr) {
    const int64_t row = part * kDwRows + rr;
    const bool live = row < a.rows;
    const float rstd = live ? a.rstd[row] : 0.0f;
    uint4 dy[NCH];
    float xh[NCH][8];
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int col = 8 * (lane + 64 * WAVES * i);
      const bool ok = live && col < a.cols;
      dy[i] = ok ? load_stream16(a.dy + row * a.ld_dy + col) : make_uint4(0, 0, 0, 0);
      if constexpr (CK) {
        uint2 q = make_uint2(0, 0);
        uint32_t sb = 0;
        if (ok) {
          q = *reinterpret_cast<const uint2*>(a.q_ck + row * a.cols + col);
          sb = a.k128 ? a.s_ck[((int64_t)(col >> 7) * a.rows + row) * 4 + ((col >> 5) & 3)]
                      : a.s_ck[row * (a.cols / kBlock) + (col >> 5)];
        }
        e4m3_chunk_values(q, sb, xh[i]);
      } else {
        unpack8(ok ? load_stream16(a.x + row * a.ld_x + col) : make_uint4(0, 0, 0, 0), xh[i]);
      }
      float w[8] = {}, d[8];
      if (ok) load8f(a.w + col, w);
      unpack8(dy[i], d);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        xh[i][k] *= rstd;
        c = fmaf(d[k] * w[k], xh[i][k], c);
        dw[i][k] = fmaf(d[k], xh[i][k], dw[i][k]);
      }
    }
    c = group_sum<WAVES>(c, buf[rr & 1]) * inv_n;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int col = 8 * (lane + 64 * WAVES * i);
      const bool ok = live && col < a.cols;
      float w[8] = {}, d[8], e[8] = {};
      if (ok) load8f(a.w + col, w);
      unpack8(dy[i], d);
      if (a.dsum && ok) unpack8(load_stream16(a.dsum + row * a.ld_dsum + col), e);
#pragma unroll
      for (int k = 0; k < 8; ++k) e[k] = fmaf(fmaf(-xh[i][k], c, d[k] * w[k]), rstd, e[k]);
      const uint4 v = pack8(e);
      if (ok) *reinterpret_cast<uint4*>(a.dx + row * a.cols + col) = v;
      if (a.q_row) chunk_rowq(v, ok, a.rceil, orow, row, col);
    }
  }
  if (part * kDwRows < a.rows) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int col = 8 * (lane + 64 * WAVES * i);
      if (col < a.cols) {
        float4* p = reinterpret_cast<float4*>(a.work + part * a.cols + col);
        p[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
        p[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
      }
    }
  }
}

// dw[c] = sum over the parts of work[part, c]: 32 columns per workgroup, 32
// threads down each, joined in LDS in a fixed order.
__global__ __launch_bounds__(1024) void k_norm_dw(const float* work, int64_t parts, int64_t cols, float* dw) {
  __shared__ float acc[32][33];
  const int c = threadIdx.x & 31, p0 = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + c;
  float s = 0.0f;
  for (int64_t p = p0; p < parts; p += 32) s += work[p * cols + col];
  acc[p0][c] = s;
  __syncthreads();
  if (p0 == 0) {
    float t = 0.0f;
    for (int i = 0; i < 32; ++i) t += acc[i][c];
    dw[col] = t;
  }
}

struct NormColArgs {
  const uint16_t* x;
  int64_t ld, rows, rows_pad, cols;
  const float *rstd, *w;     // NULL: quantize x itself
  bool rceil, k128;
  uint8_t *q, *s;
};

template <class F, bool NORM, bool FULL>
__device__ __forceinline__ void norm_col_tile(const NormColArgs& a, TileLds& l, int64_t r0, int64_t c0, int rows_valid,
                                              int rows_pad, int cols_valid) {
  uint4 v[kTileChunks];
  fmt_load<FULL>(v, a.x + r0 * a.ld + c0, a.ld, rows_valid, cols_valid);
  const int t = threadIdx.x, cc = t & 15;
  if constexpr (NORM) {
    float w[8] = {};
    if (FULL || cc * 8 < cols_valid) load8f(a.w + c0 + cc * 8, w);
#pragma unroll
    for (int j = 0; j < kTileChunks; ++j) {
      const int row = (t >> 4) + 16 * j;
      // rows past the last stay +0 whatever w holds
      if (FULL || row < rows_valid) v[j] = norm_chunk(v[j], a.rstd[r0 + row], w);
    }
  }
  fmt_to_lds(v, l);
  __syncthreads();
  const TileOut o{a.q, a.s, a.rows_pad, a.cols, F::k128};
  fmt_colq<F, FULL>(l, rows_pad, cols_valid, o, r0, c0);
  __syncthreads();
  if (t < kTC) fmt_scales<F>(l.s_col, t, cols_valid, rows_pad, o, c0, r0);
}

template <class F, bool NORM>
__global__ __launch_bounds__(kTileThreads) void k_norm_col(NormColArgs a) {
  __shared__ TileLds l;
  const int64_t r0 = (int64_t)blockIdx.y * kTR;
  const int64_t c0 = (int64_t)blockIdx.x * kTC;
  const int rows_valid = (int)min<int64_t>(kTR, a.rows - r0);
  const int rows_pad = (int)min<int64_t>(kTR, a.rows_pad - r0);
  const int cols_valid = (int)min<int64_t>(kTC, a.cols - c0);
  if (rows_valid == kTR && cols_valid == kTC)
    norm_col_tile<F, NORM, true>(a, l, r0, c0, kTR, kTR, kTC);
  else
    norm_col_tile<F, NORM, false>(a, l, r0, c0, rows_valid, rows_pad, cols_valid);
}

// ---------------------------------------------------------------- launch

// Calls f with std::integral_constant-like tags: the waves of a row and the
// chunks of a lane. Rows of up to 512 values fit one wave; longer ones are
// spread over 4 waves.
template <int W, int N>
struct RowShape {
  static constexpr int waves = W, chunks = N;
};

template <class F>
static void with_row_shape(int64_t cols, F f) {
  if (cols <= 512) f(RowShape<1, 1>{});
  else if (cols <= 2048) f(RowShape<4, 1>{});
  else if (cols <= 4096) f(RowShape<4, 2>{});
  else if (cols <= 6144) f(RowShape<4, 3>{});
  else if (cols <= 8192) f(RowShape<4, 4>{});
  else f(RowShape<4, 8>{});
}

template <bool NORM>
static void launch_col(const NormColArgs& c, hipStream_t s) {
  const dim3 grid((unsigned)((c.cols + kTC - 1) / kTC), (unsigned)((c.rows_pad + kTR - 1) / kTR));
  with_fmt(c.rceil, c.k128, [&](auto f) {
    hipLaunchKernelGGL((k_norm_col<decltype(f), NORM>), grid, dim3(kTileThreads), 0, s, c);
  });
}

hipError_t launch_norm_fwd(const NormFwdArgs& a, hipStream_t s) {
  with_row_shape(a.cols, [&](auto sh) {
    constexpr int kRows = 4 / decltype(sh)::waves;
    hipLaunchKernelGGL((k_norm_row<decltype(sh)::waves, decltype(sh)::chunks>),
                       dim3((unsigned)((a.rows + kRows - 1) / kRows)), dim3(256), 0, s, a);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.q_col) return e;
  launch_col<true>(NormColArgs{a.r ? a.sum : a.x, a.r ? a.cols : a.ld_x, a.rows, a.rows_pad, a.cols, a.rstd, a.w,
                               a.rceil, a.k128, a.q_col, a.s_col}, s);
  return hipGetLastError();
}

int64_t norm_bwd_work(int64_t rows, int64_t cols) { return dw_parts(rows) * cols; }

hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t s) {
  const int64_t parts = dw_parts(a.rows);
  if (parts > 0) {
    with_row_shape(a.cols, [&](auto sh) {
      constexpr int W = decltype(sh)::waves, N = decltype(sh)::chunks, kParts = 4 / W;
      const dim3 grid((unsigned)((parts + kParts - 1) / kParts));
      if (a.q_ck) hipLaunchKernelGGL((k_norm_bwd<W, N, true>), grid, dim3(256), 0, s, a);
      else hipLaunchKernelGGL((k_norm_bwd<W, N, false>), grid, dim3(256), 0, s, a);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(k_norm_dw, dim3((unsigned)(a.cols / 32)), dim3(1024), 0, s, a.work, parts, a.cols, a.dw);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.q_col || parts == 0) return e;
  launch_col<false>(NormColArgs{a.dx, a.cols, a.rows, a.rows_pad, a.cols, nullptr, nullptr, a.rceil, a.k128, a.q_col,
                                a.s_col}, s);
  return hipGetLastError();
}

}  // namespace mxk
