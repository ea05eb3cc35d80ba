// Residual addition + RMS norm + MX quantization, and its gradient:
//   k_norm_row    s = x + r, rstd, row-wise codes of y and of s (checkpoint)
//   k_norm_bwd    dx, its row-wise codes, partial sums of dw
//   k_norm_tail   column-wise codes of y (recomputed from s and rstd) or of
//                 dx, and the join of dw's partial sums
//
// Row-wise work needs the whole row's statistic before its first output, and
// column-wise blocks span 32 rows, so the two directions are two launches:
// the row kernels hold whole rows in registers (mx_row.h), the tail reads s or
// dx back in 128 x 128 tiles (mx_fmt.h), in reverse order, the rows written
// last first: they are the ones still in the Infinity Cache. What only the
// backward pass reads (the forward's checkpoint and column-wise codes) is
// stored non-temporally: k_norm_row 16384 x 5120 129 -> 122 us, the tail 39 -> 42.

#include "mx_device.h"
#include "mx_fmt.h"
#include "mx_lm.h"
#include "mx_row.h"
#include "mx_tile.h"

#include <algorithm>

namespace mxk {

// A row belongs to `waves` waves of a workgroup, each thread holding NCH
// chunks of it; a workgroup has `groups` such rows at a time.
struct RowShape {
  int waves, groups, nch;
};

__host__ __device__ inline int row_groups(int waves) { return waves >= 4 ? 1 : 4 / waves; }

static RowShape row_shape(int64_t cols, int nch) {
  const int waves = (int)((cols + 512 * nch - 1) / (512 * nch));
  return RowShape{waves, row_groups(waves), nch};
}

// Where this thread works: its group's index in the grid, its place in the row.
struct RowPlace {
  int64_t group;
  uint32_t lane, threads;   // thread within the group, threads of the group
  int first_wave;
};

__device__ __forceinline__ RowPlace row_place(int waves, uint32_t units, bool bands) {
  const uint32_t groups = row_groups(waves);
  const uint32_t block = bands ? band_id(blockIdx.x, (units + groups - 1) / groups, false) : blockIdx.x;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = w / waves;
  return RowPlace{(int64_t)block * groups + g, (uint32_t)(threadIdx.x - 64 * g * waves), (uint32_t)(64 * waves),
                  g * waves};
}

// Sum over the waves of this thread's group; every thread of the workgroup
// calls it. `buf`: one value per wave, free again at the next barrier.
template <class T>
__device__ __forceinline__ T group_sum(T v, const RowPlace& p, int waves, T* buf) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
  if (waves > 1) {
    if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
    __syncthreads();
    v = buf[p.first_wave];
    for (int i = 1; i < waves; ++i) v += buf[p.first_wave + i];
  }
  return v;
}

struct NormRowPack {
  const uint16_t *x, *r;
  const float* w;
  uint16_t* sum;
  float* rstd;
  uint8_t *q_row, *s_row, *q_ck, *s_ck;
  int32_t ld_x, ld_r, rows, cols;
  float eps;
  int16_t waves, bands;

  __device__ NormFwdArgs wide() const {
    NormFwdArgs a{};
    a.x = x; a.r = r; a.w = w; a.ld_x = ld_x; a.ld_r = ld_r; a.rows = rows; a.cols = cols; a.eps = eps;
    a.sum = sum; a.rstd = rstd; a.q_row = q_row; a.s_row = s_row; a.q_ck = q_ck; a.s_ck = s_ck;
    return a;
  }
};
static_assert(sizeof(NormRowPack) <= kArgBytes);

// Rows whose s (or dx) fits the XCDs' L2s (4 MB each) go in bands (band_id),
// in the row kernels and in the tail, which then finds them in its own L2 (and
// the scale dwords of neighbouring rows meet in one): 2000 x 2048 forward 15.7 ->
// 13.7 us, 4096 x 1024 backward 21.9 -> 20.7. Larger ones keep the plain order
// (4096 x 7168 forward 62.7 against 64.6).
static bool in_l2(int64_t rows, int64_t cols) { return rows * cols <= (8ll << 20); }

template <class F, int NCH>
__global__ __launch_bounds__(1024) void k_norm_row(NormRowPack pack) {
  __shared__ double buf[16];
  const NormFwdArgs a = pack.wide();
  const int waves = pack.waves;
  const RowPlace p = row_place(waves, pack.rows, pack.bands);
  const int64_t row = p.group;
  const bool live = row < a.rows;
  uint4 v[NCH];
  float w[NCH][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const uint32_t col = 8 * (p.lane + p.threads * i);
    const bool ok = live && col < a.cols;
    v[i] = ok ? load_stream16(a.x + row * a.ld_x + col) : make_uint4(0, 0, 0, 0);
    const uint4 u = ok && a.r ? load_stream16(a.r + row * a.ld_r + col) : make_uint4(0, 0, 0, 0);
    if (ok) load8f(a.w + col, w[i]);
    float f[8];
    unpack8(v[i], f);
    if (a.r) {
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
  // Each thread's sum of at most 16 squares in float32, their join and the
  // root in float64: rstd is then the correctly rounded value but for rare
  // ties. Float32 throughout leaves it an ulp off, which every value of the
  // row shares.
  const double ms = group_sum<double>((double)ss, p, waves, buf) / (double)a.cols + (double)a.eps;
  double rs = (double)(1.0f / sqrtf((float)ms));
  if (rs > 0.0 && ms > 0.0 && rs < INFINITY) rs = fma(0.5 * rs, fma(-ms * rs, rs, 1.0), rs);   // Newton
  const float rstd = (float)rs;
  if (live && p.lane == 0) a.rstd[row] = rstd;
  const TileOut orow{a.q_row, a.s_row, a.cols, a.rows, F::k128};
  const TileOut ock{a.q_ck, a.s_ck, a.cols, a.rows, F::k128};
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const uint32_t col = 8 * (p.lane + p.threads * i);
    const bool ok = live && col < a.cols;
    if (a.q_ck) fmt_chunk<F, true>(v[i], ok, ock, row, col);
    fmt_chunk<F, false>(ok ? norm_chunk(v[i], rstd, w[i]) : make_uint4(0, 0, 0, 0), ok, orow, row, col);
  }
}

// The forward holds little per chunk and takes 2 of them a thread: 16384 x
// 5120 in 171 us against 179 with one and 173 with three.
//
// The backward holds 8 sums of dw and two rows in flight per chunk: one a
// thread while a row fits 16 waves.
static RowShape bwd_shape(int64_t cols) { return row_shape(cols, cols <= 8192 ? 1 : 2); }

// Rows per partial sum of dw: one partial sum a group, 16 rows at most, fewer
// where that would leave less than 4096 waves (16 a CU) to hide the latency of
// memory; each partial sum costs a row of float32 written and read.
static int64_t part_rows(int64_t rows, int64_t cols) {
  const int64_t r = (rows * bwd_shape(cols).waves + 4095) / 4096;
  return std::min<int64_t>(std::max<int64_t>(r, 1), 16);
}

static int64_t dw_parts(int64_t rows, int64_t cols) {
  const int64_t r = part_rows(rows, cols);
  return (rows + r - 1) / r;
}

struct NormBwdPack {
  const uint16_t* dy;
  const void* x;             // x, or the checkpoint's codes
  const uint8_t* s_ck;
  const uint16_t* dsum;
  const float *w, *rstd;
  uint16_t* dx;
  uint8_t *q_row, *s_row;
  float* work;
  int32_t ld_dy, ld_x, ld_dsum, rows, cols;
  int16_t waves, per;        // waves and rows of a group
  int32_t bands;

  template <bool CK>
  __device__ NormBwdArgs wide() const {
    NormBwdArgs a{};
    a.dy = dy; a.dsum = dsum; a.w = w; a.rstd = rstd; a.dx = dx; a.q_row = q_row; a.s_row = s_row; a.work = work;
    if constexpr (CK) { a.q_ck = static_cast<const uint8_t*>(x); a.s_ck = s_ck; }
    else { a.x = static_cast<const uint16_t*>(x); a.ld_x = ld_x; }
    a.ld_dy = ld_dy; a.ld_dsum = ld_dsum; a.rows = rows; a.cols = cols;
    return a;
  }
};
static_assert(sizeof(NormBwdPack) <= kArgBytes);

// What a thread reads of a row.
template <int NCH, bool CK>
struct BwdRow {
  uint4 dy[NCH], ds[NCH], x[CK ? 1 : NCH];
  uint2 q[CK ? NCH : 1];
  uint32_t sb[CK ? NCH : 1];
  float rstd;
};

template <class F, int NCH, bool CK>
__device__ __forceinline__ void bwd_load(BwdRow<NCH, CK>& b, const NormBwdArgs& a, const RowPlace& p, int64_t row) {
  const bool live = row < a.rows;
  b.rstd = live ? a.rstd[row] : 0.0f;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const uint32_t col = 8 * (p.lane + p.threads * i);
    const bool ok = live && col < a.cols;
    b.dy[i] = ok ? load_stream16(a.dy + row * a.ld_dy + col) : make_uint4(0, 0, 0, 0);
    b.ds[i] = ok && a.dsum ? load_stream16(a.dsum + row * a.ld_dsum + col) : make_uint4(0, 0, 0, 0);
    if constexpr (CK) {
      b.q[i] = make_uint2(0, 0);
      b.sb[i] = 0;
      if (ok) {
        b.q[i] = *reinterpret_cast<const uint2*>(a.q_ck + row * a.cols + col);
        b.sb[i] = F::k128 ? a.s_ck[((int64_t)(col >> 7) * a.rows + row) * 4 + ((col >> 5) & 3)]
                          : a.s_ck[row * (a.cols / kBlock) + (col >> 5)];
      }
    } else {
      b.x[i] = ok ? load_stream16(a.x + row * a.ld_x + col) : make_uint4(0, 0, 0, 0);
    }
  }
}

// A group takes `rows` consecutive rows, the next one's loads in flight while
// it works on one (with one chunk a thread; two would spill); dw's sums over
// them stay in registers.
template <class F, int NCH, bool CK>
__global__ __launch_bounds__(1024) void k_norm_bwd(NormBwdPack pack) {
  __shared__ float buf[2][16];
  const NormBwdArgs a = pack.wide<CK>();
  const int waves = pack.waves, rows = pack.per;
  const RowPlace p = row_place(waves, (uint32_t)(pack.rows + rows - 1) / rows, pack.bands);
  const int64_t row0 = p.group * rows;
  float dw[NCH][8] = {}, w[NCH][8] = {};
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const uint32_t col = 8 * (p.lane + p.threads * i);
    if (col < a.cols) load8f(a.w + col, w[i]);
  }
  const float inv_n = 1.0f / (float)a.cols;
  const TileOut orow{a.q_row, a.s_row, a.cols, a.rows, F::k128};
  BwdRow<NCH, CK> cur, nxt;
  bwd_load<F>(cur, a, p, row0);
  for (int rr = 0; rr < rows; ++rr) {
    const int64_t row = row0 + rr;
    const bool live = row < a.rows;
    if (NCH == 1 && rr + 1 < rows) bwd_load<F>(nxt, a, p, row + 1);
    float xh[NCH][8], g[NCH][8];
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      float d[8];
      if constexpr (CK) e4m3_chunk_values(cur.q[i], cur.sb[i], xh[i]);
      else unpack8(cur.x[i], xh[i]);
      unpack8(cur.dy[i], d);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        xh[i][k] *= cur.rstd;
        g[i][k] = d[k] * w[i][k];
        c = fmaf(g[i][k], xh[i][k], c);
        dw[i][k] = fmaf(d[k], xh[i][k], dw[i][k]);
      }
    }
    c = group_sum<float>(c, p, waves, buf[rr & 1]) * inv_n;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const uint32_t col = 8 * (p.lane + p.threads * i);
      const bool ok = live && col < a.cols;
      float e[8];
      unpack8(cur.ds[i], e);
#pragma unroll
      for (int k = 0; k < 8; ++k) e[k] = fmaf(fmaf(-xh[i][k], c, g[i][k]), cur.rstd, e[k]);
      const uint4 v = pack8(e);
      if (ok) *reinterpret_cast<uint4*>(a.dx + row * a.cols + col) = v;
      if (a.q_row) fmt_chunk<F, false>(v, ok, orow, row, col);
    }
    if (NCH == 1) cur = nxt;
    else if (rr + 1 < rows) bwd_load<F>(cur, a, p, row + 1);
  }
  if (row0 < a.rows) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const uint32_t col = 8 * (p.lane + p.threads * i);
      if (col < a.cols) {
        float4* out = reinterpret_cast<float4*>(a.work + p.group * a.cols + col);
        out[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
        out[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
      }
    }
  }
}

struct NormTailArgs {
  const uint16_t* x;         // s or dx
  int64_t ld, rows, rows_pad, cols;
  const float *rstd, *w;     // forward
  uint8_t *q, *s;            // NULL: no column-wise codes
  int32_t dw_blocks, tiles;  // workgroups that join dw, and the tiles' behind them
  const float* work;
  int64_t parts;
  float* dw;
  int32_t bands;
};
static_assert(sizeof(NormTailArgs) <= kArgBytes);

template <class F, bool NORM, bool FULL>
__device__ __forceinline__ void norm_col_tile(const NormTailArgs& a, TileLds& l, int64_t r0, int64_t c0, int rows_valid,
                                              int rows_pad, int cols_valid) {
  uint4 v[kChunks];
  fmt_load<FULL>(v, a.x + r0 * a.ld + c0, a.ld, rows_valid, cols_valid);
  const int t = threadIdx.x, cc = t & 15;
  if constexpr (NORM) {
    float w[8] = {};
    if (FULL || cc * 8 < cols_valid) load8f(a.w + c0 + cc * 8, w);
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int row = (t >> 4) + kRowStep * j;
      // rows past the last stay +0 whatever w holds
      if (FULL || row < rows_valid) v[j] = norm_chunk(v[j], a.rstd[r0 + row], w);
    }
  }
  fmt_to_lds(v, l);
  __syncthreads();
  const TileOut o{a.q, a.s, a.rows_pad, a.cols, F::k128};
  fmt_colq<F, FULL, NORM>(l, rows_pad, cols_valid, o, r0, c0);
  __syncthreads();
  if (t < kTC) fmt_scales<F>(l.s_col, t, cols_valid, rows_pad, o, c0, r0);
}

// dw[c] = sum over the parts of work[part, c]: 32 columns per workgroup, 64
// threads down each group of 4, joined in LDS in a fixed order.
__device__ __forceinline__ void join_dw(const NormTailArgs& a, float4* acc) {
  const int c = threadIdx.x & 7, p0 = threadIdx.x >> 3;
  const float4* src = reinterpret_cast<const float4*>(a.work + (int64_t)blockIdx.x * 32) + c;
  const int64_t ld = a.cols / 4;
  auto add = [](float4 u, float4 v) { return make_float4(u.x + v.x, u.y + v.y, u.z + v.z, u.w + v.w); };
  float4 s0 = make_float4(0, 0, 0, 0), s1 = s0, s2 = s0, s3 = s0;
  int64_t p = p0;
  for (; p + 192 < a.parts; p += 256) {
    s0 = add(s0, src[p * ld]);
    s1 = add(s1, src[(p + 64) * ld]);
    s2 = add(s2, src[(p + 128) * ld]);
    s3 = add(s3, src[(p + 192) * ld]);
  }
  for (; p < a.parts; p += 64) s0 = add(s0, src[p * ld]);
  acc[threadIdx.x] = add(add(s0, s1), add(s2, s3));
  __syncthreads();
  if (p0 == 0) {
    float4 t = make_float4(0, 0, 0, 0);
    for (int i = 0; i < 64; ++i) t = add(t, acc[8 * i + c]);
    reinterpret_cast<float4*>(a.dw + (int64_t)blockIdx.x * 32)[c] = t;
  }
}

template <class F, bool NORM>
__global__ __launch_bounds__(kFmtThreads) void k_norm_tail(NormTailArgs a) {
  __shared__ TileLds l;
  if ((int)blockIdx.x < a.dw_blocks) {
    if ((int64_t)blockIdx.x * 32 >= a.cols) return;
    join_dw(a, reinterpret_cast<float4*>(l.v));
    return;
  }
  // the rows written last first: of the whole, or of each band
  const uint32_t id = blockIdx.x - a.dw_blocks;
  const uint32_t b = a.bands ? band_id(id, a.tiles, true) : a.tiles - 1 - id;
  const uint32_t per_row = (uint32_t)((a.cols + kTC - 1) / kTC);
  const int64_t r0 = (int64_t)(b / per_row) * kTR;
  const int64_t c0 = (int64_t)(b % per_row) * kTC;
  const int rows_valid = (int)min<int64_t>(kTR, a.rows - r0);
  const int rows_pad = (int)min<int64_t>(kTR, a.rows_pad - r0);
  const int cols_valid = (int)min<int64_t>(kTC, a.cols - c0);
  if (rows_valid == kTR && cols_valid == kTC)
    norm_col_tile<F, NORM, true>(a, l, r0, c0, kTR, kTR, kTC);
  else
    norm_col_tile<F, NORM, false>(a, l, r0, c0, rows_valid, rows_pad, cols_valid);
}

// ---------------------------------------------------------------- launch

template <bool NORM>
static hipError_t launch_tail(NormTailArgs c, bool rceil, bool k128, hipStream_t s) {
  c.bands = in_l2(c.rows, c.cols);
  c.dw_blocks = (c.dw_blocks + (c.bands ? 7 : 0)) & (c.bands ? ~7 : ~0);   // keeps the tiles' XCDs
  c.tiles = c.q ? (int32_t)((c.cols + kTC - 1) / kTC * ((c.rows_pad + kTR - 1) / kTR)) : 0;
  const dim3 grid((unsigned)(c.dw_blocks + c.tiles));
  with_fmt(rceil, k128, [&](auto f) {
    hipLaunchKernelGGL((k_norm_tail<decltype(f), NORM>), grid, dim3(kFmtThreads), 0, s, c);
  });
  return hipGetLastError();
}

hipError_t launch_norm_fwd(const NormFwdArgs& a, hipStream_t s) {
  const RowShape sh = row_shape(a.cols, a.cols <= 512 ? 1 : 2);
  const dim3 grid((unsigned)((a.rows + sh.groups - 1) / sh.groups)), block(64 * sh.waves * sh.groups);
  const NormRowPack p{a.x, a.r, a.w, a.sum, a.rstd, a.q_row, a.s_row, a.q_ck, a.s_ck, (int32_t)a.ld_x, (int32_t)a.ld_r,
                      (int32_t)a.rows, (int32_t)a.cols, a.eps, (int16_t)sh.waves, (int16_t)in_l2(a.rows, a.cols)};
  with_fmt(a.rceil, a.k128, [&](auto f) {
    using F = decltype(f);
    if (sh.nch == 1) hipLaunchKernelGGL((k_norm_row<F, 1>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((k_norm_row<F, 2>), grid, block, 0, s, p);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.q_col) return e;
  NormTailArgs c{};
  c.x = a.r ? a.sum : a.x;
  c.ld = a.r ? a.cols : a.ld_x;
  c.rows = a.rows; c.rows_pad = a.rows_pad; c.cols = a.cols;
  c.rstd = a.rstd; c.w = a.w; c.q = a.q_col; c.s = a.s_col;
  return launch_tail<true>(c, a.rceil, a.k128, s);
}

int64_t norm_bwd_work(int64_t rows, int64_t cols) { return dw_parts(rows, cols) * cols; }

hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t s) {
  const RowShape sh = bwd_shape(a.cols);
  const int64_t parts = a.rows ? dw_parts(a.rows, a.cols) : 0;
  if (parts > 0) {
    const int per = (int)part_rows(a.rows, a.cols);
    const dim3 grid((unsigned)((parts + sh.groups - 1) / sh.groups)), block(64 * sh.waves * sh.groups);
    const NormBwdPack p{a.dy, a.q_ck ? (const void*)a.q_ck : a.x, a.s_ck, a.dsum, a.w, a.rstd, a.dx, a.q_row, a.s_row,
                        a.work, (int32_t)a.ld_dy, (int32_t)a.ld_x, (int32_t)a.ld_dsum, (int32_t)a.rows, (int32_t)a.cols,
                        (int16_t)sh.waves, (int16_t)per, in_l2(a.rows, a.cols)};
    with_fmt(a.rceil, a.k128, [&](auto f) {
      using F = decltype(f);
      if (sh.nch == 1) {
        if (a.q_ck) hipLaunchKernelGGL((k_norm_bwd<F, 1, true>), grid, block, 0, s, p);
        else hipLaunchKernelGGL((k_norm_bwd<F, 1, false>), grid, block, 0, s, p);
      } else {
        if (a.q_ck) hipLaunchKernelGGL((k_norm_bwd<F, 2, true>), grid, block, 0, s, p);
        else hipLaunchKernelGGL((k_norm_bwd<F, 2, false>), grid, block, 0, s, p);
      }
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  NormTailArgs c{};
  c.x = a.dx;
  c.ld = a.cols;
  c.rows = a.rows; c.rows_pad = a.rows_pad; c.cols = a.cols;
  c.q = parts ? a.q_col : nullptr; c.s = a.s_col;
  c.dw_blocks = (int32_t)(a.cols / 32);
  c.work = a.work; c.parts = parts; c.dw = a.dw;
  return launch_tail<false>(c, a.rceil, a.k128, s);
}

}  // namespace mxk
