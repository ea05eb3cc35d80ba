// Log probabilities of given tokens, with entropy and top alternatives, and
// the gradient of the logits as an MX operand:
//   k_logprob_fwd   one workgroup per row
//   k_logprob_bwd   one 128 x 128 tile per workgroup (mx_tile.h)
//
// In base 2: with c = scale log2(e) and d_j = (x_j - m) c, the row's sums are
// S = sum 2^d_j and A = sum 2^d_j d_j, kept relative to a running maximum m
// (a new maximum m' multiplies S by f = 2^((m - m') c) and turns A into
// f (A + S (m - m') c)); then ls = ln S, entropy = ln S - ln2 A / S. Nothing
// overflows and a masked entry (-infinity) adds exactly 0.
//
// Rows may start at any element (an odd vocabulary), so chunks are read with
// 16-byte loads of 2- or 4-byte alignment and the last one of a row element
// by element.

#include "mx_device.h"
#include "mx_fmt.h"
#include "mx_lm.h"
#include "mx_row.h"
#include "mx_tile.h"

#include <algorithm>
#include <cmath>

namespace mxk {

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;

// 8 logits starting at element `i` of a row of n; `fill` past the end.
template <bool F32>
__device__ __forceinline__ void load_logits(const void* row, int64_t i, int64_t n, float fill, float (&f)[8]) {
  if constexpr (F32) {
    const float* p = static_cast<const float*>(row) + i;
    if (i + 8 <= n) {
      __builtin_memcpy(f, p, 32);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = i + k < n ? p[k] : fill;
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(row) + i;
    if (i + 8 <= n) {
      uint4 v;
      __builtin_memcpy(&v, p, 16);
      unpack8(v, f);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = i + k < n ? __uint_as_float((uint32_t)p[k] << 16) : fill;
    }
  }
}

template <bool F32>
__device__ __forceinline__ const void* logits_row(const LogprobArgs& a, int64_t row) {
  return static_cast<const char*>(a.x) + row * a.ld * (F32 ? 4 : 2);
}

// The row's target, or -1 if it is not scored.
__device__ __forceinline__ int64_t row_target(const LogprobArgs& a, int64_t row) {
  const int64_t t = a.targets[row];
  return t == a.ignore_index || t < 0 || t >= a.vocab ? -1 : t;
}

// Order of the alternatives as one number: larger for a larger value, then
// for a lower index (the sign of zero does not count).
__device__ __forceinline__ uint64_t top_key(float x, uint32_t idx) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  const uint32_t o = u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
  return ((uint64_t)o << 32) | (0xFFFFFFFFu - idx);
}

__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ uint32_t key_index(uint64_t key) { return 0xFFFFFFFFu - (uint32_t)key; }

// m, S, A of a set of logits (see the top of the file); m = -infinity, S = A
// = 0 for the empty set.
struct Soft {
  float m, s, a;
};

__device__ __forceinline__ Soft soft_rebase(Soft v, float m, float c) {
  if (v.m == m || v.m == -INFINITY) {
    v.m = m;
    return v;
  }
  const float d = (v.m - m) * c;
  const float f = __builtin_amdgcn_exp2f(d);
  return Soft{m, v.s * f, (v.a + v.s * fmaxf(d, -1e4f)) * f};
}

__device__ __forceinline__ Soft soft_join(Soft u, Soft v, float c) {
  const float m = fmaxf(u.m, v.m);
  u = soft_rebase(u, m, c);
  v = soft_rebase(v, m, c);
  return Soft{m, u.s + v.s, u.a + v.a};
}

template <bool F32>
__global__ __launch_bounds__(256) void k_logprob_fwd(LogprobArgs a) {
  __shared__ Soft part[4];
  __shared__ uint64_t best[4];
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x;
  const void* x = logits_row<F32>(a, row);
  const float c = a.scale * kLog2e;
  Soft v{-INFINITY, 0.0f, 0.0f};
  for (int64_t i = 8 * (int64_t)t; i < a.vocab; i += 8 * 256) {
    float f[8];
    load_logits<F32>(x, i, a.vocab, -INFINITY, f);
    float m = v.m;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, f[k]);
    v = soft_rebase(v, m, c);
    const float base = m == -INFINITY ? 0.0f : m;   // -inf - 0 keeps e = 0
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = (f[k] - base) * c;
      const float e = __builtin_amdgcn_exp2f(d);
      v.s += e;
      v.a = fmaf(e, fmaxf(d, -1e4f), v.a);
    }
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1)
    v = soft_join(v, Soft{__shfl_xor(v.m, o), __shfl_xor(v.s, o), __shfl_xor(v.a, o)}, c);
  if ((t & 63) == 0) part[t >> 6] = v;
  __syncthreads();
  v = part[0];
  for (int i = 1; i < 4; ++i) v = soft_join(v, part[i], c);
  const bool empty = v.m == -INFINITY && v.s == 0.0f;
  const float ls = empty ? -INFINITY : logf(v.s);
  if (t == 0) {
    const int64_t tg = row_target(a, row);
    if (a.dev_err && tg < 0 && a.targets[row] != a.ignore_index) atomicOr(a.dev_err, 8);
    float xt = 0.0f;
    if (tg >= 0)
      xt = F32 ? static_cast<const float*>(x)[tg]
               : __uint_as_float((uint32_t)static_cast<const uint16_t*>(x)[tg] << 16);
    a.logp[row] = tg < 0 ? 0.0f : empty ? -INFINITY : (xt - v.m) * a.scale - ls;
    a.entropy[row] = empty ? 0.0f : ls - kLn2 * (v.a / v.s);
    a.stats_out[2 * row] = v.m;
    a.stats_out[2 * row + 1] = ls;
  }
  uint64_t last = ~0ull;
  for (int j = 0; j < a.top; ++j) {
    uint64_t b = 0;
    for (int64_t i = 8 * (int64_t)t; i < a.vocab; i += 8 * 256) {
      float f[8];
      load_logits<F32>(x, i, a.vocab, -INFINITY, f);
      for (int k = 0; k < 8; ++k) {
        const uint64_t key = top_key(f[k], (uint32_t)(i + k));
        if (i + k < a.vocab && key < last && key > b) b = key;
      }
    }
    for (int o = 32; o >= 1; o >>= 1) b = max(b, (uint64_t)__shfl_xor((unsigned long long)b, o));
    __syncthreads();
    if ((t & 63) == 0) best[t >> 6] = b;
    __syncthreads();
    last = max(max(best[0], best[1]), max(best[2], best[3]));
    if (t == 0) {
      a.top_idx[row * a.top + j] = (int32_t)key_index(last);
      a.top_logp[row * a.top + j] = empty ? -INFINITY : (key_value(last) - v.m) * a.scale - ls;
    }
  }
}

// ---------------------------------------------------------------- backward

// With l_j = (x_j - m) scale - ls, p_j = e^l_j and
//   k1 = -scale dent, k0 = -scale (dlogp + dent entropy), add = scale dlogp
// the gradient is p_j (k1 l_j + k0), plus `add` at the target. l is bounded
// below where it multiplies k1, so that a masked entry gives p = 0 times a
// finite number; a NaN still reaches the result through p.
struct GradRow {
  float m, nls, k1, k0, add;
  int32_t target;   // column within the tile, out of [0, 128) if elsewhere
};

// Raw logits of a thread's chunks.
template <bool F32>
struct RawChunk {
  uint4 w[F32 ? 2 : 1];
};

template <class F, bool F32, bool FULL>
__device__ __forceinline__ void logprob_bwd_tile(const LogprobArgs& a, TileLds& l, GradRow* rows, int64_t r0, int64_t c0,
                                                 int rows_valid, int rows_pad, int cols_valid, int cols_pad) {
  constexpr int kB = F32 ? 4 : 2;
  const uint32_t t = threadIdx.x, cc = t & 15, tr = t >> 4;
  const char* base = static_cast<const char*>(a.x) + (r0 * a.ld + c0) * kB;
  RawChunk<F32> raw[kTileChunks];
#pragma unroll
  for (int j = 0; j < kTileChunks; ++j) {
    if constexpr (FULL) {
      __builtin_memcpy(&raw[j], base + (int64_t)(16 * j) * a.ld * kB + (tr * (uint32_t)a.ld + cc * 8) * kB, sizeof(raw[j]));
    } else {
      float f[8];
      const int row = tr + 16 * j;
      if (row < rows_valid && (int)cc * 8 < cols_valid)
        load_logits<F32>(base + row * a.ld * kB, cc * 8, cols_valid, -INFINITY, f);
      else
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = -INFINITY;
      if constexpr (F32) __builtin_memcpy(&raw[j], f, 32);
      else raw[j].w[0] = pack8(f);
    }
  }
  if ((int)t < kTR) {
    GradRow g{0.0f, 0.0f, 0.0f, 0.0f, 0.0f, -1};
    if (FULL || (int)t < rows_valid) {
      const int64_t row = r0 + t;
      const float m = a.stats[2 * row], ls = a.stats[2 * row + 1];
      const int64_t tg = row_target(a, row);
      if (blockIdx.x == 0 && a.dev_err && tg < 0 && a.targets[row] != a.ignore_index) atomicOr(a.dev_err, 8);
      if (!(m == -INFINITY && ls == -INFINITY)) {   // a row with nothing left has gradient 0
        const float d = tg >= 0 && a.dlogp ? a.dlogp[row] : 0.0f;
        const float dent = a.dent ? a.dent[row] : 0.0f;
        g = GradRow{m, -ls, -a.scale * dent, -a.scale * (a.dent ? fmaf(dent, a.ent_in[row], d) : d), a.scale * d,
                    tg >= c0 && tg < c0 + kTC ? (int32_t)(tg - c0) : -1};
      }
    }
    rows[t] = g;
  }
  __syncthreads();
  uint4 v[kTileChunks];
#pragma unroll
  for (int j = 0; j < kTileChunks; ++j) {
    const GradRow g = rows[tr + 16 * j];
    float f[8];
    if constexpr (F32) __builtin_memcpy(f, &raw[j], 32);
    else unpack8(raw[j].w[0], f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float lp = fmaf(f[k] - g.m, a.scale, g.nls);
      const float p = __builtin_amdgcn_exp2f(lp * kLog2e);
      f[k] = fmaf(p, fmaf(fmaxf(lp, -1e4f), g.k1, g.k0), 0.0f);
    }
    const uint32_t hit = (uint32_t)g.target - cc * 8;
    if (hit < 8) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if ((int)hit == k) f[k] += g.add;
    }
    v[j] = pack8(f);
    if constexpr (!FULL) {   // rows and columns that only fill up: +0
      const int left = (int)(tr + 16 * j) < rows_valid ? cols_valid - (int)cc * 8 : 0;
      uint32_t* w = reinterpret_cast<uint32_t*>(&v[j]);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = left >= 2 * k + 2 ? w[k] : left == 2 * k + 1 ? w[k] & 0xFFFFu : 0u;
    }
  }
  fmt_dual<F, FULL>(v, l, rows_valid, rows_pad, cols_pad, TileOut{a.q_row, a.s_row, a.vocab_pad, a.rows, F::k128},
                    TileOut{a.q_col, a.s_col, a.rows_pad, a.vocab_pad, F::k128}, r0, c0, false);
}

template <class F, bool F32>
__global__ __launch_bounds__(kTileThreads) void k_logprob_bwd(LogprobArgs a) {
  __shared__ TileLds l;
  __shared__ GradRow rows[kTR];
  const int64_t r0 = (int64_t)blockIdx.y * kTR;
  const int64_t c0 = (int64_t)blockIdx.x * kTC;
  const int rows_valid = (int)min<int64_t>(kTR, a.rows - r0);
  const int rows_pad = (int)min<int64_t>(kTR, a.rows_pad - r0);
  const int cols_valid = (int)min<int64_t>(kTC, a.vocab - c0);
  const int cols_pad = (int)min<int64_t>(kTC, a.vocab_pad - c0);
  if (rows_valid == kTR && cols_valid == kTC)
    logprob_bwd_tile<F, F32, true>(a, l, rows, r0, c0, kTR, kTR, kTC, kTC);
  else
    logprob_bwd_tile<F, F32, false>(a, l, rows, r0, c0, rows_valid, rows_pad, cols_valid, cols_pad);
}

// ---------------------------------------------------------------- launch

int64_t logprob_work(int64_t, int64_t, int32_t) { return 0; }

hipError_t launch_logprob_fwd(const LogprobArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.rows);
  if (a.f32) hipLaunchKernelGGL(k_logprob_fwd<true>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(k_logprob_fwd<false>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_logprob_bwd(const LogprobArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.vocab_pad + kTC - 1) / kTC), (unsigned)((a.rows_pad + kTR - 1) / kTR));
  with_fmt(a.rceil, a.k128, [&](auto f) {
    if (a.f32) hipLaunchKernelGGL((k_logprob_bwd<decltype(f), true>), grid, dim3(kTileThreads), 0, s, a);
    else hipLaunchKernelGGL((k_logprob_bwd<decltype(f), false>), grid, dim3(kTileThreads), 0, s, a);
  });
  return hipGetLastError();
}

}  // namespace mxk
