// SwiGLU between two MXFP8 GEMMs with its input kept for the backward in
// 8 bits, for any number of rows:
//   k_swiglu_ck_fwd   h = silu(a) b quantized both ways, [a | b] quantized
//                     along its rows (the checkpoint)
//   k_swiglu_ck_bwd   a, b from the checkpoint; [dA | dB] quantized both ways
//
// One 128 x 128 tile of h per workgroup in the tile scheme of mx_tile.h: each
// input is read once into registers, everything else happens on chip. Rows
// past the last one enter as zeros, so the column-wise blocks that they fill
// up quantize to zeros.

#include "mx_device.h"
#include "mx_lm.h"
#include "mx_row.h"
#include "mx_tile.h"

namespace mxk {

__global__ __launch_bounds__(kTileThreads) void k_swiglu_ck_fwd(SwigluCkArgs a) {
  __shared__ uint4 lds[kTR * kTC / 8];
  const int64_t r0 = (int64_t)blockIdx.y * kTR;
  const int64_t c0 = (int64_t)blockIdx.x * kTC;
  const int rows_valid = (int)min<int64_t>(kTR, a.rows - r0);
  const int rows_pad = (int)min<int64_t>(kTR, a.rows_pad - r0);
  const int cols_valid = (int)min<int64_t>(kTC, a.hidden - c0);
  uint4 v[kTileChunks], w[kTileChunks];
  tile_load<true>(v, a.a + r0 * a.ld_ab + c0, a.ld_ab, rows_valid, cols_valid);
  tile_load<true>(w, a.b + r0 * a.ld_ab + c0, a.ld_ab, rows_valid, cols_valid);
  const TileOut ock{a.q_ck, a.s_ck, 2 * a.hidden, a.rows, a.k128};
  tile_rowq(v, rows_valid, cols_valid, a.rceil, ock, r0, c0);
  tile_rowq(w, rows_valid, cols_valid, a.rceil, ock, r0, a.hidden + c0);
#pragma unroll
  for (int j = 0; j < kTileChunks; ++j)
    v[j] = make_uint4(swiglu_pair(v[j].x, w[j].x), swiglu_pair(v[j].y, w[j].y),
                      swiglu_pair(v[j].z, w[j].z), swiglu_pair(v[j].w, w[j].w));
  tile_rowq(v, rows_valid, cols_valid, a.rceil, TileOut{a.q_row, a.s_row, a.hidden, a.rows, a.k128}, r0, c0);
  tile_to_lds(v, lds);
  __syncthreads();
  tile_colq(lds, rows_pad, cols_valid, a.rceil, TileOut{a.q_col, a.s_col, a.rows_pad, a.hidden, a.k128}, r0, c0);
}

// Codes and scale bytes of the thread's chunks of a tile whose (0,0) is row
// r0, column c0 of the checkpoint [rows, ld]. Chunks outside the valid region
// read its last row or column in their place (loads without a branch: with
// one, the compiler carried the widened float32 values of all chunks through
// it, 256 VGPRs); the caller drops what comes of them.
__device__ __forceinline__ void tile_load_codes(uint2 (&q)[kTileChunks], uint32_t (&sb)[kTileChunks], const uint8_t* qp,
                                                const uint8_t* sp, int64_t ld, int64_t rows, bool k128, int64_t r0,
                                                int64_t c0, int rows_valid, int cols_valid) {
  const int t = threadIdx.x;
  const int64_t c = c0 + min((t & 15) * 8, cols_valid - 8);
#pragma unroll
  for (int j = 0; j < kTileChunks; ++j) {
    const int64_t r = r0 + min((t >> 4) + 16 * j, rows_valid - 1);
    q[j] = *reinterpret_cast<const uint2*>(qp + r * ld + c);
    sb[j] = sp[k128 ? ((c >> 7) * rows + r) * 4 + ((c >> 5) & 3) : r * (ld / kBlock) + (c >> 5)];
  }
}

__global__ __launch_bounds__(kTileThreads, 4) void k_swiglu_ck_bwd(SwigluCkArgs a) {
  __shared__ uint4 lds[kTR * kTC / 8];
  const int64_t r0 = (int64_t)blockIdx.y * kTR;
  const int64_t c0 = (int64_t)blockIdx.x * kTC;
  const int rows_valid = (int)min<int64_t>(kTR, a.rows - r0);
  const int rows_pad = (int)min<int64_t>(kTR, a.rows_pad - r0);
  const int cols_valid = (int)min<int64_t>(kTC, a.hidden - c0);
  const int64_t H2 = 2 * a.hidden;
  uint4 da[kTileChunks], db[kTileChunks];
  {
    uint2 qa[kTileChunks], qb[kTileChunks];
    uint32_t sa[kTileChunks], sb[kTileChunks];
    tile_load<true>(da, a.dh + r0 * a.ld_dh + c0, a.ld_dh, rows_valid, cols_valid);
    tile_load_codes(qa, sa, a.q_ck, a.s_ck, H2, a.rows, a.k128, r0, c0, rows_valid, cols_valid);
    tile_load_codes(qb, sb, a.q_ck, a.s_ck, H2, a.rows, a.k128, r0, a.hidden + c0, rows_valid, cols_valid);
#pragma unroll
    for (int j = 0; j < kTileChunks; ++j) {
      float fa[8], fb[8], ga[8], gb[8];
      e4m3_chunk_values(qa[j], sa[j], fa);
      e4m3_chunk_values(qb[j], sb[j], fb);
      const uint32_t wd[4] = {da[j].x, da[j].y, da[j].z, da[j].w};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        swiglu_grad_f32(i & 1 ? bf16_hi(wd[i >> 1]) : bf16_lo(wd[i >> 1]), fa[i], fb[i], ga[i], gb[i]);
      const bool ok = (int)(threadIdx.x >> 4) + 16 * j < rows_valid && (int)(threadIdx.x & 15) * 8 < cols_valid;
      da[j] = ok ? pack8(ga) : make_uint4(0, 0, 0, 0);
      db[j] = ok ? pack8(gb) : make_uint4(0, 0, 0, 0);
      // one chunk's 32 float32 values at a time: left to itself the scheduler
      // widens all eight chunks first (256 VGPRs, 1 wave per SIMD)
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  const TileOut orow{a.q_row, a.s_row, H2, a.rows, a.k128};
  tile_rowq(da, rows_valid, cols_valid, a.rceil, orow, r0, c0);
  tile_rowq(db, rows_valid, cols_valid, a.rceil, orow, r0, a.hidden + c0);
  const TileOut ocol{a.q_col, a.s_col, a.rows_pad, H2, a.k128};
  tile_to_lds(da, lds);
  __syncthreads();
  tile_colq(lds, rows_pad, cols_valid, a.rceil, ocol, r0, c0);
  __syncthreads();
  tile_to_lds(db, lds);
  __syncthreads();
  tile_colq(lds, rows_pad, cols_valid, a.rceil, ocol, r0, a.hidden + c0);
}

static dim3 tile_grid(const SwigluCkArgs& a) {
  return dim3((unsigned)((a.hidden + kTC - 1) / kTC), (unsigned)((a.rows_pad + kTR - 1) / kTR));
}

hipError_t launch_swiglu_ck_fwd(const SwigluCkArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_swiglu_ck_fwd, tile_grid(a), dim3(kTileThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_swiglu_ck_bwd(const SwigluCkArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_swiglu_ck_bwd, tile_grid(a), dim3(kTileThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace mxk
