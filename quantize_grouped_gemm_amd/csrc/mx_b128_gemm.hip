// FP8 products with one float32 scale for a block of 128 along the
// contraction:
//   C[m, n] = sum_kb sa[kb, m] * sb[kb, n or n / 128] * sum_k A[m, k] B[n, k]
// (k over the 128 codes of block kb), float32 accumulation, C bf16 or float32.
//
// The scales are no powers of two, so the matrix unit's own block scales do not
// serve. One v_mfma_f32_16x16x128_f8f6f4 sums exactly one block of 128 into four
// zeroed registers, and four fused multiply-adds bring them into the accumulators
// under the block's scale. Per block and output that is one vector instruction
// for weights (their scale is one for 128 columns, so a lane's factor is one
// number) and two for the weight gradient (1 x 128 on both sides). A wave needs
// 32 clocks of the matrix unit and 16 (32) of the vector unit for each; two
// waves a SIMD keep both busy. The accumulators have to be ordinary registers
// (the vector unit cannot write the others), so a wave's tile is 64 x 128: 128
// accumulators of its 256 registers. Alone, a product of the matrix unit takes 15.6 ns,
// beside four fused multiply-adds 17.2, beside eight 22.4.
//
// Large products are bound by power as much as by issue: the clock falls to 2.0 GHz
// while the matrix unit is busy 55% and the vector unit 37% of the time. 65536 rows
// to 32 experts of 4096 x 7168 1824 us (2.1 PFLOP/s), the weight gradient 7168 x 2048
// from as many rows 1103 to 1153 us (1.7; float32 results 1257), 8192 x 8192 x 8192 440 us
// (2.5; with 1 x 128 scales on both sides 524); the products with scales in the matrix
// unit reach 2.2 to 2.7 on this card.
//
// The matrix unit holds groups of 8 products to 2^-13 of the largest, which leaves
// float32 results off by 1.5e-5 of their size (root mean square).
//
// Operand layout (any order of k serves, as long as both sides share it): lane l
// holds row l & 15 of its 16-row block, bytes 16 q .. + 15 and 64 + 16 q .. + 15
// of the row's 128, q = l >> 4. Register c of the result is row 4 q + c, column
// l & 15. B's rows are the result's rows, in an order in which a lane ends with
// 8 consecutive columns of C (see b_row), so that C leaves in 16-byte stores
// straight from the registers.

#include "mx_device.h"
#include "mx_moe.h"

#include <algorithm>

namespace mxk {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr;

__device__ __forceinline__ v4f mfma128(const v8i& a, const v8i& b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, v4f{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ v8i join16(uint4 x, uint4 y) {
  return v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
}

__device__ __forceinline__ int uniform(int v) { return (int)__builtin_amdgcn_readfirstlane((uint32_t)v); }

// A buffer of `bytes` bytes from p on; both are read from lane 0, so that the
// descriptor is in scalar registers also where they come from a group's table.
// Loads past its end give 0.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, int64_t bytes) {
  const uint64_t v = (uint64_t)(uintptr_t)p;
  const uint64_t u = (uint64_t)(uint32_t)uniform((int)(uint32_t)v) | ((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32);
  return __builtin_amdgcn_make_buffer_rsrc((void*)(uintptr_t)u, (short)0, uniform((int)bytes), 0x00020000);
}

// ---------------------------------------------------------------- groups

// Where piece `want` of the groups' rows lies: the groups cut into pieces of
// `unit` rows each (or, unit 0, one piece a group with rows), in order. Every
// wave looks it up by itself, 64 groups at a time. Ends that fall, are negative
// or pass `cap` (or, with align, are no multiples of 128) are reported and moved
// to where they do no harm.
struct Piece {
  int32_t group;      // -1: past the groups' pieces
  int32_t start, end; // the group's rows
  int32_t index;      // piece within the group, or past the groups' pieces
  int32_t last;       // end of the last group
};

// Inclusive prefix over the wave (row shifts, then broadcasts across the rows); values are >= 0.
template <bool MAX>
__device__ __forceinline__ int32_t scan(int32_t v) {
  auto join = [&](int32_t o) { v = MAX ? max(v, o) : v + o; };
  join(__builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false));
  join(__builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false));
  join(__builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false));
  join(__builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false));
  join(__builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false));
  join(__builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false));
  return v;
}

__device__ __forceinline__ int32_t clean_end(int32_t v, int32_t cap, bool align) {
  v = min(max(v, 0), cap);
  return align ? v & ~127 : v;
}

__device__ __forceinline__ Piece find_piece(const int32_t* offs, int E, int32_t cap, int unit, int want, bool align,
                                            int32_t* dev_err) {
  const int lane = threadIdx.x & 63;
  int32_t end_before = 0, pieces_before = 0;
  bool bad = false;
  Piece p{-1, 0, 0, 0, 0};
  int32_t next = lane < E ? offs[lane] : 0;      // the next 64 are on their way meanwhile
  for (int g0 = 0; g0 < E; g0 += 64) {
    const int g = g0 + lane;
    const int32_t raw = next;
    next = g + 64 < E ? offs[g + 64] : 0;
    int32_t end = g < E ? clean_end(raw, cap, align) : 0;
    end = max(scan<true>(end), end_before);
    bad |= g < E && raw != end;
    int32_t start = __shfl_up(end, 1);
    if (lane == 0) start = end_before;
    const int32_t n = unit ? (end - start + unit - 1) / unit : (end > start ? 1 : 0);
    const int32_t incl = scan<false>(n) + pieces_before;
    const uint64_t hit = __ballot(incl > want);
    if (p.group < 0 && hit) {
      const int at = __builtin_ctzll(hit);
      p.group = g0 + at;
      p.start = __builtin_amdgcn_readlane(start, at);
      p.end = __builtin_amdgcn_readlane(end, at);
      p.index = want - __builtin_amdgcn_readlane(incl - n, at);
    }
    end_before = __builtin_amdgcn_readlane(end, 63);
    pieces_before = __builtin_amdgcn_readlane(incl, 63);
  }
  if (p.group < 0) p.index = want - pieces_before;
  p.last = end_before;
  if (dev_err && blockIdx.x == 0 && threadIdx.x < 64 && __any(bad) && lane == 0) atomicOr(dev_err, 1);
  return p;
}

// Rows of one group alone: the `want`-th by size, largest first (up to 64
// groups, ties by index), so that the longest tiles do not start last; the
// want-th itself of more groups.
__device__ __forceinline__ Piece group_rows(const int32_t* offs, int E, int32_t cap, int want, int32_t* dev_err) {
  const int lane = threadIdx.x & 63;
  int32_t end_before = 0;
  bool bad = false;
  int g = want;
  Piece p{g, 0, 0, 0, 0};
  for (int g0 = 0; g0 < E; g0 += 64) {
    const int32_t raw = g0 + lane < E ? offs[g0 + lane] : 0;
    int32_t end = g0 + lane < E ? clean_end(raw, cap, true) : 0;
    end = max(scan<true>(end), end_before);
    bad |= g0 + lane < E && raw != end;
    int32_t start = __shfl_up(end, 1);
    if (lane == 0) start = end_before;
    if (E <= 64) {
      const int32_t size = end - start;
      int rank = 0;
      for (int h = 0; h < E; ++h) {
        const int32_t o = __builtin_amdgcn_readlane(size, h);
        rank += o > size || (o == size && h < lane);
      }
      g = __builtin_ctzll(__ballot(lane < E && rank == want));
      p.group = g;
    }
    if (g >= g0 && g < g0 + 64) {
      p.start = __builtin_amdgcn_readlane(start, g - g0);
      p.end = __builtin_amdgcn_readlane(end, g - g0);
    }
    end_before = __builtin_amdgcn_readlane(end, 63);
  }
  if (dev_err && blockIdx.x == 0 && threadIdx.x < 64 && __any(bad) && lane == 0) atomicOr(dev_err, 1);
  return p;
}

// ---------------------------------------------------------------- tiles

// One tile's operands; every field is the same in all lanes.
struct Tile {
  const uint8_t *a, *b;       // codes of the tile's first rows at the first block
  const float *sa, *sb;       // scales of the first rows (sb: first row, or its block of 128)
  int64_t lda, ldb;           // bytes from row to row
  int64_t na, nb;             // scales from block to block of k
  int64_t sa_left, sb_left;   // scales from sa / sb to the end of their matrices
  int valid_m, valid_n;       // rows of A and B that exist in the tile
  int nk;                     // blocks of k
  void* out;
  int64_t ldo;
};

template <int WM_, int WN_, int TM_, int TN_>
struct Shape {
  static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_;   // waves; 16-row blocks a wave
  static constexpr int BM = WM * TM * 16, BN = WN * TN * 16, waves = WM * WN, threads = waves * 64;
  static constexpr int kA = BM * 128, kB = BN * 128, kS = (BM + BN) * 4, stage = kA + kB + kS;   // kS: scales, where B's rows have their own
  static constexpr int dma_a = BM / 8 / waves, dma_b = BN / 8 / waves;   // 8-row DMA instructions a wave
  static_assert(dma_a % 2 == 0 && dma_b % 4 == 0 && TN % 2 == 0);
};

// Row of B that block i of a wave holds as its row r. For bf16 results (WIDE)
// registers 0..3 of blocks 2 p and 2 p + 1 are columns 32 p + 8 q + 0..3 and + 4..7 of
// C, 16 bytes of bf16; 4 float32 columns are 16 bytes already.
template <bool WIDE>
__device__ __forceinline__ int b_row(int i, int r) {
  return WIDE ? 32 * (i >> 1) + 8 * (r >> 2) + 4 * (i & 1) + (r & 3) : 16 * i + r;
}

// Rows are 128 bytes in LDS; a row's 16-byte piece p sits in slot p ^ f(row). A
// 16-byte read serves 16 lanes, one piece of 16 rows, at a time over 64 banks:
// rows of one parity share a half of them, and f takes 8 values on the 8 even
// and on the 8 odd rows of such a read: consecutive rows, or those of b_row<true>.
__device__ __forceinline__ int fa(int row) { return (row >> 1) & 7; }
template <bool WIDE>
__device__ __forceinline__ int fb(int row) {
  return WIDE ? ((row >> 1) & 1) | (((row >> 3) & 3) << 1) : fa(row);
}

// 64 lanes x BYTES from a buffer to consecutive LDS, written as inline assembly:
// the compiler would let LDS reads of the other stage wait for it. The step loop
// waits for it itself, before the barrier that hands the stage over. M0 is named
// as clobbered.
#pragma clang diagnostic ignored "-Winline-asm"
template <int BYTES>
__device__ __forceinline__ void dma_lds(const __amdgpu_buffer_rsrc_t& r, const uint8_t* dst, uint32_t voff, uint32_t soff) {
  const uint32_t m0 = (uint32_t)(uintptr_t)(lds_ptr) const_cast<uint8_t*>(dst);
  if constexpr (BYTES == 16)
    asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(m0), "v"(voff), "s"(r), "s"(soff)
                 : "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(m0), "v"(voff), "s"(r), "s"(soff)
                 : "m0");
}

template <class S, bool ROWB, bool F32>
struct TileRun {
  __amdgpu_buffer_rsrc_t ra, rb, rsa, rsb;
  uint32_t voff_a[2], voff_b[4];
  uint32_t lda, ldb, na4, nb4;
  int w, wm, wn, lane;
  uint32_t sa_off, sb_off, schunk, soff;

  __device__ __forceinline__ void init(const Tile& t) {
    lane = threadIdx.x & 63;
    w = uniform((int)threadIdx.x >> 6);
    wm = w / S::WN;
    wn = w % S::WN;
    // each resource ends behind the last valid row: what lies past it reads 0
    ra = buffer(t.a, t.valid_m * t.lda);
    rb = buffer(t.b, t.valid_n * t.ldb);
    // row scales of both sides: 64 a wave, A's first (waves without any repeat some)
    constexpr int kChunks64 = (S::BM + S::BN) / 64;
    const bool mine_a = !ROWB || w % kChunks64 < S::BM / 64;
    schunk = ROWB ? w % kChunks64 : 0;
    soff = 256 * (mine_a ? schunk : schunk - S::BM / 64);
    rsa = buffer(mine_a ? t.sa : t.sb, (mine_a ? t.sa_left : t.sb_left) * 4);
    rsb = buffer(t.sb, t.sb_left * 4);
    lda = (uint32_t)t.lda;
    ldb = (uint32_t)t.ldb;
    na4 = (uint32_t)(mine_a ? t.na : t.nb) * 4;
    nb4 = (uint32_t)t.nb * 4;
    const int r = lane >> 3, slot = lane & 7;
#pragma unroll
    for (int i = 0; i < 2; ++i) voff_a[i] = r * lda + 16 * (slot ^ fa(8 * i + r));
#pragma unroll
    for (int i = 0; i < 4; ++i) voff_b[i] = r * ldb + 16 * (slot ^ fb<!F32>(8 * i + r));
    sa_off = ROWB ? 4 * lane : 4 * (wm * S::TM * 16 + (lane & 15));
    sb_off = 4 * (wn * S::TN * 16 / 128);
  }

  __device__ __forceinline__ void dma(int ks, uint8_t* st) const {
#pragma unroll
    for (int i = 0; i < S::dma_a; ++i) {
      const uint32_t rb8 = w * S::dma_a + i;
      dma_lds<16>(ra, st + rb8 * 1024, voff_a[i & 1], rb8 * 8 * lda + ks * 128);
    }
#pragma unroll
    for (int i = 0; i < S::dma_b; ++i) {
      const uint32_t rb8 = w * S::dma_b + i;
      dma_lds<16>(rb, st + S::kA + rb8 * 1024, voff_b[i & 3], rb8 * 8 * ldb + ks * 128);
    }
    if constexpr (ROWB) dma_lds<4>(rsa, st + S::kA + S::kB + schunk * 256, sa_off, ks * na4 + soff);
  }

  // Scales of block ks: the lane's rows of A and the wave's one of B (those of
  // single rows come by DMA with the codes).
  __device__ __forceinline__ void scales(int ks, float (&sa)[S::TM], float& sb) const {
    if constexpr (!ROWB) {
#pragma unroll
      for (int j = 0; j < S::TM; ++j)
        sa[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsa, sa_off + 64 * j, ks * na4, 0));
      sb = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsb, sb_off, ks * nb4, 0));
    }
  }

  __device__ __forceinline__ v8i frag_a(const uint8_t* st, int j) const {
    const int row = (wm * S::TM + j) * 16 + (lane & 15);
    const int s = (lane >> 4) ^ fa(lane & 15);
    const uint4* p = reinterpret_cast<const uint4*>(st) + row * 8;
    return join16(p[s], p[s ^ 4]);
  }

  __device__ __forceinline__ v8i frag_b(const uint8_t* st, int i) const {
    const int r = lane & 15, row = wn * S::TN * 16 + b_row<!F32>(i, r);
    const int s = (lane >> 4) ^ fb<!F32>(b_row<!F32>(0, r));
    const uint4* p = reinterpret_cast<const uint4*>(st + S::kA) + row * 8;
    return join16(p[s], p[s ^ 4]);
  }

  // Scales of the 4 rows of B that block i's result registers hold.
  __device__ __forceinline__ v4f row_scales(const uint8_t* st, int i) const {
    if constexpr (!ROWB) return v4f{};
    const int n = wn * S::TN * 16 + b_row<!F32>(i, 4 * (lane >> 4));
    return *reinterpret_cast<const v4f*>(st + S::kA + S::kB + 4 * (S::BM + n));
  }

  __device__ __forceinline__ void add(v4f& acc, const v4f& p, float sa, const v4f& sb) const {
    if constexpr (ROWB) {
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c] = fmaf(p[c] * sb[c], sa, acc[c]);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c] = fmaf(p[c], sa, acc[c]);
    }
  }

  __device__ __forceinline__ void compute(const uint8_t* st, const float (&sa)[S::TM], float sb,
                                          v4f (&acc)[S::TN][S::TM]) const {
    // the first product waits for two operands only
    v8i a[S::TM], b[2] = {frag_b(st, 0)};
    float s[S::TM];
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < S::TM; ++j) {
      a[j] = frag_a(st, j);
      s[j] = ROWB ? reinterpret_cast<const float*>(st + S::kA + S::kB)[(wm * S::TM + j) * 16 + (lane & 15)] : sa[j] * sb;
    }
    // a product's sums are added three products later, when it has left the matrix unit
    constexpr int kLag = 3, kAll = S::TN * S::TM;
    v4f p[kLag + 1], sr[2] = {row_scales(st, 0), row_scales(st, 1)};
    b[1] = frag_b(st, 1);
#pragma unroll
    for (int t = 0; t < kAll + kLag; ++t) {
      const int i = t / S::TM, j = t % S::TM, u = t - kLag;
      if (t < kAll && j == 0) __builtin_amdgcn_sched_barrier(0);
      if (t < kAll) p[t % (kLag + 1)] = mfma128(b[i & 1], a[j]);
      if (t < kAll && j == S::TM - 1 && i + 2 < S::TN) b[i & 1] = frag_b(st, i + 2);
      if (u >= 0) {
        const int ui = u / S::TM, uj = u % S::TM;
        add(acc[ui][uj], p[u % (kLag + 1)], s[uj], sr[ui & 1]);
        if (ROWB && uj == S::TM - 1 && ui + 2 < S::TN) sr[ui & 1] = row_scales(st, ui + 2);
      }
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, ROWB ? 8 : 4, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }

  // (Stores past the caches were slower: half-line pieces then reach HBM one by one,
  // 32 weight gradients of 7168 x 2048 in float32 from 128 rows each 384 -> 540 us.)
  __device__ __forceinline__ void store(const Tile& t, const v4f (&acc)[S::TN][S::TM]) const {
    constexpr int esz = F32 ? 4 : 2;
    const int m0 = wm * S::TM * 16 + (lane & 15), n0 = wn * S::TN * 16;
#pragma unroll
    for (int j = 0; j < S::TM; ++j) {
      const int m = m0 + 16 * j;
      if (m >= t.valid_m) continue;
      uint8_t* row = reinterpret_cast<uint8_t*>(t.out) + (int64_t)m * t.ldo * esz;
#pragma unroll
      for (int i = 0; i < S::TN; i += F32 ? 1 : 2) {
        const int n = n0 + b_row<!F32>(i, 4 * (lane >> 4));
        if (n >= t.valid_n) continue;     // rows of B come in multiples of 8
        const v4f x = acc[i][j];
        if constexpr (F32) {
          *reinterpret_cast<v4f*>(row + n * 4) = x;
        } else {
          const v4f y = acc[i + 1][j];
          *reinterpret_cast<uint4*>(row + n * 2) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                              pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
        }
      }
    }
  }
};

// Waits for this wave's loads and LDS accesses, then for the other waves.
__device__ __forceinline__ void step_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0), lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <class S, bool F32>
__device__ __forceinline__ void zero_tile(const Tile& t) {
  constexpr int esz = F32 ? 4 : 2, per = 16 / esz;
  const int chunks = (t.valid_n + per - 1) / per;      // valid_n is a multiple of 8
  for (int i = threadIdx.x; i < t.valid_m * chunks; i += S::threads) {
    const int r = i / chunks, c = i - r * chunks;
    *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(t.out) + (int64_t)r * t.ldo * esz + 16 * c) = make_uint4(0, 0, 0, 0);
  }
}

// Two stages in LDS, one barrier a block of k: the next block's codes come by
// DMA while this one's are multiplied.
template <class S, bool ROWB, bool F32>
__device__ __forceinline__ void run_tile(const Tile& t) {
  __shared__ __align__(16) uint8_t st0[S::stage];
  __shared__ __align__(16) uint8_t st1[S::stage];
  if (t.nk <= 0) return zero_tile<S, F32>(t);
  TileRun<S, ROWB, F32> x;
  x.init(t);
  v4f acc[S::TN][S::TM];
#pragma unroll
  for (int i = 0; i < S::TN; ++i)
#pragma unroll
    for (int j = 0; j < S::TM; ++j) acc[i][j] = v4f{0, 0, 0, 0};
  float sa0[S::TM], sb0 = 0, sa1[S::TM], sb1 = 0;
  // of the two waves of a SIMD one goes first: its products run while the other reads its operands
  if (S::waves == 8 && x.w < 4) __builtin_amdgcn_s_setprio(2);
  x.dma(0, st0);
  x.scales(0, sa0, sb0);
  step_barrier();
  const int last = t.nk - 1;
  int ks = 0;
  for (; ks + 1 < t.nk; ks += 2) {
    x.dma(ks + 1, st1);
    x.scales(ks + 1, sa1, sb1);
    x.compute(st0, sa0, sb0, acc);
    step_barrier();
    const int next = min(ks + 2, last);    // past the end: a block that is not used
    x.dma(next, st0);
    x.scales(next, sa0, sb0);
    x.compute(st1, sa1, sb1, acc);
    step_barrier();
  }
  if (ks < t.nk) x.compute(st0, sa0, sb0, acc);
  x.store(t, acc);
}

using Big = Shape<4, 2, 4, 8>;      // 256 x 256, 8 waves of 64 x 128
using Small = Shape<2, 2, 2, 4>;    // 64 x 128, 4 waves of 32 x 64

// Tile number of a workgroup: chunks of 16 tiles go to the XCDs in turn (they
// get workgroups round-robin), so those that run on one XCD share operands in
// its L2.
__device__ __forceinline__ int xcd_tile(int id, int n) {
  const int whole = n / 128 * 128;
  if (id >= whole) return id;
  const int x = id & 7, i = id >> 3;
  return (i / 16) * 128 + x * 16 + i % 16;
}

// The same for the weight gradient's tiles of one group: a contiguous eighth an XCD.
__device__ __forceinline__ int xcd_share(int id, int n) {
  const int x = id & 7;
  return x * (n / 8) + min(x, n % 8) + (id >> 3);
}

// Tile t of mt x nt in bands of `band` row tiles, column by column.
__device__ __forceinline__ void band_tile(int t, int mt, int nt, int band, int& tm, int& tn) {
  const int b = t / (band * nt), rows = min(band, mt - b * band), r = t - b * band * nt;
  tn = r / rows;
  tm = b * band + r - tn * rows;
}

template <class S, bool ROWB, bool F32>
__global__ __launch_bounds__(S::threads) void k_b128_mm(B128GemmArgs a) {
  const int mt = (int)((a.M + S::BM - 1) / S::BM), nt = (int)((a.N + S::BN - 1) / S::BN);
  int tm, tn;
  band_tile(xcd_tile(blockIdx.x, mt * nt), mt, nt, 4, tm, tn);
  const int64_t m0 = (int64_t)tm * S::BM, n0 = (int64_t)tn * S::BN, nb = ROWB ? a.N : (a.N + 127) / 128;
  Tile t;
  t.a = a.qa + m0 * a.K;
  t.b = a.qb + n0 * a.K;
  t.lda = t.ldb = a.K;
  t.nk = (int)(a.K / 128);
  t.sa = a.sa + m0;
  t.sb = a.sb + (ROWB ? n0 : n0 / 128);
  t.na = a.M;
  t.nb = nb;
  t.sa_left = t.nk * a.M - m0;
  t.sb_left = t.nk * nb - (ROWB ? n0 : n0 / 128);
  t.valid_m = (int)min<int64_t>(S::BM, a.M - m0);
  t.valid_n = (int)min<int64_t>(S::BN, a.N - n0);
  t.out = reinterpret_cast<uint8_t*>(a.out) + (m0 * a.ldo + n0) * (F32 ? 4 : 2);
  t.ldo = a.ldo;
  run_tile<S, ROWB, F32>(t);
}

// Row tiles of the groups in order, then of the rows behind the last group
// (written as zeros); the grid is an upper bound.
template <class S>
__global__ __launch_bounds__(S::threads) void k_b128_grouped(B128GemmArgs a, int max_mt) {
  const int nt = (int)((a.N + S::BN - 1) / S::BN);
  int tm, tn;
  band_tile(xcd_tile(blockIdx.x, max_mt * nt), max_mt, nt, 2, tm, tn);
  const Piece p = find_piece(a.offs, a.E, (int32_t)a.M, S::BM, tm, false, a.dev_err);
  const int64_t n0 = (int64_t)tn * S::BN, nb = (a.N + 127) / 128, nk = a.K / 128;
  const int64_t m0 = (p.group < 0 ? p.last : p.start) + (int64_t)p.index * S::BM;
  const int64_t end = p.group < 0 ? a.M : p.end;
  if (m0 >= end) return;
  const int64_t e = max(p.group, 0);
  Tile t;
  t.a = a.qa + m0 * a.K;
  t.b = a.qb + (e * a.N + n0) * a.K;
  t.lda = t.ldb = a.K;
  t.nk = p.group < 0 ? 0 : (int)nk;
  t.sa = a.sa + m0;
  t.sb = a.sb + e * nk * nb + n0 / 128;
  t.na = a.M;
  t.nb = nb;
  t.sa_left = nk * a.M - m0;
  t.sb_left = nk * nb - n0 / 128;
  t.valid_m = (int)min<int64_t>(S::BM, end - m0);
  t.valid_n = (int)min<int64_t>(S::BN, a.N - n0);
  t.out = reinterpret_cast<uint8_t*>(a.out) + (m0 * a.ldo + n0) * 2;
  t.ldo = a.ldo;
  run_tile<S, false, false>(t);
}

// dW[g] = A[:, rows of g] B[:, rows of g]^T: a group's tiles together, a group
// without rows gets zeros.
template <class S, bool F32>
__global__ __launch_bounds__(S::threads) void k_b128_wgrad(B128GemmArgs a) {
  const int mt = (int)((a.M + S::BM - 1) / S::BM), nt = (int)((a.N + S::BN - 1) / S::BN), per = mt * nt;
  const int want = (int)blockIdx.x / per;
  int tm, tn;
  band_tile(xcd_share((int)blockIdx.x - want * per, per), mt, nt, 4, tm, tn);
  const Piece p = group_rows(a.offs, a.E, (int32_t)a.K, want, a.dev_err);
  const int64_t g = p.group;
  const int64_t m0 = (int64_t)tm * S::BM, n0 = (int64_t)tn * S::BN, kb = p.start / 128;
  Tile t;
  t.a = a.qa + m0 * a.K + p.start;
  t.b = a.qb + n0 * a.K + p.start;
  t.lda = t.ldb = a.K;
  t.nk = (p.end - p.start) / 128;
  t.sa = a.sa + kb * a.M + m0;
  t.sb = a.sb + kb * a.N + n0;
  t.na = a.M;
  t.nb = a.N;
  t.sa_left = t.nk * a.M - m0;
  t.sb_left = t.nk * a.N - n0;
  t.valid_m = (int)min<int64_t>(S::BM, a.M - m0);
  t.valid_n = (int)min<int64_t>(S::BN, a.N - n0);
  t.out = reinterpret_cast<uint8_t*>(a.out) + ((g * a.M + m0) * a.ldo + n0) * (F32 ? 4 : 2);
  t.ldo = a.ldo;
  run_tile<S, true, F32>(t);
}

// ---------------------------------------------------------------- few rows
//
// With few rows of A the product is bound by streaming B, and tiles of 256 leave
// most of the card idle. A workgroup here holds teams of waves, each with a ring of
// STAGES stages in LDS of its own. G teams split the contraction (they take its
// blocks in turn and join their sums in LDS in a fixed order), H teams stand side by
// side along N. A team of one wave needs no barrier.
//
// Codes and scales all come by DMA, 128 contiguous bytes of a row to 8 lanes:
// loads straight into the matrix unit's layout touch 16 rows with 16 consecutive
// lanes, 64 separate pieces an instruction (one row, 4096 x 7168: 8.7 against 6.7 us).
template <int WM_, int WN_, int TM_, int TN_, int G_, int H_, int STAGES_>
struct Split {
  static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_, G = G_, H = H_, STAGES = STAGES_;
  static constexpr int team = WM * WN, waves = team * G * H, threads = waves * 64;
  static constexpr int BM = WM * TM * 16, BT = WN * TN * 16, BN = BT * H;      // BT: columns of a team
  static constexpr int dma_a = BM / 8 / team, dma_b = BT / 8 / team, dma_s = (BM + 63) / 64;
  static constexpr int kA = BM * 128, kB = BT * 128, kSA = dma_s * 256, stage = kA + kB + kSA + 256;
  static constexpr int ops = dma_a + dma_b + dma_s + 1;      // DMA instructions of a wave and block of k
  static constexpr int lds = G * H * STAGES * stage;
  static_assert(BT <= 64 && BM / 8 % team == 0 && BT / 8 % team == 0);
  static_assert(ops * (STAGES - 1) <= 63 && (G == 1 || waves * TM * TN * 1024 <= lds));
};

// Waits until at most N of this wave's loads are in flight, and for its LDS
// accesses; nothing moves across.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x70);
  asm volatile("" ::: "memory");
}

template <class S, bool ROWB, bool F32>
__device__ __forceinline__ void run_split(const Tile& t) {
  __shared__ __align__(16) uint8_t lds[S::lds];
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), team = wave / S::team, w = wave % S::team;
  const int g = team % S::G, h = team / S::G;
  const int wm = w / S::WN, wn = w % S::WN, r = lane & 15, q = lane >> 4;
  uint8_t* mine = lds + team * S::STAGES * S::stage;
  const __amdgpu_buffer_rsrc_t ra = buffer(t.a, t.valid_m * t.lda);
  const int valid_n = max(min(t.valid_n - h * S::BT, S::BT), 0);      // this team's rows of B
  const __amdgpu_buffer_rsrc_t rb = buffer(t.b + h * S::BT * t.ldb, valid_n * t.ldb);
  const __amdgpu_buffer_rsrc_t rsa = buffer(t.sa, t.sa_left * 4);
  const __amdgpu_buffer_rsrc_t rsb = buffer(t.sb, t.sb_left * 4);
  const uint32_t lda = (uint32_t)t.lda, ldb = (uint32_t)t.ldb, na4 = (uint32_t)t.na * 4, nb4 = (uint32_t)t.nb * 4;
  // lane: row lane >> 3 of an 8-row instruction, slot lane & 7 (see fa)
  uint32_t va[S::dma_a], vb[S::dma_b];
#pragma unroll
  for (int i = 0; i < S::dma_a; ++i) {
    const int row = 8 * (w * S::dma_a + i) + (lane >> 3);
    va[i] = row * lda + 16 * ((lane & 7) ^ fa(row));
  }
#pragma unroll
  for (int i = 0; i < S::dma_b; ++i) {
    const int row = 8 * (w * S::dma_b + i) + (lane >> 3);
    vb[i] = row * ldb + 16 * ((lane & 7) ^ fa(row));
  }
  // a tile of blocked B lies within one block of 128 columns, or starts with one
  const uint32_t vsb = ROWB ? 4 * (h * S::BT + lane) : 4 * (h * S::BT / 128);
  const int last = t.nk - 1;
  auto fetch = [&](int ks, int stage) {
    ks = min(ks, last);       // past the end: a block that is not used
    uint8_t* st = mine + stage * S::stage;
#pragma unroll
    for (int i = 0; i < S::dma_a; ++i) dma_lds<16>(ra, st + (w * S::dma_a + i) * 1024, va[i], ks * 128);
#pragma unroll
    for (int i = 0; i < S::dma_b; ++i) dma_lds<16>(rb, st + S::kA + (w * S::dma_b + i) * 1024, vb[i], ks * 128);
    // (the waves of a team write the same scales)
#pragma unroll
    for (int i = 0; i < S::dma_s; ++i) dma_lds<4>(rsa, st + S::kA + S::kB + 256 * i, 256 * i + 4 * lane, ks * na4);
    dma_lds<4>(rsb, st + S::kA + S::kB + S::kSA, vsb, ks * nb4);
  };
  v4f acc[S::TN][S::TM];
#pragma unroll
  for (int i = 0; i < S::TN; ++i)
#pragma unroll
    for (int j = 0; j < S::TM; ++j) acc[i][j] = v4f{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < S::STAGES - 1; ++i) fetch(i * S::G + g, i);
  const int rounds = (t.nk + S::G - 1) / S::G;
  int stage = 0;
  for (int it = 0; it < rounds; ++it) {
    wait_loads<S::ops*(S::STAGES - 2)>();
    if constexpr (S::team > 1) __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    // the stage that was read in the last round is free
    fetch((it + S::STAGES - 1) * S::G + g, stage == 0 ? S::STAGES - 1 : stage - 1);
    if (it * S::G + g < t.nk) {
      const uint8_t* st = mine + stage * S::stage;
      const float* sa = reinterpret_cast<const float*>(st + S::kA + S::kB);
      const float* sb = sa + S::kSA / 4;
      const int slot = q ^ fa(r);
      v8i a[S::TM];
      float s[S::TM];
#pragma unroll
      for (int j = 0; j < S::TM; ++j) {
        const int row = (wm * S::TM + j) * 16 + r;
        const uint4* p = reinterpret_cast<const uint4*>(st) + row * 8;
        a[j] = join16(p[slot], p[slot ^ 4]);
        s[j] = ROWB ? sa[row] : sa[row] * sb[0];
      }
#pragma unroll
      for (int i = 0; i < S::TN; ++i) {
        const int row = (wn * S::TN + i) * 16;
        const uint4* p = reinterpret_cast<const uint4*>(st + S::kA) + (row + r) * 8;
        const v8i b = join16(p[slot], p[slot ^ 4]);
        const v4f sr = ROWB ? *reinterpret_cast<const v4f*>(sb + row + 4 * q) : v4f{};
        v4f x[S::TM];
#pragma unroll
        for (int j = 0; j < S::TM; ++j) x[j] = mfma128(b, a[j]);
#pragma unroll
        for (int j = 0; j < S::TM; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[i][j][c] = fmaf(ROWB ? x[j][c] * sr[c] : x[j][c], s[j], acc[i][j][c]);
      }
    }
    stage = stage + 1 == S::STAGES ? 0 : stage + 1;
  }
  wait_loads<0>();
  constexpr int kParts = S::team * S::TN * S::TM;      // 16 x 16 pieces of a team's tile
  auto put = [&](int u, const v4f& c) {
    const int uw = u / (S::TN * S::TM), i = u / S::TM % S::TN, j = u % S::TM;
    const int m = ((uw / S::WN) * S::TM + j) * 16 + r, n = h * S::BT + ((uw % S::WN) * S::TN + i) * 16 + 4 * q;
    if (m < t.valid_m && n < t.valid_n) {
      if constexpr (F32)
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(t.out) + m * t.ldo + n) = make_float4(c[0], c[1], c[2], c[3]);
      else
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(t.out) + m * t.ldo + n) =
            make_uint2(pack_bf16x2(c[0], c[1]), pack_bf16x2(c[2], c[3]));
    }
  };
  if constexpr (S::G == 1) {
#pragma unroll
    for (int i = 0; i < S::TN; ++i)
#pragma unroll
      for (int j = 0; j < S::TM; ++j) put((w * S::TN + i) * S::TM + j, acc[i][j]);
  } else {
    static_assert(S::H == 1);
    __syncthreads();
    v4f* part = reinterpret_cast<v4f*>(lds);      // [G][kParts][64]
#pragma unroll
    for (int i = 0; i < S::TN; ++i)
#pragma unroll
      for (int j = 0; j < S::TM; ++j) part[((wave * S::TN + i) * S::TM + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    for (int u = wave; u < kParts; u += S::waves) {
      v4f c = part[u * 64 + lane];
#pragma unroll
      for (int k = 1; k < S::G; ++k) c += part[(k * kParts + u) * 64 + lane];
      put(u, c);
    }
  }
}

// 16 TM rows and 16 columns a workgroup; 16 rows and 16 columns a wave, which takes
// all of k; more rows: 64 x 64 and 128 x 64.
template <int TM>
using Few = Split<1, 1, TM, 1, TM == 4 ? 4 : 8, 1, TM == 1 ? 4 : 3>;
using FewWide = Split<1, 1, 1, 1, 1, 8, 4>;
using Mid = Split<2, 2, 2, 2, 2, 1, 4>;
using Mid2 = Split<2, 2, 4, 2, 2, 1, 3>;

template <class S, bool ROWB, bool F32>
__global__ __launch_bounds__(S::threads) void k_b128_split(B128GemmArgs a, int mt) {
  // the row tiles of one column tile run on one XCD, which reads B once
  const int xcd = blockIdx.x & 7, j = blockIdx.x >> 3;
  const int64_t m0 = (int64_t)(j % mt) * S::BM, n0 = (int64_t)(j / mt * 8 + xcd) * S::BN;
  if (n0 >= a.N) return;
  const int64_t nb = ROWB ? a.N : (a.N + 127) / 128, nk = a.K / 128;
  Tile t;
  t.a = a.qa + m0 * a.K;
  t.b = a.qb + n0 * a.K;
  t.lda = t.ldb = a.K;
  t.nk = (int)nk;
  t.sa = a.sa + m0;
  t.sb = a.sb + (ROWB ? n0 : n0 / 128);
  t.na = a.M;
  t.nb = nb;
  t.sa_left = nk * a.M - m0;
  t.sb_left = nk * nb - (ROWB ? n0 : n0 / 128);
  t.valid_m = (int)min<int64_t>(S::BM, a.M - m0);
  t.valid_n = (int)min<int64_t>(S::BN, a.N - n0);
  t.out = reinterpret_cast<uint8_t*>(a.out) + (m0 * a.ldo + n0) * (F32 ? 4 : 2);
  t.ldo = a.ldo;
  run_split<S, ROWB, F32>(t);
}

// One workgroup for S::BN columns of one group with rows, walking the group's
// rows; the piece behind the last such group: the rows behind it, written as zeros.
template <class S>
__global__ __launch_bounds__(S::threads) void k_b128_split_grouped(B128GemmArgs a, int nt) {
  const int r = (int)blockIdx.x / nt;
  const int64_t n0 = (int64_t)((int)blockIdx.x - r * nt) * S::BN, nk = a.K / 128, nb = (a.N + 127) / 128;
  const Piece p = find_piece(a.offs, a.E, (int32_t)a.M, 0, r, false, a.dev_err);
  if (p.group < 0 && p.index > 0) return;
  const int64_t e = max(p.group, 0), end = p.group < 0 ? a.M : p.end;
  Tile t;
  t.b = a.qb + (e * a.N + n0) * a.K;
  t.lda = t.ldb = a.K;
  t.sb = a.sb + e * nk * nb + n0 / 128;
  t.na = a.M;
  t.nb = nb;
  t.sb_left = nk * nb - n0 / 128;
  t.valid_n = (int)min<int64_t>(S::BN, a.N - n0);
  t.ldo = a.ldo;
  for (int64_t m0 = p.group < 0 ? p.last : p.start; m0 < end; m0 += S::BM) {
    t.out = reinterpret_cast<uint16_t*>(a.out) + m0 * a.ldo + n0;
    t.valid_m = (int)min<int64_t>(S::BM, end - m0);
    if (p.group < 0) {
      zero_tile<S, false>(t);
      continue;
    }
    t.nk = (int)nk;
    t.a = a.qa + m0 * a.K;
    t.sa = a.sa + m0;
    t.sa_left = nk * a.M - m0;
    run_split<S, false, false>(t);
    __syncthreads();      // before the next rows' codes go where sums are still read
  }
}

// ---------------------------------------------------------------- launch

// Which kernel, by the columns of B (of all groups with rows) and the rows of A (a
// group). Few: k split eight ways, best while there is a workgroup or two of 16
// columns a CU. Mid: up to a workgroup or two of 64 columns a CU. FewWide, Small: a
// wave's or tile's whole k, from columns enough to fill the card on. us of
// Few / FewWide / Mid / Small, codes from HBM:
//      16 x  4096 x 7168    6.8   20   16    31        64 x  4096 x 7168   9.6    -   16    32
//      16 x  8192 x 7168     16   33   18    48        64 x  8192 x 7168    25    -   22    48
//      16 x 16384 x 7168     30   36   22    50        64 x 16384 x 7168    47    -   25    50
//      16 x 24576 x 2048     20   12   15    16        64 x 24576 x 7168    70    -   45    53
//      16 x 32768 x 2048     27   14   17    18        64 x 32768 x 7168    64    -   39    38
//      16 x 65536 x 2048     42   24   28    21        64 x 65536 x 7168   184    -   98    86
//    4 x  8 x 4096 x 7168    29   33   24    50   4 x 64 x 4096 x 7168      50    -   26    51
//    4 x  1 x 7168 x 2048    24   12   15    13   8 x 32 x 7168 x 2048      61    -   33    24
//   32 x  1 x 1024 x 2048    27   13   17    16  32 x 64 x 4096 x 7168     391    -  199   173
//  256 x  1 x 4096 x 7168  1824 1227 1292  1202 256 x 32 x 7168 x 2048    2293    -  967   701
// (groups first where there are four numbers.) Few, FewWide and Mid walk a group's
// rows one after the other, Small's tiles do not: with half of 32 x 32 rows in one group
// of 1024 x 2048, 38, 56, 49 and 18.
constexpr int64_t kFewColumns = 4096, kMidColumns = 16384, kWideColumns = 32768;

constexpr int kCUs = 256;

template <class Fn>
static void with_out(const B128GemmArgs& a, Fn f) {
  using T = std::true_type;
  using F = std::false_type;
  if (a.block_b) {
    if (a.out_f32) f(F{}, T{});
    else f(F{}, F{});
  } else {
    if (a.out_f32) f(T{}, T{});
    else f(T{}, F{});
  }
}

// The variant of a dense product: f(shape, whether it is a split one, its workgroups).
template <class Fn>
static auto with_mm(const B128GemmArgs& a, Fn f) {
  auto tiles = [&](auto shape) {
    using S = decltype(shape);
    return ((a.M + S::BM - 1) / S::BM) * ((a.N + S::BN - 1) / S::BN);
  };
  auto split = [&](auto shape) {
    using S = decltype(shape);
    const int64_t mt = (a.M + S::BM - 1) / S::BM, nt = (a.N + S::BN - 1) / S::BN;
    return f(shape, std::true_type{}, mt * ((nt + 7) / 8 * 8));
  };
  if (a.K > 0 && a.M <= 64) {
    if (a.M <= 16 && a.N <= 2 * kFewColumns) return split(Few<1>{});
    if (a.M <= 32 && a.N <= 2 * kFewColumns) return split(Few<2>{});
    if (a.N <= kFewColumns) return split(Few<4>{});
    if (a.M <= 16 && a.N > kMidColumns && a.N < 2 * kWideColumns) return split(FewWide{});
    if (a.N < kWideColumns) return split(Mid{});
  }
  // more rows: split tiles while the card takes them all at once, large ones from half of the CUs on. us of Mid /
  // Mid2 / Small / Big: 256 x 4096 x 7168 17, 26, 32, 81; 512 x 4096 x 7168 32, 27, 34, 82; 512 x 7168 x 2048 25, 20,
  // 15, 29; 1024 x 4096 x 7168 64, 53, 41, 82; 2304 x 4096 x 7168 -, -, 88, 83; 1536 x 7168 x 2048 -, -, 36, 31.
  if (a.K > 0 && tiles(Mid{}) <= kCUs) return split(Mid{});
  if (a.K > 0 && tiles(Mid2{}) <= kCUs) return split(Mid2{});
  if (tiles(Big{}) > kCUs / 2) return f(Big{}, std::false_type{}, tiles(Big{}));
  return f(Small{}, std::false_type{}, tiles(Small{}));
}

int64_t b128_mm_grid(const B128GemmArgs& a) {
  return with_mm(a, [](auto, auto, int64_t n) { return n; });
}

hipError_t launch_b128_mm(const B128GemmArgs& a, hipStream_t s) {
  if (a.M == 0 || a.N == 0) return hipSuccess;
  return with_mm(a, [&](auto shape, auto split, int64_t n) {
    using S = decltype(shape);
    with_out(a, [&](auto rowb, auto f32) {
      if constexpr (decltype(split)::value)
        hipLaunchKernelGGL((k_b128_split<S, rowb, f32>), dim3((unsigned)n), dim3(S::threads), 0, s, a,
                           (int)((a.M + S::BM - 1) / S::BM));
      else
        hipLaunchKernelGGL((k_b128_mm<S, rowb, f32>), dim3((unsigned)n), dim3(S::threads), 0, s, a);
    });
    return hipGetLastError();
  });
}

// The same for a grouped product, whose workgroups are n for each column tile.
template <class Fn>
static auto with_grouped(const B128GemmArgs& a, Fn f) {
  const int64_t active = std::min<int64_t>(a.E, a.M);
  auto split = [&](auto shape) { return f(shape, std::true_type{}, active + 1); };
  auto whole = [&](auto shape) { return f(shape, std::false_type{}, a.M / decltype(shape)::BM + active + 1); };
  const int64_t columns = active * a.N;
  if (a.M <= 64 * active) {
    if (a.M <= 16 * active && columns <= 2 * kFewColumns) return split(Few<1>{});
    if (columns <= kFewColumns) return split(Few<4>{});
    // (a few rows a group on the average: hardly any group then needs a second walk)
    if (a.M <= 4 * active && columns > kMidColumns && columns < 2 * kWideColumns) return split(FewWide{});
    if (columns < kWideColumns) return split(Mid{});
  }
  // Large tiles for 128 rows a group and more, if they give half of the CUs one and have rows enough: their time hardly
  // depends on how many they hold. Rows a group times large tiles says how much there is to share out; from 16384 (the
  // third example) to 28672 (the fifth) the order turns. us of Small / Big: 32 x 128 x 4096 x 7168 254, 221; 32 x 100 x 7168 x 2048 122, 128; 8 x 128 x
  // 4096 x 7168 66, 87; 8 x 256 x 4096 x 7168 122, 98; 8 x 128 x 7168 x 2048 40, 34; 32 x 256 x 768 x 2048 22, 31;
  // 8 x 512 x 1536 x 7168 82, 92; 8 x 768 x 1536 x 7168 114, 92.
  const int64_t large = std::max(active, a.M / Big::BM) * ((a.N + Big::BN - 1) / Big::BN);
  if (a.M >= 128 * active && large >= kCUs / 2 && a.M / active * large >= 160 * (kCUs / 2)) return whole(Big{});
  return whole(Small{});
}

int64_t b128_grouped_grid(const B128GemmArgs& a) {
  return with_grouped(a, [&](auto shape, auto, int64_t n) { return n * ((a.N + shape.BN - 1) / shape.BN); });
}

hipError_t launch_b128_grouped(const B128GemmArgs& a, hipStream_t s) {
  if (a.M == 0 || a.N == 0) return hipSuccess;
  return with_grouped(a, [&](auto shape, auto split, int64_t n) {
    using S = decltype(shape);
    const int64_t nt = (a.N + S::BN - 1) / S::BN;
    const dim3 grid((unsigned)(n * nt));
    if constexpr (decltype(split)::value) hipLaunchKernelGGL(k_b128_split_grouped<S>, grid, dim3(S::threads), 0, s, a, (int)nt);
    else hipLaunchKernelGGL(k_b128_grouped<S>, grid, dim3(S::threads), 0, s, a, (int)n);
    return hipGetLastError();
  });
}

int64_t b128_wgrad_grid(const B128GemmArgs& a) {
  return a.E * ((a.M + Big::BM - 1) / Big::BM) * ((a.N + Big::BN - 1) / Big::BN);
}

hipError_t launch_b128_wgrad(const B128GemmArgs& a, hipStream_t s) {
  if (a.M == 0 || a.N == 0) return hipSuccess;
  using S = Big;
  const dim3 grid((unsigned)b128_wgrad_grid(a)), block(S::threads);
  if (a.out_f32) hipLaunchKernelGGL((k_b128_wgrad<S, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_b128_wgrad<S, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace mxk
