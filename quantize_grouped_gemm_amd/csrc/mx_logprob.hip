// Log probabilities of given tokens, with entropy and top alternatives, and
// the gradient of the logits as an MX operand:
//   k_logprob_part   sums, maximum and best entries of a row or of a segment
//   k_logprob_join   joins the segments of a row
//   k_logprob_bwd    one 128 x 128 tile of the gradient per workgroup
//
// In base 2: with c = scale log2(e) and d_j = (x_j - m) c, the row's sums are
// S = sum 2^d_j and A = sum 2^d_j d_j, m the row's maximum; then ls = ln S,
// entropy = ln S - ln2 A / S. Nothing overflows and a masked entry
// (-infinity) adds exactly 0.
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
#include <type_traits>

namespace mxk {

constexpr float kLog2e = 1.44269504088896341f;
constexpr double kLog2eD = 1.4426950408889634074;
constexpr float kLn2 = 0.693147180559945309f;

// N logits starting at element `i` < n of a row of n; `fill` past the end.
template <bool F32, int N>
__device__ __forceinline__ void load_logits(const void* row, int64_t i, int64_t n, float fill, float (&f)[N]) {
  if constexpr (F32) {
    const float* p = static_cast<const float*>(row) + i;
    if (i + N <= n) {
      __builtin_memcpy(f, p, 4 * N);
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) f[k] = i + k < n ? p[k] : fill;
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(row) + i;
    if (i + N <= n) {
      uint16_t v[N];
      __builtin_memcpy(v, p, 2 * N);
#pragma unroll
      for (int k = 0; k < N; ++k) f[k] = __uint_as_float((uint32_t)v[k] << 16);
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) f[k] = i + k < n ? __uint_as_float((uint32_t)p[k] << 16) : fill;
    }
  }
}

template <bool F32>
__device__ __forceinline__ const void* logits_row(const LogprobArgs& a, int64_t row) {
  return static_cast<const char*>(a.x) + row * a.ld * (F32 ? 4 : 2);
}

// Arguments of the forward kernels; part_work and the rest see them widened.
struct LogprobPack {
  const void* x;
  const int64_t* targets;
  int32_t* dev_err;
  float *logp, *entropy, *stats, *top_logp;
  int32_t* top_idx;
  void* work;
  int64_t ignore_index, ld;
  int32_t rows, vocab, top;
  float scale;
  int32_t parts, seg;        // of a row's split

  __device__ LogprobArgs wide() const {
    LogprobArgs a{};
    a.x = x; a.ld = ld; a.rows = rows; a.vocab = vocab; a.targets = targets; a.ignore_index = ignore_index;
    a.scale = scale; a.dev_err = dev_err; a.top = top; a.logp = logp; a.entropy = entropy; a.stats_out = stats;
    a.top_logp = top_logp; a.top_idx = top_idx; a.work = work;
    return a;
  }
};
static_assert(sizeof(LogprobPack) <= kArgBytes);

struct LogprobBwdPack {
  const void* x;
  const int64_t* targets;
  int32_t* dev_err;
  const float *stats, *ent_in, *dlogp, *dent;
  uint8_t *q_row, *s_row, *q_col, *s_col;
  int64_t ignore_index;
  uint32_t ld_bands;         // 2 ld + bands
  int32_t rows, vocab;
  float scale;

  template <class F>
  __device__ LogprobArgs wide() const {
    LogprobArgs a{};
    a.x = x; a.ld = ld_bands >> 1; a.bands = ld_bands & 1; a.rows = rows; a.vocab = vocab; a.targets = targets;
    a.ignore_index = ignore_index; a.scale = scale; a.dev_err = dev_err; a.stats = stats; a.ent_in = ent_in;
    a.dlogp = dlogp; a.dent = dent; a.vocab_pad = padded<F>(vocab); a.rows_pad = padded<F>(rows);
    a.q_row = q_row; a.s_row = s_row; a.q_col = q_col; a.s_col = s_col;
    return a;
  }
};
static_assert(sizeof(LogprobBwdPack) <= kArgBytes);

// The row's target, or -1 if it is not scored.
__device__ __forceinline__ int64_t row_target(const LogprobArgs& a, int64_t row) {
  const int64_t t = a.targets[row];
  return t == a.ignore_index || t < 0 || t >= a.vocab ? -1 : t;
}

// Order of the alternatives as one number: larger for a larger value, then
// for a lower index (the sign of zero does not count, a NaN comes first).
__device__ __forceinline__ uint64_t top_key(float x, uint32_t idx) {
  const uint32_t u = x == x ? __float_as_uint(x + 0.0f) : 0x7FC00000u;
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

// Raw logits of a thread's chunks.
template <bool F32>
struct RawChunk {
  uint4 w[F32 ? 2 : 1];
};

// 8 logits at p, aligned to their element only.
template <bool F32, bool STREAM>
__device__ __forceinline__ RawChunk<F32> load_raw(const char* p) {
  typedef unsigned v4u __attribute__((ext_vector_type(4), aligned(2)));
  RawChunk<F32> r;
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) {
    const v4u* q = reinterpret_cast<const v4u*>(p + 16 * i);
    const v4u v = STREAM ? __builtin_nontemporal_load(q) : *q;
    r.w[i] = make_uint4(v.x, v.y, v.z, v.w);
  }
  return r;
}

// ---------------------------------------------------------------- forward
//
// One read of the logits. A workgroup streams its segment in tiles of
// NT x U chunks of 8; while it sums, each thread keeps the maximum of every
// *slot* of its share (a slot: the thread's chunks of one or a few tiles) in
// LDS, at the cost of the maximum that the softmax needs anyway. The `top`
// best entries then follow from the slots: the top-th largest of the
// threads' maxima is a lower bound of the top-th largest entry, so only slots
// that reach it can hold one (about `top` of some 4096), and only those are
// read again, from cache.
//
// Softmax sums are kept per thread relative to an integer r: 2^(x c - r) with
// r = rint(c times the thread's maximum so far), raised when a tile passes it by
// 2^kRaise. One fused multiply-add forms the exponent, changes of r are exact
// powers of two, and no per-element maximum is needed. A tile's sums are formed by
// themselves and then added to the thread's: next to a term that outweighs the rest
// (a token predicted almost surely), terms added one by one fall below its last
// place, and A holds that term times its distance to r, which its shift to m takes
// away again. With sums running over the segment and r up to 32 below the maximum, the
// entropy of rows with p = 0.9 was off by 4e-5 at a vocabulary of 131072, now 3e-7
// (a plain float32 form: 1e-7), in the same time.

constexpr float kRaise = 8.0f;
constexpr int kSlots = 16;
constexpr int kRound = 1024;                // entries looked at between two checks of the candidate count
constexpr int kCand = kRound + kMaxTop;
constexpr int kList = 512;                  // slots worth reading one by one
// The fast sums hold exponents up to kFarExp in size: x c - r is rounded once,
// but r is the rounded m c, off by up to 2^-24 |m c|, which has to stay small as
// an exponent (at 2^32 the largest term would be 2^256). Rows whose maximum lies
// beyond take far_sums. Entries below kNoRef never set r, so a run of them
// (a finite mask) leaves nothing in the sums.
constexpr float kNoRef = -0x1p28f;
constexpr float kFarExp = 0x1p27f;

template <bool F32>
constexpr int kUnroll = F32 ? 2 : 4;

__device__ __forceinline__ uint32_t key16(float x) { return (uint32_t)(top_key(x, 0) >> 48); }
constexpr uint32_t kLowest16 = 0x007F;      // key16(-infinity), no other value's

template <int N>
__device__ __forceinline__ float max_of(const float (&f)[N], float m) {
#pragma unroll
  for (int k = 0; k < N; ++k) m = fmaxf(m, f[k]);
  return m;
}

// How many of n keys in LDS are larger than `key`. Unrolled: one read in flight
// at a time would pay LDS's latency for each.
__device__ __forceinline__ int count_larger(const uint64_t* keys, int n, uint64_t key) {
  int r = 0, j = 0;
  for (; j + 8 <= n; j += 8) {
#pragma unroll
    for (int u = 0; u < 8; ++u) r += keys[j + u] > key ? 1 : 0;
  }
  for (; j < n; ++j) r += keys[j] > key ? 1 : 0;
  return r;
}

template <int NT>
struct TopLds {
  uint16_t slot[kSlots][NT];
  uint64_t cand[kCand];
  uint64_t best[kMaxTop];
  uint64_t thr;          // entries with a larger key are candidates
  uint16_t list[kList];
  uint16_t tkey[NT];
  bool any[2][NT / 64];
  int count, hits;
};

// Keeps the `top` largest of l.cand[0 .. count), in descending order, and
// raises the threshold to the last of them once there are `top`. Keys are
// unique, so an entry's rank is the number of larger ones. All threads call
// it; barriers inside, the last one after the writes.
template <int NT>
__device__ __forceinline__ void keep_top(TopLds<NT>& l, int top) {
  const int t = threadIdx.x;
  __syncthreads();
  const int n = l.count;
#pragma unroll 1
  for (int i = t; i < n; i += NT) {
    const uint64_t key = l.cand[i];
    const int r = count_larger(l.cand, n, key);
    if (r < top) l.best[r] = key;
  }
  __syncthreads();
  const int kept = min(n, top);
  if (t < kept) l.cand[t] = l.best[t];
  if (t == 0) {
    l.count = kept;
    if (kept == top) l.thr = l.best[top - 1];
  }
  __syncthreads();
}

// Between two rounds of offers: makes room if the next one might not fit. All
// threads call it.
template <int NT>
__device__ __forceinline__ void make_room(TopLds<NT>& l, int top) {
  __syncthreads();
  const bool full = l.count > kCand - kRound;
  if (full) keep_top(l, top);
  else __syncthreads();
}

// Offers N consecutive entries of a thread from index i on: those of keys above
// thr become candidates (those past kCand are only counted).
template <bool F32, int N, int NT>
__device__ __forceinline__ void offer(TopLds<NT>& l, const void* x, int64_t i, int64_t n, uint32_t idx0, uint64_t thr) {
  float f[N];
  load_logits<F32>(x, i, n, -INFINITY, f);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const uint64_t key = top_key(f[k], idx0 + (uint32_t)(i + k));
    if (key > thr && i + k < n) {
      const int at = atomicAdd(&l.count, 1);
      if (at < kCand) l.cand[at] = key;
    }
  }
}

// Lists the slots whose maximum is at least `bound`; returns their number (all
// threads call it, barriers inside).
template <int NT>
__device__ __forceinline__ int list_slots(TopLds<NT>& l, int slots, uint32_t bound) {
  const int t = threadIdx.x;
  __syncthreads();
  if (t == 0) l.hits = 0;
  __syncthreads();
  for (int s = 0; s < slots; ++s) {
    if (l.slot[s][t] >= bound) {
      const int at = atomicAdd(&l.hits, 1);
      if (at < kList) l.list[at] = (uint16_t)(s * NT + t);
    }
  }
  __syncthreads();
  return l.hits;
}

// Candidates from the listed slots: entries of keys above thr. No barriers
// between its loads: few entries pass, and if more do than there is room for,
// l.count says so afterwards.
template <bool F32, int NT>
__device__ __forceinline__ void offer_list(TopLds<NT>& l, const void* x, int64_t n, uint32_t idx0, int hits, int tiles,
                                           uint64_t thr) {
  constexpr int kEach = kRound / NT, kSplit = 8 / kEach;   // entries at a time, pieces of a chunk
  const int per = kUnroll<F32> * tiles;                    // chunks of a slot
  for (int item = threadIdx.x; item < hits * per * kSplit; item += NT) {
    const int e = l.list[item / (per * kSplit)], h = item % (per * kSplit);
    const int64_t i = 8 * ((int64_t)(e / NT) * per * NT + (int64_t)(h / kSplit) * NT + e % NT) + kEach * (h % kSplit);
    if (i < n) offer<F32, kEach, NT>(l, x, i, n, idx0, thr);
  }
  __syncthreads();
}

// Candidates from the whole segment, read again: first one entry a thread, whose
// best raise the threshold, then in pieces that cost a barrier where nothing
// passes.
template <bool F32, int NT>
__device__ __forceinline__ void offer_all(TopLds<NT>& l, const void* x, int64_t n, uint32_t idx0, int top) {
  constexpr int kEach = kRound / NT, kPiece = 8 * kRound;
  const int t = threadIdx.x;
  __syncthreads();
  if (t == 0) l.count = 0;
  __syncthreads();
  if (t < n) offer<F32, 1, NT>(l, x, t, n, idx0, l.thr);
  keep_top(l, top);
  for (int64_t base = NT; base < n; base += kPiece) {
    const uint64_t thr = l.thr;
    bool any = false;
    for (int j = 0; j < 8; ++j) {
      const int64_t i = base + (int64_t)kRound * j + kEach * t;
      float f[kEach];
      if (i < n) {
        load_logits<F32>(x, i, n, -INFINITY, f);
#pragma unroll
        for (int k = 0; k < kEach; ++k) any |= top_key(f[k], idx0 + (uint32_t)(i + k)) > thr && i + k < n;
      }
    }
    const int turn = (int)(base / kPiece) & 1;   // the other one may still be read
    any = __any(any);
    if ((t & 63) == 0) l.any[turn][t >> 6] = any;
    __syncthreads();
    any = false;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) any |= l.any[turn][w];
    if (!__builtin_amdgcn_readfirstlane(any)) continue;
    for (int j = 0; j < 8; ++j) {
      const int64_t i = base + (int64_t)kRound * j + kEach * t;
      if (i < n) offer<F32, kEach, NT>(l, x, i, n, idx0, l.thr);
      make_room(l, top);
    }
  }
}

// The `top` best entries of the segment [0, n) of x (first index idx0), in
// descending order in l.cand[0 .. l.count). `slots` slots of `tiles` tiles
// each; tmax the thread's maximum. Maxima leave NaN out, so a segment that has
// one (`nan`; an infinity may count as one) is read again as a whole.
//
// Where most slots reach the bound, a mask (or a constant) has made it the
// value of most entries. If equal upper halves of float32 mean equal values (bf16, and
// -infinity in either type), the entries above it come from the few slots above it, and
// the others are the first ones in order of their index.
template <bool F32, int NT>
__device__ __forceinline__ void find_top(TopLds<NT>& l, const void* x, int64_t n, uint32_t idx0, float tmax, bool nan,
                                         int slots, int tiles, int top) {
  constexpr int kFill = 128;
  const int t = threadIdx.x;
  l.tkey[t] = (uint16_t)key16(tmax);
  if (t == 0) l.count = 0;
  __syncthreads();
  if (t < 64) {
    // the top-th largest of the NT keys, bit by bit
    uint32_t k[NT / 64];
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) k[i] = l.tkey[t + 64 * i];
    uint32_t bound = 0;
    for (int b = 15; b >= 0; --b) {
      const uint32_t tryb = bound | (1u << b);
      int c = 0;
#pragma unroll
      for (int i = 0; i < NT / 64; ++i) c += __popcll(__ballot(k[i] >= tryb));
      if (c >= top) bound = tryb;
    }
    if (t == 0) l.thr = bound ? ((uint64_t)bound << 48) - 1 : 0;
  }
  __syncthreads();
  int hits = list_slots(l, slots, (uint32_t)((l.thr + 1) >> 48));
  const uint64_t thr = l.thr;
  const uint32_t bound = (uint32_t)((thr + 1) >> 48);
  bool whole = true;
  if (!nan && 2 * hits > slots * NT && (!F32 || bound == kLowest16)) {
    hits = list_slots(l, slots, bound + 1);
    if (hits <= kList) {
      offer_list<F32, NT>(l, x, n, idx0, hits, tiles, thr + (1ull << 48));
      whole = l.count > kCand;
      // a few at a time, as most are of that value: ranking takes the square of their number
      for (int64_t base = 0; !whole && l.count < top && base < n; base += kFill) {
        __syncthreads();
        const int64_t i = base + t;
        if (t < kFill && i < n) {
          float f[1];
          load_logits<F32>(x, i, n, -INFINITY, f);
          const uint64_t key = top_key(f[0], idx0 + (uint32_t)i);
          if ((uint32_t)(key >> 48) == bound) l.cand[atomicAdd(&l.count, 1)] = key;
        }
        __syncthreads();
      }
    }
  } else if (!nan && hits <= kList) {
    offer_list<F32, NT>(l, x, n, idx0, hits, tiles, thr);
    whole = l.count > kCand;
  }
  if (whole) offer_all<F32, NT>(l, x, n, idx0, top);
  keep_top(l, top);
}

// A of sums s whose exponents all gain d. The product is rounded by itself (no
// fused product-sum): where s is one term 2^-d, A is its product with -d, rounded,
// and both cancel to exactly 0, the entropy of a row with one token left.
__device__ __forceinline__ float shift_a(float A, float s, float d) {
#pragma clang fp contract(off)
  const float sd = s * d;
  return A + sd;
}

// S and A of the segment relative to its maximum m, by the definition; for
// maxima whose exponents the fast sums cannot hold.
template <bool F32, int NT>
__device__ __forceinline__ Soft far_sums(const void* x, int64_t n, float m, float c) {
  Soft v{m, 0.0f, 0.0f};
  for (int64_t i = 8 * (int64_t)threadIdx.x; i < n; i += 8 * NT) {
    float f[8];
    load_logits<F32>(x, i, n, -INFINITY, f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = (f[k] - m) * c;
      const float e = __builtin_amdgcn_exp2f(d);
      v.s += e;
      v.a = fmaf(e, fmaxf(d, -1e4f), v.a);
    }
  }
  return v;
}

// What a row's (joined) sums give.
struct RowOut {
  float m, ls;
  bool empty;
};

// Target index (-1: not scored) and its logit, if that lies in the segment
// [first, first + n); thread 0 only.
struct TargetLogit {
  int64_t tg;
  float x;
};

template <bool F32>
__device__ __forceinline__ TargetLogit target_logit(const LogprobArgs& a, int64_t row, int64_t first, int64_t n) {
  TargetLogit r{-1, 0.0f};
  if (threadIdx.x == 0) {
    const void* x = logits_row<F32>(a, row);
    r.tg = row_target(a, row);
    if (first == 0 && a.dev_err && r.tg < 0 && a.targets[row] != a.ignore_index) atomicOr(a.dev_err, 8);
    if (r.tg >= first && r.tg < first + n)
      r.x = F32 ? static_cast<const float*>(x)[r.tg]
                : __uint_as_float((uint32_t)static_cast<const uint16_t*>(x)[r.tg] << 16);
  }
  return r;
}

// S >= 1 (it holds the maximum's own term 1) and A <= 0 but for rounding, which
// is kept from the entropy (by a comparison that leaves NaN alone).
__device__ __forceinline__ RowOut store_row(const LogprobArgs& a, int64_t row, Soft v, TargetLogit tl) {
  const bool empty = v.m == -INFINITY && v.s == 0.0f;
  const float ls = empty ? -INFINITY : logf(v.s);
  const float ent = ls - kLn2 * (v.a / v.s);
  if (threadIdx.x == 0) {
    a.logp[row] = tl.tg < 0 ? 0.0f : empty ? -INFINITY : (tl.x - v.m) * a.scale - ls;
    a.entropy[row] = empty || ent < 0.0f ? 0.0f : ent;
    a.stats_out[2 * row] = v.m;
    a.stats_out[2 * row + 1] = ls;
  }
  return RowOut{v.m, ls, empty};
}

constexpr int kMaxParts = 16;
constexpr int kJoinThreads = 256;

// What a segment leaves for the join: its sums and, if it holds the target, that
// logit (the join would read it behind the target's index, one latency later).
struct alignas(16) SegSums {
  Soft v;
  float xt;
};

// Joins the sums of a wave's first kMaxParts lanes, the segments of `seg` logits
// (every wave does the same work), and stores the row.
__device__ __forceinline__ RowOut join_row(const LogprobArgs& a, int64_t row, SegSums part, int64_t seg, float c) {
  Soft v = part.v;
  TargetLogit tl{row_target(a, row), 0.0f};
  tl.x = __shfl(part.xt, tl.tg < 0 ? 0 : (int)((uint32_t)tl.tg / (uint32_t)seg));
#pragma unroll
  for (int o = kMaxParts / 2; o >= 1; o >>= 1)
    v = soft_join(v, Soft{__shfl_xor(v.m, o), __shfl_xor(v.s, o), __shfl_xor(v.a, o)}, c);
  v = Soft{__shfl(v.m, 0), __shfl(v.s, 0), __shfl(v.a, 0)};
  return store_row(a, row, v, tl);
}

__device__ __forceinline__ void store_top(const LogprobArgs& a, int64_t row, const uint64_t* sorted, RowOut o) {
  const int t = threadIdx.x;
  if (t < a.top) {
    const uint64_t key = sorted[t];
    a.top_idx[row * a.top + t] = (int32_t)key_index(key);
    a.top_logp[row * a.top + t] = o.empty ? -INFINITY : (key_value(key) - o.m) * a.scale - o.ls;
  }
}

// A row's segments: `parts` of `seg` logits each (the last one shorter).
struct Split {
  int32_t parts;
  int64_t seg;
};

// Workspace of a split row: parts SegSums, then parts x top keys, 0 where a
// segment has fewer entries.
struct PartWork {
  SegSums* soft;
  uint64_t* keys;
};

__host__ __device__ inline int64_t soft_bytes(int64_t rows, int64_t parts) {
  return rows * parts * (int64_t)sizeof(SegSums);
}

__device__ __forceinline__ PartWork part_work(const LogprobArgs& a, const Split& sp) {
  char* w = static_cast<char*>(a.work);
  return PartWork{reinterpret_cast<SegSums*>(w), reinterpret_cast<uint64_t*>(w + soft_bytes(a.rows, sp.parts))};
}

template <bool F32, bool TOP, int NT, bool STREAM>
__global__ __launch_bounds__(NT) void k_logprob_part(LogprobPack pack) {
  const LogprobArgs a = pack.wide();
  const Split sp{pack.parts, pack.seg};
  constexpr int U = kUnroll<F32>;
  constexpr int kTile = 8 * U * NT, kWaves = NT / 64;
  __shared__ float red[3][kWaves];
  __shared__ std::conditional_t<TOP, TopLds<NT>, int> l;
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x / (unsigned)sp.parts;
  const int64_t part = blockIdx.x - row * sp.parts;
  const int64_t first = part * sp.seg;
  const int64_t n = min(sp.seg, a.vocab - first);
  const char* x = static_cast<const char*>(logits_row<F32>(a, row)) + first * (F32 ? 4 : 2);
  const float c = a.scale * kLog2e;
  const int tiles = (int)((n + kTile - 1) / kTile);
  const int per_slot = (tiles + kSlots - 1) / kSlots;

  float ref = kNoRef, s = 0.0f, A = 0.0f, tmax = -INFINITY, smax = -INFINITY;
  RawChunk<F32> cur[U], nxt[U];
  auto fetch = [&](int tile, RawChunk<F32> (&r)[U]) {
    const int64_t base = (int64_t)tile * kTile;
    if (base + kTile <= n) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        r[u] = load_raw<F32, STREAM>(x + (base + 8 * NT * u) * (F32 ? 4 : 2) + 8 * t * (F32 ? 4 : 2));
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[8];
        const int64_t i = base + 8 * (NT * u + t);
        if (i < n) load_logits<F32>(x, i, n, -INFINITY, f);
        else
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] = -INFINITY;
        if constexpr (F32) __builtin_memcpy(&r[u], f, 32);
        else r[u].w[0] = pack8(f);
      }
    }
  };
  fetch(0, cur);
  const TargetLogit tl = target_logit<F32>(a, row, first, n);
  int slot = 0, left = per_slot;
  for (int tile = 0; tile < tiles; ++tile) {
    if (tile + 1 < tiles) fetch(tile + 1, nxt);
    float f[U][8];
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (F32) __builtin_memcpy(f[u], &cur[u], 32);
      else unpack8(cur[u].w[0], f[u]);
      m = max_of(f[u], m);
    }
    if (m * c > ref + kRaise) {
      const float r = __builtin_rintf(m * c);
      const float d = ref - r;
      const float g = __builtin_amdgcn_exp2f(d);
      A = shift_a(A, s, d) * g;
      s *= g;
      ref = r;
    }
    float ts = 0.0f, ta = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float d = fmaf(f[u][k], c, -ref);
        const float e = __builtin_amdgcn_exp2f(d);
        ts += e;
        ta = fmaf(e, fmaxf(d, -1e4f), ta);
      }
    s += ts;
    A += ta;
    smax = fmaxf(smax, m);
    if (--left == 0 || tile + 1 == tiles) {
      tmax = fmaxf(tmax, smax);
      if constexpr (TOP) l.slot[slot][t] = (uint16_t)key16(smax);
      smax = -INFINITY;
      left = per_slot;
      ++slot;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) cur[u] = nxt[u];
  }

  float M = tmax;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor(M, o));
  if ((t & 63) == 0) red[0][t >> 6] = M;
  __syncthreads();
  M = red[0][0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) M = fmaxf(M, red[0][i]);
  Soft v;
  if (M != -INFINITY && !(fabsf(M) * c <= kFarExp)) {
    v = far_sums<F32, NT>(x, n, M, c);
  } else {
    // relative to M itself: divided by M's own term, which the sums hold with
    // these very bits. So S is never below 1, and exactly 1 (A exactly 0) where one
    // token is left; a factor 2^(r - M c) would be a second rounded exponential, with
    // log probabilities an ulp above 0. (Infinite where all of a thread's terms
    // are 0.)
    const float base = M == -INFINITY ? 0.0f : M;
    const float d = fmaf(base, c, -ref);
    const float e = __builtin_amdgcn_exp2f(d);
    v = Soft{M, s / e, shift_a(A, s, -d) / e};
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    v.s += __shfl_xor(v.s, o);
    v.a += __shfl_xor(v.a, o);
  }
  if ((t & 63) == 0) {
    red[1][t >> 6] = v.s;
    red[2][t >> 6] = v.a;
  }
  __syncthreads();
  v.s = red[1][0];
  v.a = red[2][0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) {
    v.s += red[1][i];
    v.a += red[2][i];
  }

  if constexpr (TOP) find_top<F32, NT>(l, x, n, (uint32_t)first, tmax, !(v.s == v.s), slot, per_slot, a.top);
  if (sp.parts == 1) {
    const RowOut o = store_row(a, row, v, tl);
    if constexpr (TOP) store_top(a, row, l.cand, o);
  } else {
    const PartWork w = part_work(a, sp);
    if (t == 0) w.soft[row * sp.parts + part] = SegSums{v, tl.x};
    if constexpr (TOP) {
      if (t < a.top) w.keys[(row * sp.parts + part) * a.top + t] = t < l.count ? l.cand[t] : 0;
    }
  }
}


// One workgroup per row. The alternatives: the top-th largest of the lists'
// first entries (`lead` of each, at least `top` in all) bounds the result from
// below; what reaches it, rarely many more than `top`, is ranked. All loads of
// global memory are issued at the start: the kernel is a chain of latencies.
template <bool TOP>
__global__ __launch_bounds__(kJoinThreads) void k_logprob_join(LogprobPack pack) {
  const LogprobArgs a = pack.wide();
  const Split sp{pack.parts, pack.seg};
  const int t = threadIdx.x, lane = t & 63;
  const int64_t row = blockIdx.x;
  const PartWork w = part_work(a, sp);
  const float c = a.scale * kLog2e;
  SegSums v{{-INFINITY, 0.0f, 0.0f}, 0.0f};
  if (lane < sp.parts) v = w.soft[row * sp.parts + lane];
  if constexpr (TOP) {
    __shared__ uint64_t keys[kMaxParts * kMaxTop], cand[kMaxParts * kMaxTop], best[kMaxTop];
    __shared__ uint64_t bound;
    __shared__ int count;
    const int total = sp.parts * a.top;
    const uint64_t* src = w.keys + row * total;
    for (int i = t; i < total; i += kJoinThreads) keys[i] = src[i];
    if (t == 0) {
      bound = 1;
      count = 0;
    }
    const RowOut o = join_row(a, row, v, sp.seg, c);
    const int lead = min((2 * a.top + sp.parts - 1) / sp.parts, a.top);
    const int leads = lead * sp.parts;   // at most 2 top + parts
    __syncthreads();
    uint64_t k0 = 0;
    if (t < leads) cand[t] = k0 = keys[(t / lead) * a.top + t % lead];
    __syncthreads();
    if (t < leads && k0 && count_larger(cand, leads, k0) == a.top - 1) bound = k0;
    __syncthreads();
    const uint64_t b = bound;
    for (int i = t; i < total; i += kJoinThreads) {
      const uint64_t k = keys[i];
      if (k >= b) cand[atomicAdd(&count, 1)] = k;
    }
    __syncthreads();
    const int n = count;
    for (int i = t; i < n; i += kJoinThreads) {
      const uint64_t k = cand[i];
      const int r = count_larger(cand, n, k);
      if (r < a.top) best[r] = k;
    }
    __syncthreads();
    store_top(a, row, best, o);
  } else {
    join_row(a, row, v, sp.seg, c);
  }
}

// ---------------------------------------------------------------- backward

// With l_j = (x_j - m) scale - ls, p_j = e^l_j, the gradient is
//   scale (dlogp ([j = target] - p_j) - dent p_j (l_j + entropy)).
// In base 2, with c = scale log2(e) and K = m c + ls log2(e), p = 2^(x c - K).
// The exponent is some 20 in size, where a float32 is spaced 2^-19: rounding it
// would leave p off by 2^-20, ten times an ulp, and a probability's error
// decides which way values next to a rounding border go (a block's scale can
// hang on one). So K = ki + kf with ki an integer, and with the integer n next
// to x c - ki (it appears in the low bits of w = x c - ki + 1.5 * 2^23, one
// fused multiply-add), f = x c - (ki + n), about 1/2 in size, is another one:
// p = 2^f 2^n 2^-kf, where 2^n is added to the exponent field and 2^-kf is
// folded into the row's constants. What c lost when it was rounded to float32,
// c (1 + r), would add r x c to the exponent; K takes its value at p = 2^-16, and
// what is left, r (16 + log2 p), is 2^-20 at most (2^-22 for scale 1), at p near 1.
//
// The kernel is as close to its VALU issue rate as to HBM's: these 11 slots a
// logit (4 of them v_exp_f32) in place of 14, with c's correction and the scaling
// by 2^n as instructions of their own, took 4096 x 131072 from 429 to 407 us (399
// now, 5.5 TB/s).
//
// The exponent field holds n + up, and the constants the factor 2^-up; x is
// bounded below where n + up is -122, so that a masked entry stays a number. up
// follows the size of the row's gradient, 2^(up - 60): the constants are then about
// 2^-60, far from float32's ends, and a masked entry gives 2^-180, 0 in bf16 (up is
// at most 124, for fields up to 252: exact zeros up to 2^100). A NaN among the logits
// has made the row's statistics NaN, and with them every constant.
//
// l_j is formed from x c as well, so rows whose m c is large (at the extreme, all
// entries at the lowest finite value) take their differences from m first: base =
// m, else 0. So do rows in which the two parts of k1 x + k0 are far larger than what
// they leave at x = m: those that only the entropy reaches and where one token holds
// nearly all of the probability, with l + entropy a few times 1e-4 there.
struct RowLine {
  float low;         // bound of x - base
  float mk;          // 1.5 * 2^23 + up - ki
  float k1, k0;      // gradient = 2^f 2^(n + up) (k1 (x - base) + k0)
  int32_t target;    // column within the tile, out of [0, 128) if elsewhere
  float base;
};
struct GradRow : RowLine {
  float at;          // the gradient at the target, formed by other waves than the rest
};

// The gradient at the target itself,
//   scale dlogp (1 - p) - scale dent p (l + entropy),
// cancels where p is near 1, as well-predicted targets have it: 1 - p taken from
// the p above would keep few digits of it (an error of 1 to 5% at 1 - p = 6e-6). So
// it is formed once a row, from l = (x - m) scale - ls, whose two parts have one
// sign and which is as exact as they are, and 1 - e^l. dlogp, dent: times scale.
__device__ __forceinline__ float target_value(float x, float m, float ls, float scale, float dlogp, float dent,
                                              float entropy) {
  float l = fmaf(x - m, scale, -ls);
  l = l < -1e4f ? -1e4f : l;               // keeps NaN; e^l is 0 from -104 on
  // 1 - e^l: above -ln 2 by its power series (what follows l^9 / 9! is below 2^-26
  // of it), below by e^l <= 1/2, which costs no digits
  float q = 1.0f / 362880;
  q = fmaf(q, l, 1.0f / 40320);
  q = fmaf(q, l, 1.0f / 5040);
  q = fmaf(q, l, 1.0f / 720);
  q = fmaf(q, l, 1.0f / 120);
  q = fmaf(q, l, 1.0f / 24);
  q = fmaf(q, l, 1.0f / 6);
  q = fmaf(q, l, 0.5f);
  q = -l * fmaf(q, l, 1.0f);
  const float e = exp_nonpos(l);
  const bool near = l > -0.6931f;
  const float p = near ? 1.0f - q : e;
  q = near ? q : 1.0f - e;
  return fmaf(dlogp, q, -dent * (p * (l + entropy)));
}

constexpr float kMagic = 12582912.0f;      // 1.5 * 2^23
constexpr float kFarRow = 1024.0f;         // |m c| from which base = m,
constexpr float kFarSum = 256.0f;          // and |k1 m| in its sum with k0: 2^-24 |k0| is then 2^-16 of the sum
constexpr double kAt = -16.0;              // log2 p where c's rounding is made up for

// up for a gradient of this size (any bits: infinity and NaN count as 2^128).
__device__ __forceinline__ int grad_up(float size) {
  return min((int)((__float_as_uint(size) >> 23) & 255) - 127 + 60, 124);
}

template <bool FAR>
__device__ __forceinline__ float grad_value(float x, const GradRow& g, float c) {
  const float y = fmaxf(FAR ? x - g.base : x, g.low);
  const float w = fmaf(y, c, g.mk);
  const float f = fmaf(y, c, g.mk - w);    // mk - w = -(ki + n), exactly
  const uint32_t p = __float_as_uint(__builtin_amdgcn_exp2f(f)) + (__float_as_uint(w) << 23);
  return fmaf(__uint_as_float(p), fmaf(y, g.k1, g.k0), 0.0f);
}

// What a row's gradient is formed from. A missing operand's load is issued as
// well (of an entropy), which keeps all of them in flight together: behind
// branches they wait for each other, 57.6 us in place of 53.3 at 1024 x 50304
// float32.
struct RowIn {
  int64_t target;                      // -1: not scored
  bool outside;                        // not in the vocabulary
  float m, ls, dlogp, dent, entropy;   // dlogp 0 if not scored, entropy 0 without dent
};

__device__ __forceinline__ RowIn row_in(const LogprobArgs& a, int64_t row) {
  const int64_t t = a.targets[row];
  const float2 stats = reinterpret_cast<const float2*>(a.stats)[row];
  const float d = (a.dlogp ? a.dlogp : a.ent_in)[row], e = (a.dent ? a.dent : a.ent_in)[row], h = a.ent_in[row];
  const bool in = t >= 0 && t < a.vocab, scored = in && t != a.ignore_index;
  return RowIn{scored ? t : -1, !in && t != a.ignore_index, stats.x, stats.y, scored && a.dlogp ? d : 0.0f,
               a.dent ? e : 0.0f, a.dent ? h : 0.0f};
}

template <bool F32, bool FAR>
__device__ __forceinline__ uint4 grad_chunk(RawChunk<F32> raw, const GradRow& row, float c, uint32_t col) {
  // one chunk after the other: left to interleave four of them, the compiler
  // takes 82 VGPRs, too many for a fourth tile on the CU (495 us against 460 at
  // 4096 x 131072)
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i)
    asm volatile("" : "+v"(raw.w[i].x), "+v"(raw.w[i].y), "+v"(raw.w[i].z), "+v"(raw.w[i].w) : : "memory");
  const GradRow g = row;
  float f[8];
  if constexpr (F32) __builtin_memcpy(f, &raw, 32);
  else unpack8(raw.w[0], f);
  const uint32_t hit = (uint32_t)g.target - col;
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = grad_value<FAR>(f[k], g, c);
  uint4 v = pack8(f);
  if (hit < 8) {
    const uint32_t t = pack_bf16x2(g.at, g.at), sel = hit & 1 ? 0x05040100u : 0x03020504u;
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = (int)(hit >> 1) == k ? __builtin_amdgcn_perm(t, w[k], sel) : w[k];
  }
  asm volatile("" : "+v"(v.x), "+v"(v.y), "+v"(v.z), "+v"(v.w));
  return v;
}

// What goes past the Infinity Cache (256 MB) on its way, see launch_logprob_bwd.
enum GradKind {
  kGradSmall,    // the row-wise codes
  kGradLarge,    // and the column-wise ones
  kGradStream,   // and the logits
};

template <class F, bool F32, GradKind KIND, bool FULL>
__device__ __forceinline__ void logprob_bwd_tile(const LogprobArgs& a, TileLds& l, GradRow* rows, bool* far_rows,
                                                 int64_t r0, int64_t c0, int rows_valid, int rows_pad, int cols_valid, int cols_pad) {
  constexpr int kB = F32 ? 4 : 2;
  const uint32_t t = threadIdx.x, cc = t & 15, tr = t >> 4;
  const double cd = (double)a.scale * kLog2eD;
  const float c = (float)cd;
  const char* base = static_cast<const char*>(a.x) + (r0 * a.ld + c0) * kB;
  RawChunk<F32> raw[kChunks];
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    if constexpr (FULL) {
      raw[j] = load_raw<F32, KIND == kGradStream>(base + (int64_t)(kRowStep * j) * a.ld * kB +
                                                  (tr * (uint32_t)a.ld + cc * 8) * kB);
    } else {
      float f[8];
      const int row = tr + kRowStep * j;
      if (row < rows_valid && (int)cc * 8 < cols_valid)
        load_logits<F32>(base + row * a.ld * kB, cc * 8, cols_valid, -INFINITY, f);
      else
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = -INFINITY;
      if constexpr (F32) __builtin_memcpy(&raw[j], f, 32);
      else raw[j].w[0] = pack8(f);
    }
  }
  bool row_far = false;
  if ((int)t < kTR) {
    RowLine g{};
    g.mk = kMagic;
    g.target = -1;
    if (FULL || (int)t < rows_valid) {
      const RowIn in = row_in(a, r0 + t);
      const float m = in.m, ls = in.ls;
      if (c0 == 0 && a.dev_err && in.outside) atomicOr(a.dev_err, 8);
      if (!(m == -INFINITY && ls == -INFINITY)) {   // a row with nothing left has gradient 0
        // first what does not need K (the registers for all of it at once would
        // spill, with the tile's logits in flight): k1, and the value at x = m
        const int up = grad_up(a.scale * (fabsf(in.dlogp) + 1024.0f * fabsf(in.dent)));   // |l + entropy| reaches some 1000
        const float unit = ldexpf(1.0f, -up), dent = in.dent * unit;
        g.k1 = -a.scale * (a.scale * dent);
        const float at_m = -a.scale * fmaf(dent, in.entropy - ls, in.dlogp * unit);
        row_far = !(fabsf(m) * c <= kFarRow && fabsf(g.k1 * m) <= kFarSum * fabsf(at_m));
        g.k0 = (float)fma(-(double)g.k1, row_far ? 0.0 : (double)m, (double)at_m);
        asm volatile("" : "+v"(g.k1), "+v"(g.k0));
        const float rc = __builtin_amdgcn_rcpf(c);
        double K = fma(row_far ? 0.0 : (double)m, cd, (double)ls * kLog2eD);
        K -= (K + kAt) * (double)((float)(cd - (double)c) * rc);
        const double ki = rint(K);
        const float fold = __builtin_amdgcn_exp2f((float)(ki - K));
        g.low = ((float)ki - (float)(up + 122)) * rc;
        g.mk = kMagic + (float)up - (float)ki;
        g.k1 *= fold;
        g.k0 *= fold;
        g.base = row_far ? m : 0.0f;
        g.target = in.target >= c0 && in.target < c0 + kTC ? (int32_t)(in.target - c0) : -1;
      }
    }
    static_cast<RowLine&>(rows[t]) = g;
  } else if ((int)t < 2 * kTR && (FULL || (int)t - kTR < rows_valid)) {   // waves without a row: the targets' own values
    const RowIn in = row_in(a, r0 + t - kTR);
    if (in.target >= c0 && in.target < c0 + kTC) {
      float x[1];
      load_logits<F32>(logits_row<F32>(a, r0 + t - kTR), in.target, a.vocab, 0.0f, x);
      rows[t - kTR].at = target_value(x[0], in.m, in.ls, a.scale, a.scale * in.dlogp, a.scale * in.dent, in.entropy);
    }
  }
  if ((int)t < kTR) {
    const bool any = __any(row_far);
    if ((t & 63) == 0) far_rows[t >> 6] = any;
  }
  __syncthreads();
  const bool far = __builtin_amdgcn_readfirstlane(far_rows[0] | far_rows[1]);
  uint4 v[kChunks];
  if (!far) {
#pragma unroll
    for (int j = 0; j < kChunks; ++j) v[j] = grad_chunk<F32, false>(raw[j], rows[tr + kRowStep * j], c, cc * 8);
  } else {
#pragma unroll
    for (int j = 0; j < kChunks; ++j) v[j] = grad_chunk<F32, true>(raw[j], rows[tr + kRowStep * j], c, cc * 8);
  }
  if constexpr (!FULL) {   // rows and columns that only fill up: +0
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int left = (int)(tr + kRowStep * j) < rows_valid ? cols_valid - (int)cc * 8 : 0;
      uint32_t* w = reinterpret_cast<uint32_t*>(&v[j]);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = left >= 2 * k + 2 ? w[k] : left == 2 * k + 1 ? w[k] & 0xFFFFu : 0u;
    }
  }
  fmt_dual<F, FULL, true, KIND != kGradSmall>(v, l, rows_valid, rows_pad, cols_pad,
                                 TileOut{a.q_row, a.s_row, a.vocab_pad, a.rows, F::k128},
                                 TileOut{a.q_col, a.s_col, a.rows_pad, a.vocab_pad, F::k128}, r0, c0, false);
}

template <class F, bool F32, GradKind KIND>
__global__ __launch_bounds__(kFmtThreads, F32 ? 6 : 8) void k_logprob_bwd(LogprobBwdPack pack) {
  __shared__ TileLds l;
  __shared__ GradRow rows[kTR];
  __shared__ bool far_rows[kTR / 64];
  const LogprobArgs a = pack.wide<F>();
  const TilePos at = tile_pos(blockIdx.x, (uint32_t)((a.vocab_pad + kTC - 1) / kTC), (uint32_t)((a.rows_pad + kTR - 1) / kTR),
                              a.bands);
  const int64_t r0 = at.r0, c0 = at.c0;
  const int rows_valid = (int)min<int64_t>(kTR, a.rows - r0);
  const int rows_pad = (int)min<int64_t>(kTR, a.rows_pad - r0);
  const int cols_valid = (int)min<int64_t>(kTC, a.vocab - c0);
  const int cols_pad = (int)min<int64_t>(kTC, a.vocab_pad - c0);
  if (rows_valid == kTR && cols_valid == kTC)
    logprob_bwd_tile<F, F32, KIND, true>(a, l, rows, far_rows, r0, c0, kTR, kTR, kTC, kTC);
  else
    logprob_bwd_tile<F, F32, KIND, false>(a, l, rows, far_rows, r0, c0, rows_valid, rows_pad, cols_valid, cols_pad);
}

// ---------------------------------------------------------------- launch

// A row is split over the vocabulary, into up to 16 segments of at least 8192
// logits, where rows are few and long: the join costs a launch and 4 us. One
// row of 131072 with 20 alternatives takes 11.0 us in 16 segments and 15.4
// whole, 64 such rows 14.2 and 16.6, 128 rows 17.5 and 17.1; 200 rows with 5 are
// slower in segments (19.7 against 17.5), and so are rows of up to 65536 (84 x
// 48907 13.9 against 12.0, one row of 50000 11.8 against 11.1).
static Split split_rows(int64_t rows, int64_t vocab) {
  int64_t parts = 1;
  if (rows <= 128 && vocab > 65536)
    while (parts < kMaxParts && rows * parts < 1024 && vocab / (2 * parts) >= 8192) parts *= 2;
  const int64_t seg = ((vocab + parts - 1) / parts + 7) / 8 * 8;
  return Split{(int32_t)((vocab + seg - 1) / seg), seg};
}

// Threads of a workgroup: 512 where every CU gets at most one of them and its
// segment is long (200 x 131072: 17.5 us against 21.4 with 256, 84 x 48907 12.2
// against 13.0), else 256 (500 x 131072: 26.9 against 29.5 with 512, 128 x 8520
// 6.9 against 7.4).
static bool wide_groups(int64_t groups, int64_t seg) { return groups <= 256 && seg >= 32768; }

// Logits that the Infinity Cache (256 MB) cannot hold are not kept there: 4096 x
// 131072 197 -> 192 us, 3000 x 50001 76 -> 74.6 (200 x 131072, which it can hold,
// 17.7 -> 19.8 where it does).
static bool past_caches(const LogprobArgs& a) { return a.rows * a.vocab * (a.f32 ? 4 : 2) > (1ll << 28); }

int64_t logprob_work(int64_t rows, int64_t vocab, int32_t top) {
  const Split sp = split_rows(rows, vocab);
  return sp.parts == 1 ? 0 : soft_bytes(rows, sp.parts) + rows * sp.parts * top * (int64_t)sizeof(uint64_t);
}

template <bool F32, bool TOP>
static hipError_t launch_fwd(const LogprobArgs& a, hipStream_t s) {
  const Split sp = split_rows(a.rows, a.vocab);
  const dim3 grid((unsigned)(a.rows * sp.parts));
  const LogprobPack p{a.x, a.targets, a.dev_err, a.logp, a.entropy, a.stats_out, a.top_logp, a.top_idx, a.work,
                      a.ignore_index, a.ld, (int32_t)a.rows, (int32_t)a.vocab, a.top, a.scale, sp.parts,
                      (int32_t)sp.seg};
  if (wide_groups(a.rows * sp.parts, sp.seg))
    hipLaunchKernelGGL((k_logprob_part<F32, TOP, 512, false>), grid, dim3(512), 0, s, p);
  else if (past_caches(a))
    hipLaunchKernelGGL((k_logprob_part<F32, TOP, 256, true>), grid, dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((k_logprob_part<F32, TOP, 256, false>), grid, dim3(256), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || sp.parts == 1) return e;
  hipLaunchKernelGGL(k_logprob_join<TOP>, dim3((unsigned)a.rows), dim3(kJoinThreads), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_logprob_fwd(const LogprobArgs& a, hipStream_t s) {
  if (a.f32) return a.top ? launch_fwd<true, true>(a, s) : launch_fwd<true, false>(a, s);
  return a.top ? launch_fwd<false, true>(a, s) : launch_fwd<false, false>(a, s);
}

// Bands (tile_pos) for large gradients whose rows are aligned: their pitch
// sends the 128 rows of a tile to few memory channels at a time, and eight
// bands spread that. 4096 x 131072 495 -> 399 us, 8192 x 65536 509 -> 398,
// 4096 x 50304 float32 246 -> 244; without it smaller gradients are faster
// (8192 x 16384 107 against 124 us, 2048 x 131072 float32 295 against 318), and
// so are unaligned rows (6000 x 100001 457 against 509).
static bool aligned_rows(const LogprobArgs& a) {
  return a.ld * (a.f32 ? 4 : 2) % 16 == 0 && reinterpret_cast<uintptr_t>(a.x) % 16 == 0;
}

static bool grad_bands(const LogprobArgs& a, int64_t nx, int64_t ny) {
  return nx * ny >= 48 * 256 && ny >= 32 && aligned_rows(a);
}

// Where each direction's codes are past what the 256 MB Infinity Cache can hold
// for the head's gradient GEMMs, both go past it: 4096 x 131072 434 -> 425 us; and
// so do the logits, read here for the last time, where no line is shared by two
// tiles: 425 -> 399 (6000 x 100001, unaligned, 457 against 552 with them). Below that
// size only the row-wise codes do: 333 x 50001 float32 24.2 -> 22.8 us, 1000 x 32000
// 32.2 -> 31.5; the column-wise ones gain the kernel nothing more (22.8), and cost
// the two GEMMs behind it 3 us (7 us behind 1000 x 32000).
static GradKind grad_kind(const LogprobArgs& a) {
  if (a.rows_pad * a.vocab_pad <= (1ll << 28)) return kGradSmall;
  return aligned_rows(a) ? kGradStream : kGradLarge;
}

template <class F, bool F32>
static void launch_bwd(const LogprobArgs& a, dim3 grid, hipStream_t s) {
  const LogprobBwdPack p{a.x, a.targets, a.dev_err, a.stats, a.ent_in, a.dlogp, a.dent, a.q_row, a.s_row, a.q_col,
                         a.s_col, a.ignore_index, (uint32_t)(2 * a.ld + a.bands), (int32_t)a.rows, (int32_t)a.vocab,
                         a.scale};
  switch (grad_kind(a)) {
    case kGradSmall: hipLaunchKernelGGL((k_logprob_bwd<F, F32, kGradSmall>), grid, dim3(kFmtThreads), 0, s, p); break;
    case kGradLarge: hipLaunchKernelGGL((k_logprob_bwd<F, F32, kGradLarge>), grid, dim3(kFmtThreads), 0, s, p); break;
    case kGradStream: hipLaunchKernelGGL((k_logprob_bwd<F, F32, kGradStream>), grid, dim3(kFmtThreads), 0, s, p); break;
  }
}

hipError_t launch_logprob_bwd(const LogprobArgs& args, hipStream_t s) {
  LogprobArgs a = args;
  const int64_t nx = (a.vocab_pad + kTC - 1) / kTC, ny = (a.rows_pad + kTR - 1) / kTR;
  a.bands = grad_bands(a, nx, ny);
  const dim3 grid((unsigned)(nx * ny));
  with_fmt(a.rceil, a.k128, [&](auto f) {
    if (a.f32) launch_bwd<decltype(f), true>(a, grid, s);
    else launch_bwd<decltype(f), false>(a, grid, s);
  });
  return hipGetLastError();
}

}  // namespace mxk
