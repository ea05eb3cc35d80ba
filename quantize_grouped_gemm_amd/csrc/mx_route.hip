// Routing of tokens to experts and its gradient.
//
// Which experts a token goes to is decided by float32 scores that are the
// nearest to softmax or sigmoid of the logits: two of them that lie next to
// each other would otherwise be ordered by the rounding of whatever computes
// them. They are formed in float64 (errors of some 2^-50, which take about one score in
// 2^25 to the neighbour of its nearest float32) and rounded once;
// choice values are the float32 sum of score and bias. Float64 costs what
// float32 does here (16 lanes a clock): a score takes about 30 instructions.
//
// A token's experts live in the registers of LPT lanes, PER consecutive ones
// each, as sortable integers: the largest is found with row-wise lane
// exchanges, ties go to the lowest lane and there to the lowest register, so to
// the lowest expert.
// (Sorting a lane's experts first, as float64 that hold key and number, and moving
// the winner's next one up was slower: maxima of float64 take four times as long,
// 17.5 against 12.3 us for 16384 tokens to 8 of 256.)
// The vector unit bounds all of it: 16384 tokens to 8 of 256 in 4 of 8 groups 13.8 us,
// one token 4.3; the gradient of 8191 x 96 logits 5.3 us, of 16384 x 256 in float32 13.8
// (sigmoid) and 16.8 (softmax).

#include <cmath>

#include "mx_device.h"
#include "mx_moe.h"

namespace mxk {

constexpr int kRouteThreads = 256;
constexpr int32_t kOut = INT32_MIN;   // key of an expert that is ruled out

// An integer that orders like the float; every NaN above +infinity. -infinity
// stands for "ruled out".
__device__ __forceinline__ int32_t sort_key(float c) {
  const int32_t b = __float_as_int(c);
  const int32_t k = b ^ ((b >> 31) & 0x7FFFFFFF);
  return c != c ? 0x7FC00000 : c == -INFINITY ? kOut : k;
}

__device__ __forceinline__ float key_value(int32_t k) { return __int_as_float(k ^ ((k >> 31) & 0x7FFFFFFF)); }

template <int CTRL>
__device__ __forceinline__ int32_t dpp_i(int32_t v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}

template <int CTRL>
__device__ __forceinline__ double dpp_d(double v) {
  const int64_t b = __double_as_longlong(v);
  const uint32_t lo = (uint32_t)dpp_i<CTRL>((int32_t)b), hi = (uint32_t)dpp_i<CTRL>((int32_t)(b >> 32));
  return __longlong_as_double((int64_t)(((uint64_t)hi << 32) | lo));
}

// Over the LPT lanes of a token (16: quad permutes, half and whole row
// mirrors; 64: then across the rows); every lane gets the same value.
template <int LPT>
__device__ __forceinline__ int32_t all_max(int32_t v) {
  v = max(v, dpp_i<0xB1>(v));
  v = max(v, dpp_i<0x4E>(v));
  v = max(v, dpp_i<0x141>(v));
  v = max(v, dpp_i<0x140>(v));
  if constexpr (LPT == 64) {
    // the last lane of each row passes its row's on, so that lane 63 holds all four
    v = max(v, __builtin_amdgcn_update_dpp(INT32_MIN, v, 0x142, 0xA, 0xF, false));
    v = max(v, __builtin_amdgcn_update_dpp(INT32_MIN, v, 0x143, 0xC, 0xF, false));
    v = __builtin_amdgcn_readlane(v, 63);
  }
  return v;
}

template <int LPT>
__device__ __forceinline__ double all_sum(double v) {
  v += dpp_d<0xB1>(v);
  v += dpp_d<0x4E>(v);
  v += dpp_d<0x141>(v);
  v += dpp_d<0x140>(v);
  if constexpr (LPT == 64) {
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
  }
  return v;
}

// The lanes of this token for which p holds, as bits.
template <int LPT>
__device__ __forceinline__ uint64_t token_ballot(bool p) {
  const uint64_t b = __ballot(p);
  if constexpr (LPT == 64) return b;
  return (b >> (threadIdx.x & 48)) & 0xFFFFu;
}

// What lanes of this wave wrote to LDS before is seen by the others after it.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Logits e0 .. e0 + PER - 1 of a row; -infinity past the last one.
template <int PER, bool F32>
__device__ __forceinline__ void load_logits(float (&x)[PER], const void* row, int e0, int E, bool vec) {
  if (vec && e0 + PER <= E) {
    constexpr int kBytes = PER * (F32 ? 4 : 2);
    if constexpr (kBytes >= 4) {
      uint32_t w[kBytes / 4];
      const char* p = reinterpret_cast<const char*>(row) + (int64_t)e0 * (F32 ? 4 : 2);
      if constexpr (kBytes >= 16) {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) {
          const uint4 q = reinterpret_cast<const uint4*>(p)[i];
          w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
        }
      } else if constexpr (kBytes == 8) {
        const uint2 q = *reinterpret_cast<const uint2*>(p);
        w[0] = q.x; w[1] = q.y;
      } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if constexpr (F32) x[i] = __uint_as_float(w[i]);
        else x[i] = i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = e0 + i;
    if constexpr (F32) x[i] = e < E ? reinterpret_cast<const float*>(row)[e] : -INFINITY;
    else x[i] = e < E ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[e] << 16) : -INFINITY;
  }
}

// exp(t) in float64 for |t| <= 710 (NaN stays NaN), off by some 2^-50: t = n ln2 / 32 +
// r, e^t = 2^(n div 32) 2^((n mod 32) / 32) e^r with the powers from a table in LDS
// and e^r, |r| <= 0.011, by its series up to r^6. 17 instructions, where the
// library's function without a table takes 25.
__constant__ double kPow2[32] = {
    0x1.0000000000000p+0, 0x1.059b0d3158574p+0, 0x1.0b5586cf9890fp+0, 0x1.11301d0125b51p+0,
    0x1.172b83c7d517bp+0, 0x1.1d4873168b9aap+0, 0x1.2387a6e756238p+0, 0x1.29e9df51fdee1p+0,
    0x1.306fe0a31b715p+0, 0x1.371a7373aa9cbp+0, 0x1.3dea64c123422p+0, 0x1.44e086061892dp+0,
    0x1.4bfdad5362a27p+0, 0x1.5342b569d4f82p+0, 0x1.5ab07dd485429p+0, 0x1.6247eb03a5585p+0,
    0x1.6a09e667f3bcdp+0, 0x1.71f75e8ec5f74p+0, 0x1.7a11473eb0187p+0, 0x1.82589994cce13p+0,
    0x1.8ace5422aa0dbp+0, 0x1.93737b0cdc5e5p+0, 0x1.9c49182a3f090p+0, 0x1.a5503b23e255dp+0,
    0x1.ae89f995ad3adp+0, 0x1.b7f76f2fb5e47p+0, 0x1.c199bdd85529cp+0, 0x1.cb720dcef9069p+0,
    0x1.d5818dcfba487p+0, 0x1.dfc97337b9b5fp+0, 0x1.ea4afa2a490dap+0, 0x1.f50765b6e4540p+0};

__device__ __forceinline__ double exp64(double t, const double* pow2) {
  const double n = rint(t * 0x1.71547652b82fep+5);
  double r = fma(n, -0x1.62e42ff000000p-6, t);
  r = fma(n, 0x1.718432a1b0e26p-40, r);
  const int i = (int)n;
  double p = fma(r, 1.0 / 720, 1.0 / 120);
  p = fma(r, p, 1.0 / 24);
  p = fma(r, p, 1.0 / 6);
  p = fma(r, p, 0.5);
  p = fma(r, p, 1.0);
  p = fma(r, p, 1.0);
  return ldexp(p * pow2[i & 31], i >> 5);
}

// 1 / v for 1 <= v < 2^1020 (or NaN): the hardware's approximation and two Newton steps.
__device__ __forceinline__ double inverse64(double v) {
  double y = __builtin_amdgcn_rcp(v);
  y = fma(fma(-v, y, 1.0), y, y);
  return fma(fma(-v, y, 1.0), y, y);
}

// Beyond +-700 the score is 1 or 0 as a float32 all the same.
__device__ __forceinline__ double sigmoid64(float x, const double* pow2) {
  const float c = x < -700.0f ? -700.0f : x > 700.0f ? 700.0f : x;
  return inverse64(1.0 + exp64(-(double)c, pow2));
}

// exp(x - max) of the lane's logits and the inverse of their sum over the row (1
// where no logit is left, so that every score is 0).
template <int LPT, int PER>
__device__ __forceinline__ double softmax64(const float (&x)[PER], double (&p)[PER], double& m, const double* pow2) {
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) mx = fmaxf(mx, x[i]);
  // no NaN in mx: the integer order is the float's
  const int32_t b = __float_as_int(mx);
  const int32_t k = all_max<LPT>(b ^ ((b >> 31) & 0x7FFFFFFF));
  mx = key_value(k);
  m = mx == -INFINITY ? 0.0 : (double)mx;
  double t = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    // e^-700 is 0 as a score, and nothing beside the largest logit's 1
    const double d = (double)x[i] - m;
    p[i] = exp64(d < -700.0 ? -700.0 : d, pow2);
    t += p[i];
  }
  t = all_sum<LPT>(t);
  return mx == -INFINITY ? 1.0 : inverse64(t);
}

__device__ __forceinline__ void load_pow2(double* pow2) {
  if (threadIdx.x < 32) pow2[threadIdx.x] = kPow2[threadIdx.x];
  __syncthreads();
}

template <int LPT, int PER, bool F32>
__global__ __launch_bounds__(kRouteThreads) void k_route(RouteArgs a, bool vec) {
  constexpr int kTokens = kRouteThreads / LPT;
  __shared__ double pow2[32];
  __shared__ float c_lds[kTokens][LPT * PER];   // choice keys, where groups straddle lanes; then the scores
  __shared__ int32_t g_lds[kTokens][kMaxExpertGroups];
  __shared__ int32_t i_lds[kTokens][kMaxTopExperts];
  const int lane = threadIdx.x % LPT, tok = threadIdx.x / LPT;
  const int64_t t = (int64_t)blockIdx.x * kTokens + tok;
  const bool live = t < a.rows;
  const int64_t row = live ? t : a.rows - 1;   // idle lanes repeat the last row: exchanges need whole waves
  const int E = a.experts, e0 = lane * PER;
  float x[PER], s[PER];
  load_logits<PER, F32>(x, reinterpret_cast<const char*>(a.x) + row * a.ld * (F32 ? 4 : 2), e0, E, vec);
  load_pow2(pow2);
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < PER; ++i) s[i] = (float)sigmoid64(x[i], pow2);
  } else {
    double p[PER], m;
    const double inv = softmax64<LPT, PER>(x, p, m, pow2);
#pragma unroll
    for (int i = 0; i < PER; ++i) s[i] = (float)(p[i] * inv);
  }
  int32_t key[PER];
  if (a.bias) {
    float b[PER];
    load_logits<PER, true>(b, a.bias, e0, E, (reinterpret_cast<uintptr_t>(a.bias) & 15) == 0);
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = sort_key(x[i] == -INFINITY ? -INFINITY : s[i] + b[i]);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = sort_key(x[i] == -INFINITY ? -INFINITY : s[i]);
  }

  if (a.top_groups < a.groups) {
    // group values: the largest choice value, or the sum of the two largest
    // that are not ruled out
    const int G = a.groups, gs = E / G, span = gs / PER;
    const bool whole = gs % PER == 0 && (span & (span - 1)) == 0 && span <= 16;
    const int shift = __builtin_ctz(max(span, 1));
    if (whole) {
      // a lane's experts belong to one group, whose lanes are neighbours
      int32_t k1 = kOut, k2 = kOut;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        k2 = max(k2, min(k1, key[i]));
        k1 = max(k1, key[i]);
      }
      auto join = [&](int32_t o1, int32_t o2) {
        k2 = max(max(k2, o2), min(k1, o1));
        k1 = max(k1, o1);
      };
      if (span > 1) join(dpp_i<0xB1>(k1), dpp_i<0xB1>(k2));
      if (span > 2) join(dpp_i<0x4E>(k1), dpp_i<0x4E>(k2));
      if (span > 4) join(dpp_i<0x141>(k1), dpp_i<0x141>(k2));
      if (span > 8) join(dpp_i<0x140>(k1), dpp_i<0x140>(k2));
      if ((lane & (span - 1)) == 0 && e0 < E)
        g_lds[tok][lane >> shift] = a.two && k2 != kOut ? sort_key(key_value(k1) + key_value(k2)) : k1;
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) c_lds[tok][e0 + i] = __int_as_float(key[i]);
      wave_sync();
      if (lane < G) {
        int32_t k1 = kOut, k2 = kOut;
        for (int j = 0; j < gs; ++j) {
          const int32_t k = __float_as_int(c_lds[tok][lane * gs + j]);
          k2 = max(k2, min(k1, k));
          k1 = max(k1, k);
        }
        g_lds[tok][lane] = a.two && k2 != kOut ? sort_key(key_value(k1) + key_value(k2)) : k1;
      }
    }
    wave_sync();
    // a group stays if fewer than top_groups come before it
    const int32_t group_key = lane < G ? g_lds[tok][lane] : kOut;
    int before = 0;
#pragma unroll
    for (int h = 0; h < kMaxExpertGroups; ++h) {
      const int32_t o = g_lds[tok][h];
      before += h < G && (o > group_key || (o == group_key && h < lane)) ? 1 : 0;
    }
    const uint32_t kept = (uint32_t)token_ballot<LPT>(lane < G && before < a.top_groups);
    if (whole) {
      const bool out = !((kept >> min(lane >> shift, 31)) & 1u);
#pragma unroll
      for (int i = 0; i < PER; ++i) key[i] = out ? kOut : key[i];
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int g = min((e0 + i) / gs, G - 1);
        key[i] = (kept >> g) & 1u ? key[i] : kOut;
      }
      wave_sync();
    }
  }

#pragma unroll
  for (int i = 0; i < PER; ++i) c_lds[tok][e0 + i] = s[i];
  for (int r = 0; r < a.top; ++r) {
    int32_t best = key[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) best = max(best, key[i]);
    const int32_t top = all_max<LPT>(best);
    const uint64_t have = token_ballot<LPT>(best == top);
    const bool win = lane == __builtin_ctzll(have);
    int at = PER;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i) at = key[i] == top ? i : at;
    at = win ? at : PER;
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = i == at ? kOut : key[i];
    if (win) i_lds[tok][r] = top == kOut ? -1 : e0 + at;
  }
  wave_sync();
  const bool mine = lane < a.top;
  const int32_t e = mine ? i_lds[tok][lane] : -1;
  const float sc = e >= 0 ? c_lds[tok][e] : 0.0f;
  double w = sc;
  if (a.renorm) {
    const double sum = all_sum<LPT>(lane < 16 ? (double)sc : 0.0);
    w = w / (sum == 0 ? 1.0 : sum);
  }
  if (live && mine) {
    a.weights[t * a.top + lane] = (float)(w * (double)a.scale);
    a.idx[t * a.top + lane] = e;
  }
}

// Gradient of the weights with respect to the logits: the scores are formed
// again as above, the rest is in float64 too (the terms cancel where one
// expert has nearly all the weight). Chosen scores that are 0 as float32 have no part.
template <int LPT, int PER, bool F32>
__global__ __launch_bounds__(kRouteThreads) void k_route_bwd(RouteArgs a, bool vec, bool vec_out) {
  constexpr int kTokens = kRouteThreads / LPT;
  __shared__ double d_lds[kTokens][LPT * PER];      // gradient of each score
  const int lane = threadIdx.x % LPT, tok = threadIdx.x / LPT;
  const int64_t t = (int64_t)blockIdx.x * kTokens + tok;
  const bool live = t < a.rows;
  const int64_t row = live ? t : a.rows - 1;
  const int E = a.experts, e0 = lane * PER;
  const char* xr = reinterpret_cast<const char*>(a.x) + row * a.ld * (F32 ? 4 : 2);
  __shared__ double pow2[32];
  load_pow2(pow2);
  float x[PER];
  double p[PER], m = 0, inv = 1;
  if (!a.sigmoid) {
    load_logits<PER, F32>(x, xr, e0, E, vec);
    inv = softmax64<LPT, PER>(x, p, m, pow2);
  }

  // lane j holds choice j
  int32_t idx = -1;
  double d = 0, s = 0, rest = 0;      // rest: 1 - s
  if (lane < a.top) {
    idx = a.idx[row * a.top + lane];
    if ((uint32_t)idx >= (uint32_t)E) idx = -1;
    if (idx >= 0) {
      float xi;
      if constexpr (F32) xi = reinterpret_cast<const float*>(xr)[idx];
      else xi = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(xr)[idx] << 16);
      if (a.sigmoid) {
        s = sigmoid64(xi, pow2);
        rest = sigmoid64(-xi, pow2);
      } else {
        const double t64 = (double)xi - m;
        s = xi == -INFINITY ? 0.0 : exp64(t64 < -700.0 ? -700.0 : t64, pow2) * inv;
      }
      // a score that is 0 as a float32 gave a weight of 0, also where all of a row's are and "a sum of 0 divides by
      // 1": in float64 it would still have a share of their sum
      if ((float)s == 0.0f) {
        idx = -1;
        s = 0;
      } else {
        d = (double)a.dweights[row * a.top + lane] * (double)a.scale;
      }
    }
  }
  if (a.renorm) {
    double S = all_sum<LPT>(s);
    S = S == 0 ? 1.0 : S;
    const double dot = all_sum<LPT>(d * s);
    if (idx >= 0) d = (d - dot / S) / S;
  }
  // sigmoid: the chosen experts' own derivative, nothing else; softmax: every expert's
  const double inner = a.sigmoid ? 0.0 : all_sum<LPT>(d * s);
  const double mine = a.sigmoid ? d * s * rest : d;
#pragma unroll
  for (int i = 0; i < PER; ++i) d_lds[tok][e0 + i] = 0.0;
  wave_sync();
  for (int j = 0; j < a.top; ++j) {      // one at a time: an expert may be there twice
    if (lane == j && idx >= 0) d_lds[tok][idx] += mine;
    wave_sync();
  }
  if (!live) return;
  float g[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const double v = d_lds[tok][e0 + i];
    g[i] = (float)(a.sigmoid ? v : p[i] * inv * (v - inner));
  }
  constexpr int esz = F32 ? 4 : 2;
  char* out = reinterpret_cast<char*>(a.dx) + (t * E + e0) * esz;
  if constexpr (PER * esz >= 16) {
    if (vec_out && e0 + PER <= E) {
#pragma unroll
      for (int i = 0; i < PER; i += 16 / esz) {
        if constexpr (F32)
          *reinterpret_cast<float4*>(out + 4 * i) = make_float4(g[i], g[i + 1], g[i + 2], g[i + 3]);
        else
          *reinterpret_cast<uint4*>(out + 2 * i) = make_uint4(pack_bf16x2(g[i], g[i + 1]), pack_bf16x2(g[i + 2], g[i + 3]),
                                                              pack_bf16x2(g[i + 4], g[i + 5]), pack_bf16x2(g[i + 6], g[i + 7]));
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (e0 + i >= E) continue;
    if constexpr (F32) reinterpret_cast<float*>(out)[i] = g[i];
    else reinterpret_cast<uint16_t*>(out)[i] = (uint16_t)f32_to_bf16(g[i]);
  }
}

// 16 lanes a token where its experts fit (256) and there are tokens enough to
// fill the card with them: a wave then serves 4 tokens for some 2 to 3 times the
// instructions of one. us for 8 of E experts, 16 lanes against 64: 16384 x 256 12.3 and
// 15.2, 8192 x 256 7.8 and 8.9, 4096 x 256 6.2 and 5.9, 16384 x 64 5.8 and 8.6, 4096 x 128
// 4.9 and 4.8.
template <class Fn>
static void with_shape(const RouteArgs& a, Fn f) {
  using std::integral_constant;
  const int E = a.experts;
  auto per = [&](auto lpt, int n) {
    if (n <= 1) f(lpt, integral_constant<int, 1>{});
    else if (n <= 2) f(lpt, integral_constant<int, 2>{});
    else if (n <= 4) f(lpt, integral_constant<int, 4>{});
    else if (n <= 8) f(lpt, integral_constant<int, 8>{});
    else f(lpt, integral_constant<int, 16>{});
  };
  if (E <= 16 || (E <= 256 && a.rows > 4096))
    per(integral_constant<int, 16>{}, (E + 15) / 16);
  else
    per(integral_constant<int, 64>{}, (E + 63) / 64);
}

static bool vector_rows(const RouteArgs& a) {
  return (reinterpret_cast<uintptr_t>(a.x) & 15) == 0 && a.ld * (a.f32 ? 4 : 2) % 16 == 0;
}

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  with_shape(a, [&](auto lpt, auto per) {
    const dim3 grid((unsigned)((a.rows + kRouteThreads / lpt - 1) / (kRouteThreads / lpt)));
    if (a.f32) hipLaunchKernelGGL((k_route<lpt, per, true>), grid, dim3(kRouteThreads), 0, s, a, vector_rows(a));
    else hipLaunchKernelGGL((k_route<lpt, per, false>), grid, dim3(kRouteThreads), 0, s, a, vector_rows(a));
  });
  return hipGetLastError();
}

hipError_t launch_route_bwd(const RouteArgs& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const bool vec_out = (reinterpret_cast<uintptr_t>(a.dx) & 15) == 0 && a.experts * (a.f32 ? 4 : 2) % 16 == 0;
  with_shape(a, [&](auto lpt, auto per) {
    const dim3 grid((unsigned)((a.rows + kRouteThreads / lpt - 1) / (kRouteThreads / lpt)));
    if (a.f32) hipLaunchKernelGGL((k_route_bwd<lpt, per, true>), grid, dim3(kRouteThreads), 0, s, a, vector_rows(a), vec_out);
    else hipLaunchKernelGGL((k_route_bwd<lpt, per, false>), grid, dim3(kRouteThreads), 0, s, a, vector_rows(a), vec_out);
  });
  return hipGetLastError();
}

}  // namespace mxk
