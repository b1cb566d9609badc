// Routing of tokens to experts and its gradient.
//
// One wave per token, grid-striding over tokens; lane l holds experts l, l + 64,
// ... (VPL of them), so each load of a row is one contiguous piece.  The choice
// must not depend on fp32 rounding: two experts whose keys lie next to each
// other have to come out in the same order however the scores are computed.
// Without a bias the key is the logit itself, which fp32 holds exactly.  With
// one, scores and keys are computed in fp64 (full-rate on CDNA4) and rounded to
// an ordered 32-bit integer; rounding is monotone, so the largest integer marks
// the largest key, and the fp64 values decide among equals alone.
#include "common.h"
#include "sg_moe.h"

namespace sg {

struct RouteArgs {
  const void* logits;
  int64_t ldl;
  int64_t T;
  int E, k;
  const float* bias;
  int n_group, per, topk_group, top2, sigmoid, renorm;
  float scale;
  int32_t* ids;
  float* weights;
};

struct RouteGradArgs {
  const float* grad;
  const void* logits;
  int64_t ldl, T;
  int E, k;
  const int32_t* ids;
  int sigmoid, renorm;
  float scale;
  void* out;
  int64_t ldd;
};

constexpr int RT_WAVES = 4, RT_EMAX = 1024, RT_KMAX = 64, RT_GMAX = 64;

// Tokens from which k_moe_route_rows is taken; us, it / k_moe_route, at 4096, 6144, 8192, 16384 tokens: 256 experts,
// 4 of 8 groups, bias 10.4 / 10.9, 13.6 / 15.3, 14.0 / 19.0, 23.2 / 34.2; 256 without either 7.7 / 6.4, 9.1 / 8.1,
// 9.5 / 10.4, 15.0 / 17.4; 128 without 5.5 / 5.4, 6.4 / 6.6, 6.4 / 8.0, 8.8 / 13.3; 60 without 4.2 / 4.1, 4.8 / 5.0,
// 4.7 / 5.9, 6.3 / 9.1.
constexpr int64_t RT_ROWS_MIN = 8192;

#if SG_DEVICE_PASS
__device__ __forceinline__ float rt_load(const void* p, int64_t i, bool bf16) {
  return bf16 ? bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[i]) : reinterpret_cast<const float*>(p)[i];
}

// fp32 -> unsigned integers of the same order; 0 is below every number (it
// stands for an expert that is out).  -0 and +0 give one integer.
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// One step of a reduction over the wave's lanes: the value CTRL moves here, 0
// where it moves none.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp0(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
}
// row_shr 1, 2, 4, 8, then each row's last lane into the next rows: lane 63
// ends with the whole wave's result.
#define SG_WAVE_STEPS(STEP) \
  STEP(0x111, 0xf) STEP(0x112, 0xf) STEP(0x114, 0xf) STEP(0x118, 0xf) STEP(0x142, 0xa) STEP(0x143, 0xc)

__device__ __forceinline__ float lane_value(float v, int l) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), l));
}
__device__ __forceinline__ double lane_value(double v, int l) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, l);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), l);
  return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#define STEP(C, R) v = max(v, dpp0<C, R>(v));
  SG_WAVE_STEPS(STEP)
#undef STEP
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ float wave_sum(float v) {
#define STEP(C, R) v += __uint_as_float(dpp0<C, R>(__float_as_uint(v)));
  SG_WAVE_STEPS(STEP)
#undef STEP
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}
__device__ __forceinline__ double wave_sum(double v) {
#define STEP(C, R)                                                                        \
  {                                                                                       \
    const uint64_t u = __builtin_bit_cast(uint64_t, v);                                   \
    const uint64_t d = dpp0<C, R>((uint32_t)u) | ((uint64_t)dpp0<C, R>((uint32_t)(u >> 32)) << 32); \
    v += __builtin_bit_cast(double, d);                                                   \
  }
  SG_WAVE_STEPS(STEP)
#undef STEP
  return lane_value(v, 63);
}
#undef SG_WAVE_STEPS

__device__ __forceinline__ double wave_max_slow(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmax(v, __shfl_xor(v, o, 64));
  return v;
}

// Orders this wave's LDS accesses of its lanes before against those after.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The lowest expert among the marked ones (lane l's bit i: expert i 64 + l).
template <int VPL>
__device__ __forceinline__ int lowest(const bool (&mark)[VPL]) {
  int e = -1;
#pragma unroll
  for (int i = VPL - 1; i >= 0; --i) {
    const uint64_t b = __ballot(mark[i]);
    if (b) e = i * 64 + __builtin_ctzll(b);
  }
  return e;
}

// The groups that stay, as a bit mask.  val (LDS, one value per expert, -inf:
// out) holds what a group's value is taken from.  LPG lanes share a group (a
// power of two) and join their two largest by exchange.
__device__ __forceinline__ uint64_t pick_groups(const double* val, const RouteArgs& a, int lane) {
  const double low = -__builtin_inf();
  const int lpg = 1 << (31 - __builtin_clz(64 / a.n_group));
  const int grp = lane / lpg, sub = lane & (lpg - 1);
  double b0 = low, b1 = low;
  if (grp < a.n_group) {
    for (int m = sub; m < a.per; m += lpg) {
      const double v = val[grp * a.per + m];
      b1 = fmax(b1, fmin(b0, v));
      b0 = fmax(b0, v);
    }
  }
  for (int o = 1; o < lpg; o <<= 1) {
    const double c0 = __shfl_xor(b0, o, 64), c1 = __shfl_xor(b1, o, 64);
    b1 = fmax(fmax(b1, c1), fmin(b0, c0));
    b0 = fmax(b0, c0);
  }
  const double v = a.top2 && b1 > low ? b0 + b1 : b0;
  int rank = 0;
  for (int g = 0; g < a.n_group; ++g) {
    const double o = __shfl(v, g * lpg, 64);
    rank += (o > v || (o == v && g < grp)) ? 1 : 0;
  }
  uint64_t keep = 0;
  const uint64_t b = __ballot(grp < a.n_group && sub == 0 && rank < a.topk_group);
  for (int g = 0; g < a.n_group; ++g) keep |= ((b >> (g * lpg)) & 1ull) << g;
  return keep;
}
#endif  // SG_DEVICE_PASS

#if SG_DEVICE_PASS
// e / per for e < 1024: (e + 1/2) / per stays 1 / 2048 away from whole numbers, far more than it is off by.
__device__ __forceinline__ int group_of(int e, float per1) { return (int)(((float)e + 0.5f) * per1); }

// What a lane knows of its experts i 64 + l in every token.
template <int VPL>
struct RouteBias {
  float bias[VPL];
  bool ok[VPL];
  int grp[VPL];
  __device__ __forceinline__ RouteBias(const RouteArgs& a, int lane) {
    // clamped indexes instead of guarded loads: a branch to each would wait for the load before
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) bias[i] = a.bias[min(i * 64 + lane, a.E - 1)];
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) bias[i] = 0.0f;
    }
    const float per1 = 1.0f / (float)a.per;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * 64 + lane;
      ok[i] = e < a.E && bias[i] > -__builtin_inff();
      bias[i] = fminf(bias[i], 3.402823466e38f);
      grp[i] = group_of(e, per1);
    }
  }
};

// Token t by the whole wave.  F64: scores of every expert in fp64 (a bias, or
// groups by their two largest scores); otherwise the keys are the logits and
// only the chosen experts' weights are computed.  val: VPL * 64 values of LDS
// where there are groups.
template <int VPL, bool F64, bool BF16>
__device__ __forceinline__ void route_token(const RouteArgs& a, const RouteBias<VPL>& rb, int64_t t, double* val,
                                            int lane) {
  const double low = -__builtin_inf();
  float x[VPL];
  bool lok[VPL], ok[VPL];   // enters the softmax; may be chosen
  uint32_t top32 = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 64 + lane;
    const float v = rt_load(a.logits, t * a.ldl + min(e, a.E - 1), BF16);
    lok[i] = e < a.E && v > -__builtin_inff();   // false for NaN
    ok[i] = lok[i] && rb.ok[i];
    x[i] = fminf(v, 3.402823466e38f);
    if (lok[i]) top32 = max(top32, ordered(x[i]));
  }
  top32 = wave_max(top32);
  const float top = __uint_as_float((top32 >> 31) ? top32 ^ 0x80000000u : ~top32);   // unused when top32 == 0

  double s[VPL], sum = 1.0;
  if (F64) {
    double part = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if (a.sigmoid) {
        s[i] = lok[i] ? 1.0 / (1.0 + exp(-(double)x[i])) : 0.0;
      } else {
        s[i] = lok[i] ? exp((double)x[i] - (double)top) : 0.0;
        part += s[i];
      }
    }
    if (!a.sigmoid) {
      sum = wave_sum(part);
#pragma unroll
      for (int i = 0; i < VPL; ++i) s[i] = top32 ? s[i] / sum : 0.0;
    }
  } else if (!a.sigmoid) {
    float part = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) part += lok[i] ? expf(x[i] - top) : 0.0f;
    sum = (double)wave_sum(part);
  }

  double key[VPL];   // fp64 key, where it is not the logit
  uint32_t k32[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    key[i] = F64 && a.bias ? s[i] + (double)rb.bias[i] : (double)x[i];
    k32[i] = ok[i] ? ordered((float)key[i]) : 0u;
  }
  if (a.n_group > 1) {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      val[i * 64 + lane] = !ok[i] ? low : F64 && a.top2 && !a.bias ? s[i] : key[i];
    wave_sync();
    const uint64_t keep = pick_groups(val, a, lane);
    wave_sync();
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (!((keep >> (rb.grp[i] & 63)) & 1)) k32[i] = 0u;
  }

  // k rounds: the largest key of the wave, the lowest expert among equals
  int my_id = -1;
  double my_s = 0.0;   // F64: the chosen score of this lane's slot
  float my_x = 0.0f;   // otherwise its logit
  for (int j = 0; j < a.k; ++j) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) m = max(m, k32[i]);
    m = wave_max(m);
    if (m == 0) break;
    bool hit[VPL];
    int n = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      hit[i] = k32[i] == m;
      if (F64) n += __builtin_popcountll(__ballot(hit[i]));
    }
    if (F64 && n > 1) {   // equal after rounding: the fp64 keys decide
      double b = low;
#pragma unroll
      for (int i = 0; i < VPL; ++i) b = hit[i] ? fmax(b, key[i]) : b;
      b = wave_max_slow(b);
#pragma unroll
      for (int i = 0; i < VPL; ++i) hit[i] = hit[i] && key[i] == b;
    }
    const int e = lowest<VPL>(hit);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if ((e >> 6) == i) {   // uniform
        if (F64) {
          const double v = lane_value(s[i], e & 63);
          if (lane == j) my_s = v;
        } else {
          const float v = lane_value(x[i], e & 63);
          if (lane == j) my_x = v;
        }
        if (lane == (e & 63)) k32[i] = 0u;
      }
    }
    if (lane == j) my_id = e;
  }

  double w = my_s;
  if (!F64) w = a.sigmoid ? 1.0 / (1.0 + exp(-(double)my_x)) : exp((double)my_x - (double)top) / sum;
  if (my_id < 0) w = 0.0;
  if (a.renorm) w = w / fmax(wave_sum(w), 1e-300);
  if (lane < a.k) {
    a.ids[t * a.k + lane] = my_id;
    a.weights[t * a.k + lane] = (float)(w * (double)a.scale);
  }
}
#endif  // SG_DEVICE_PASS

// One wave per token.
template <int VPL, bool F64, bool BF16>
__global__ void __launch_bounds__(64 * RT_WAVES) k_moe_route(RouteArgs a) {
#if SG_DEVICE_PASS
  extern __shared__ double rt_lds[];   // n_group > 1: VPL * 64 group values per wave
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const RouteBias<VPL> rb(a, lane);
  for (int64_t t = (int64_t)blockIdx.x * RT_WAVES + wave; t < a.T; t += (int64_t)gridDim.x * RT_WAVES)
    route_token<VPL, F64, BF16>(a, rb, t, rt_lds + wave * (VPL * 64), lane);
#endif  // SG_DEVICE_PASS
}

#if SG_DEVICE_PASS
// Over the 16 lanes of a row; every lane gets the result.
template <int N>
__device__ __forceinline__ uint32_t ror(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xf, 0xf, true);   // folds into its user
}
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, ror<8>(v));
  v = max(v, ror<4>(v));
  v = max(v, ror<2>(v));
  return max(v, ror<1>(v));
}
__device__ __forceinline__ float row_fmax(float v) {
  v = fmaxf(v, __uint_as_float(ror<8>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(ror<4>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(ror<2>(__float_as_uint(v))));
  return fmaxf(v, __uint_as_float(ror<1>(__float_as_uint(v))));
}
__device__ __forceinline__ float row_sum(float v) {
  v += __uint_as_float(ror<8>(__float_as_uint(v)));
  v += __uint_as_float(ror<4>(__float_as_uint(v)));
  v += __uint_as_float(ror<2>(__float_as_uint(v)));
  return v + __uint_as_float(ror<1>(__float_as_uint(v)));
}
template <int N>
__device__ __forceinline__ double ror(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)ror<N>((uint32_t)u) | ((uint64_t)ror<N>((uint32_t)(u >> 32)) << 32));
}
__device__ __forceinline__ double row_sum(double v) {
  v += ror<8>(v);
  v += ror<4>(v);
  v += ror<2>(v);
  return v + ror<1>(v);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float((u >> 31) ? u ^ 0x80000000u : ~u);
}

// Descending; the places that nobody reads cost nothing.
template <int N>
__device__ __forceinline__ void sort_down(uint32_t (&v)[N]) {   // Batcher's odd-even merge sort
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t x = v[i + j], y = v[i + j + k];
            v[i + j] = max(x, y);
            v[i + j + k] = min(x, y);
          }
}
#endif  // SG_DEVICE_PASS

// Many tokens: 16 lanes a token, four tokens a wave, VPL experts a lane (lane j:
// 64 i + 4 j .. + 3).  What bounds routing is the instructions per token, and the
// fp64 scores of every expert were most of them (16384 tokens of 256 experts in 8
// groups: 34.2 us, 23.2 this way, of which the experts' preparation, done once a wave
// and at this size for four tokens only, is 44% of the instructions); here scores are
// fp32 and keys are whole numbers of 24 bits with the expert in the low byte (255 - e,
// so that the lowest wins among equals), one 32-bit maximum finding both.  A key is off by `err` units at most; candidates
// within 2 err of each other are put in order by their fp64 keys, and where a
// group, or an expert that is no candidate, lies as near to those that stay, the
// token is done again by route_token, which decides in fp64.  bf16 logits without a bias are exact keys.
//   err, with a bias: scores are off by 2^-22 (sigmoid: exponential and reciprocal
//   of one step each, s (1 - s) |x| <= 0.23 of the argument's rounding) or 2^-19
//   (softmax: 3 steps of 2^-24 a term, 28 on the sum), taken twice as large; the
//   sum s + b by half a step of |lo| + R; three roundings more of one unit at most.
// KL: entries kept per lane (a lane gives at most k + 2).
template <int VPL, int KL, bool SCORES, bool BF16>
__global__ void __launch_bounds__(64 * RT_WAVES) k_moe_route_rows(RouteArgs a, int vec) {
#if SG_DEVICE_PASS
  constexpr int STRIDE = 16 * VPL + VPL;           // group values of one token, 32 experts and a gap of 2
  extern __shared__ double rt_lds[];               // n_group > 1: per wave, 4 tokens; at least 16 VPL doubles
  const int lane = threadIdx.x & 63, j0 = lane & 15, tok = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  double* const mine = rt_lds + wave * (VPL * 36);
  uint32_t* const val = reinterpret_cast<uint32_t*>(mine) + tok * STRIDE;
  constexpr float UNITS = 16777208.0f;             // 2^24 - 8
  const float inf = __builtin_inff();

  float bias[VPL];
  uint32_t usable = 0;
  float hi = -inf, lo = inf;   // of the usable biases
  if (a.bias) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) bias[v] = a.bias[min(64 * (v >> 2) + 4 * j0 + (v & 3), a.E - 1)];
  } else {
#pragma unroll
    for (int v = 0; v < VPL; ++v) bias[v] = 0.0f;
  }
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const bool in = 64 * (v >> 2) + 4 * j0 + (v & 3) < a.E && bias[v] > -inf;
    bias[v] = fminf(bias[v], 3.402823466e38f);
    usable |= in ? 1u << v : 0u;
    hi = fmaxf(hi, in ? bias[v] : -inf);
    lo = fminf(lo, in ? bias[v] : inf);
  }
  hi = row_fmax(hi);
  lo = -row_fmax(-lo);
  if (hi < lo) hi = lo = 0.0f;   // nothing usable
  // Finite masks (-1e4, -1e9) would leave the others too few units: keys below hi - 64
  // are all 1 then, equal to each other.  Decisions among those are made in fp64 as
  // between any keys this near; a group's value by its two largest is unknown with one.
  const bool floor = hi - lo > 1024.0f;
  if (floor) lo = hi - 64.0f;
  const float R = 1.0f + (hi - lo);
  const float scale = UNITS / R;
  const double Ld = (double)lo * (double)scale;
  bool hopeless = false;       // keys too far apart for 24 bits: every token in fp64
  int th = BF16 && !a.bias ? -1 : 0, L = 0;
  if (a.bias) {
    hopeless = !(R < 1e30f) || !(fabs(Ld) < 2.7e8);
    th = hopeless ? 0 : (int)(2.0f * ((a.sigmoid ? 8.0f : 64.0f) + (fabsf(lo) / R) + 6.0f));
    L = hopeless ? 0 : (int)rint(Ld);
  }
  // groups: values are keys, or scores where two are added up without a bias
  const bool by_score = a.top2 && !a.bias;
  const int gth = by_score ? 2 * (a.sigmoid ? 28 : 140) : a.top2 ? 2 * th + 4 : th;
  const int gL = by_score ? 0 : L;
  const int lpg = 1 << (31 - __builtin_clz(16 / a.n_group));   // lanes that share a group
  const int grp = j0 / lpg, sub = j0 & (lpg - 1);
  const float per1 = 1.0f / (float)a.per;
  uint32_t place[(VPL + 7) / 8];                   // first lane of each expert's group, 4 bits
#pragma unroll
  for (int v = 0; v < (VPL + 7) / 8; ++v) place[v] = 0;
  if (a.n_group > 1) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int e = min(64 * (v >> 2) + 4 * j0 + (v & 3), a.E - 1);
      place[v >> 3] |= (uint32_t)(group_of(e, per1) * lpg) << (4 * (v & 7));
    }
  }

  for (int64_t t0 = ((int64_t)blockIdx.x * RT_WAVES + wave) * 4; t0 < a.T; t0 += (int64_t)gridDim.x * RT_WAVES * 4) {
    int j = j0;
    asm volatile("" : "+v"(j));   // addresses and comparisons are made anew: kept over the loop they spill
    const int64_t t = t0 + tok;
    const bool here = t < a.T;
    float x[VPL];
    const int64_t row = (here ? t : a.T - 1) * a.ldl;
    if (vec) {
#pragma unroll
      for (int i = 0; i < VPL / 4; ++i) {
        const int64_t at = row + min(64 * i + 4 * j, a.E - 4);
        if (BF16) {
          const uint2 u = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(a.logits) + at);
          x[4 * i] = __uint_as_float(u.x << 16);
          x[4 * i + 1] = __uint_as_float(u.x & 0xffff0000u);
          x[4 * i + 2] = __uint_as_float(u.y << 16);
          x[4 * i + 3] = __uint_as_float(u.y & 0xffff0000u);
        } else {
          const float4 u = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.logits) + at);
          x[4 * i] = u.x;
          x[4 * i + 1] = u.y;
          x[4 * i + 2] = u.z;
          x[4 * i + 3] = u.w;
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        x[v] = rt_load(a.logits, row + min(64 * (v >> 2) + 4 * j + (v & 3), a.E - 1), BF16);
    }
    uint32_t live = 0, top32 = 0;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const bool in = here && 64 * (v >> 2) + 4 * j + (v & 3) < a.E && x[v] > -inf;   // false for NaN
      live |= in ? 1u << v : 0u;
      x[v] = in ? fminf(x[v], 3.402823466e38f) : -inf;
      if (!a.sigmoid) top32 = max(top32, in ? ordered(x[v]) : 0u);
    }
    float top = 0.0f, sum = 1.0f, s[VPL];
    if (!a.sigmoid) {
      top32 = row_max(top32);
      top = top32 ? from_ordered(top32) : 0.0f;
      float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        s[v] = __expf(x[v] - top);
        part[v & 3] += s[v];
      }
      sum = row_sum((part[0] + part[1]) + (part[2] + part[3]));
      const float r = sum > 0.0f ? __builtin_amdgcn_rcpf(sum) : 0.0f;
#pragma unroll
      for (int v = 0; v < VPL; ++v) s[v] *= r;
    } else if (SCORES) {
#pragma unroll
      for (int v = 0; v < VPL; ++v) s[v] = __builtin_amdgcn_rcpf(1.0f + __expf(-x[v]));
    }
    const uint32_t ok = live & usable;
    uint32_t key[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      // bf16: the high half (+inf, as the largest fp32, stays above the largest bf16)
      uint32_t q = BF16 ? (ordered(x[v]) + 0xffffu) >> 16 : ordered(x[v]) >> 8;
      if (SCORES && a.bias) q = 1u + (uint32_t)fminf(fmaxf((s[v] + bias[v] - lo) * scale, 0.0f), UNITS);
      key[v] = (ok >> v) & 1 ? q : 0u;
    }
    bool unsure = hopeless;
    if (a.n_group > 1) {
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        const int e = 64 * (v >> 2) + 4 * j + (v & 3);
        uint32_t q = key[v];
        if (SCORES && by_score) q = (ok >> v) & 1 ? 1u + (uint32_t)(s[v] * UNITS) : 0u;
        val[e + 2 * (e >> 5)] = q;
      }
      wave_sync();
      uint32_t b0 = 0, b1 = 0;
      for (int m = sub; m < a.per + sub; m += 4 * lpg) {   // the same count in every lane, four reads at a time
        uint32_t q[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int e = min(grp * a.per + m + c * lpg, a.E - 1);
          q[c] = val[e + 2 * (e >> 5)];
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t u = m + c * lpg < a.per && grp < a.n_group ? q[c] : 0u;
          b1 = max(b1, min(b0, u));
          b0 = max(b0, u);
        }
      }
      for (int o = 1; o < lpg; o <<= 1) {
        const uint32_t c0 = __shfl_xor(b0, o, 16), c1 = __shfl_xor(b1, o, 16);
        b1 = max(max(b1, c1), min(b0, c0));
        b0 = max(b0, c0);
      }
      wave_sync();
      const int none = -(1 << 30);   // below every value by more than gth
      const int V = grp >= a.n_group || b0 == 0 ? none : a.top2 && b1 ? (int)(b0 + b1) + 2 * gL : (int)b0 + gL;
      int surely = 0, perhaps = 0;   // groups that come before this one
      if (gth < 0) {
        for (int g = 0; g < a.n_group; ++g) {
          const int o = __shfl(V, g * lpg, 16);
          perhaps += o > V || (o == V && g < grp) ? 1 : 0;
        }
        surely = perhaps;
      } else {
        for (int g = 0; g < a.n_group; ++g) {
          const int o = __shfl(V, g * lpg, 16);
          surely += o > V + gth ? 1 : 0;
          perhaps += o >= V - gth ? 1 : 0;
        }
        perhaps -= 1;   // itself
      }
      const bool stays = grp < a.n_group && perhaps < a.topk_group;
      unsure = unsure || (grp < a.n_group && V != none && !stays && surely < a.topk_group);
      unsure = unsure || (floor && a.top2 && (b1 ? b1 : b0) == 1);
      const uint32_t kept = (uint32_t)(__ballot(stays) >> (16 * tok));
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        key[v] &= (uint32_t)__builtin_amdgcn_sbfe((int)kept, (place[v >> 3] >> (4 * (v & 7))) & 15, 1);
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v)
      key[v] = key[v] ? (key[v] << 8) | (uint32_t)(255 - (64 * (v >> 2) + 4 * j + (v & 3))) : 0u;
    sort_down<VPL>(key);

    // k rounds for the experts, one for a candidate more, one for the distance to the next
    const int c = min(a.k + 1, 16);
    uint32_t my = 0, before = 0, kth = 0;
    bool close = false;   // two candidates whose order these keys do not tell
    for (int r = 0; r <= c; ++r) {
      const uint32_t m = row_max(key[0]);
      const uint32_t won = key[0] == m ? ~0u : 0u;   // keys differ in their expert, unless all are gone
#pragma unroll
      for (int v = 0; v < KL; ++v) key[v] = (won & (v + 1 < KL ? key[v + 1] : 0u)) | (~won & key[v]);
      close = close || (r > 0 && r < c && m && (int)((before >> 8) - (m >> 8)) <= th);
      before = m;
      if (r == a.k - 1) kth = m;
      if (j == r && r < c) my = m;
    }
    // one that is no candidate may belong among the k
    unsure = unsure || (before && (int)((kth >> 8) - (before >> 8)) <= th);

    int id = my ? 255 - (int)(my & 255) : -1;
    double w = 0.0, xc = 0.0;
    if (id >= 0) {
      xc = (double)fminf(rt_load(a.logits, t * a.ldl + id, BF16), 3.402823466e38f);
      w = a.sigmoid ? 1.0 / (1.0 + exp(-xc)) : exp(xc - (double)top) / (double)sum;
    }
    if (a.bias && !a.sigmoid) {
      unsure = unsure || close;   // these scores' sum is fp32
    } else if (__ballot(close)) {
      // the candidates anew by their fp64 keys, as route_token orders them
      const double k64 = id < 0 ? 0.0 : a.bias ? w + (double)fminf(a.bias[id], 3.402823466e38f) : xc;
      int rank = id < 0 ? j : 0, from = 0;
      for (int i = 0; i < c; ++i) {
        const double o = __shfl(k64, i, 16);
        const int oid = __shfl(id, i, 16);
        rank += id >= 0 && oid >= 0 && (o > k64 || (o == k64 && oid < id)) ? 1 : 0;
      }
      for (int i = 0; i < 16; ++i) from = __shfl(rank, i, 16) == j ? i : from;
      id = __shfl(id, from, 16);
      w = __shfl(w, from, 16);
    }
    if (j >= a.k) w = 0.0;
    if (a.renorm) w = w / fmax(row_sum(w), 1e-300);
    const uint64_t again = __ballot(unsure);
    if (here && j < a.k && ((again >> (16 * tok)) & 0xffff) == 0) {
      a.ids[t * a.k + j] = id;
      a.weights[t * a.k + j] = (float)(w * (double)a.scale);
    }
    if (again) {
      int l = lane;
      asm volatile("" : "+v"(l));   // rare: nothing of it belongs before the loop
      const RouteBias<(VPL + 3) / 4> rb(a, l);
      for (int i = 0; i < 4; ++i)
        if (((again >> (16 * i)) & 0xffff) && t0 + i < a.T)
          route_token<(VPL + 3) / 4, SCORES, BF16>(a, rb, t0 + i, mine, l);
    }
  }
#endif  // SG_DEVICE_PASS
}

// One wave per token.  Lane j < k computes the gradient through slot j; the row
// is put together in LDS (zero, then the chosen experts) and leaves in
// contiguous pieces.  ALL: softmax weights kept as they are, where every
// probability of the row enters.
template <int VPL, bool ALL, bool BF16>
__global__ void __launch_bounds__(64 * RT_WAVES) k_moe_route_grad(RouteGradArgs a) {
#if SG_DEVICE_PASS
  extern __shared__ float rt_row[];   // VPL * 64 per wave
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float* const row = rt_row + wave * (VPL * 64);

  for (int64_t t = (int64_t)blockIdx.x * RT_WAVES + wave; t < a.T; t += (int64_t)gridDim.x * RT_WAVES) {
    const int id = lane < a.k ? a.ids[t * a.k + lane] : -1;
    const bool in = id >= 0 && id < a.E;
    const float g = in ? a.grad[t * a.k + lane] : 0.0f;
    float v = in ? rt_load(a.logits, t * a.ldl + id, BF16) : -__builtin_inff();
    if (!(v > -__builtin_inff())) v = -__builtin_inff();   // NaN is out too
    v = fminf(v, 3.402823466e38f);
    const bool live = v > -__builtin_inff();
#pragma unroll
    for (int i = 0; i < VPL; ++i) row[i * 64 + lane] = 0.0f;

    float d = 0.0f, dot = 0.0f, top = 0.0f, z = 1.0f;
    float x[VPL];
    if (ALL) {
      uint32_t top32 = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = i * 64 + lane;
        const float u = e < a.E ? rt_load(a.logits, t * a.ldl + e, BF16) : -__builtin_inff();
        x[i] = u > -__builtin_inff() ? fminf(u, 3.402823466e38f) : -__builtin_inff();
        if (x[i] > -__builtin_inff()) top32 = max(top32, ordered(x[i]));
      }
      top32 = wave_max(top32);
      top = top32 == 0 ? 0.0f : __uint_as_float((top32 >> 31) ? top32 ^ 0x80000000u : ~top32);
      float part = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        x[i] = expf(x[i] - top);
        part += x[i];
      }
      z = top32 == 0 ? 0.0f : 1.0f / wave_sum(part);
      const float p = live ? expf(v - top) * z : 0.0f;
      dot = wave_sum(g * p);
    } else if (a.sigmoid) {
      // s and 1 - s each from its own exponential: neither loses its small values
      const double en = exp(-(double)v), s = live ? 1.0 / (1.0 + en) : 0.0;
      const double c = live ? 1.0 / (1.0 + exp((double)v)) : 0.0;
      if (a.renorm) {
        const double r = s / fmax(wave_sum(s), 1e-300);
        const double q = wave_sum((double)g * r);
        d = (float)((double)a.scale * r * c * ((double)g - q));
      } else {
        d = (float)((double)a.scale * (double)g * s * c);
      }
    } else {   // softmax over the chosen
      const uint32_t top32 = wave_max(live ? ordered(v) : 0u);
      const float m = top32 == 0 ? 0.0f : __uint_as_float((top32 >> 31) ? top32 ^ 0x80000000u : ~top32);
      const float ex = live ? expf(v - m) : 0.0f;
      const float r = ex / fmaxf(wave_sum(ex), 1e-37f);
      d = a.scale * r * (g - wave_sum(g * r));
    }

    wave_sync();
    if (in) row[id] = ALL ? g : d;
    wave_sync();
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * 64 + lane;
      if (e >= a.E) continue;
      const float o = ALL ? a.scale * (x[i] * z) * (row[e] - dot) : row[e];
      if (BF16) reinterpret_cast<uint16_t*>(a.out)[t * a.ldd + e] = (uint16_t)f32_to_bf16(o);
      else reinterpret_cast<float*>(a.out)[t * a.ldd + e] = o;
    }
    wave_sync();
  }
#endif  // SG_DEVICE_PASS
}

// Gradients that reach the chosen experts alone, 16 lanes a token (k <= 16), four
// tokens a wave: the slots' fp64 exponentials are what the kernel above spends its
// time on (16384 tokens of 256 experts: 10.6 us with 64 lanes a token, 7.9 here).
// The four rows are put together in LDS and leave in pieces of 4 columns a lane.
template <bool BF16>
__global__ void __launch_bounds__(64 * RT_WAVES) k_moe_route_grad_rows(RouteGradArgs a, int vec) {
#if SG_DEVICE_PASS
  extern __shared__ __attribute__((aligned(16))) float rt_row[];   // per wave 4 rows of `pitch`
  const int lane = threadIdx.x & 63, j = lane & 15, tok = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), pitch = (a.E + 3) & ~3;
  float* const rows = rt_row + wave * (4 * pitch);
  for (int64_t t0 = ((int64_t)blockIdx.x * RT_WAVES + wave) * 4; t0 < a.T; t0 += (int64_t)gridDim.x * RT_WAVES * 4) {
    const int64_t t = t0 + tok;
    const bool slot = t < a.T && j < a.k;
    const int id = slot ? a.ids[t * a.k + j] : -1;
    const bool in = id >= 0 && id < a.E;
    const float g = in ? a.grad[t * a.k + j] : 0.0f;
    float v = in ? rt_load(a.logits, t * a.ldl + id, BF16) : -__builtin_inff();
    if (!(v > -__builtin_inff())) v = -__builtin_inff();   // NaN is out too
    v = fminf(v, 3.402823466e38f);
    const bool live = v > -__builtin_inff();
    for (int e = 4 * lane; e < 4 * pitch; e += 256)
      *reinterpret_cast<float4*>(rows + e) = make_float4(0.f, 0.f, 0.f, 0.f);

    float d = 0.0f;
    if (a.sigmoid) {
      // s and 1 - s each from its own exponential: neither loses its small values
      const double s = live ? 1.0 / (1.0 + exp(-(double)v)) : 0.0, c = live ? 1.0 / (1.0 + exp((double)v)) : 0.0;
      if (a.renorm) {
        const double r = s / fmax(row_sum(s), 1e-300);
        const double q = row_sum((double)g * r);
        d = (float)((double)a.scale * r * c * ((double)g - q));
      } else {
        d = (float)((double)a.scale * (double)g * s * c);
      }
    } else {   // softmax over the chosen
      const uint32_t top32 = row_max(live ? ordered(v) : 0u);
      const float m = top32 == 0 ? 0.0f : from_ordered(top32);
      const float ex = live ? expf(v - m) : 0.0f;
      const float r = ex / fmaxf(row_sum(ex), 1e-37f);
      d = a.scale * r * (g - row_sum(g * r));
    }
    wave_sync();
    if (in) rows[tok * pitch + id] = d;
    wave_sync();
    if (vec) {
      for (int i = lane; i < pitch; i += 64) {   // 4 rows of pitch / 4 pieces
        const int r = i / (pitch >> 2), e = 4 * (i - r * (pitch >> 2));
        if (t0 + r >= a.T) continue;
        const float4 o = *reinterpret_cast<const float4*>(rows + r * pitch + e);
        const int64_t at = (t0 + r) * a.ldd + e;
        if (BF16)
          *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + at) =
              make_uint2(f32x2_to_bf16x2(o.x, o.y), f32x2_to_bf16x2(o.z, o.w));
        else
          *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at) = o;
      }
    } else {
      for (int r = 0; r < 4 && t0 + r < a.T; ++r)
        for (int e = lane; e < a.E; e += 64) {
          if (BF16) reinterpret_cast<uint16_t*>(a.out)[(t0 + r) * a.ldd + e] = (uint16_t)f32_to_bf16(rows[r * pitch + e]);
          else reinterpret_cast<float*>(a.out)[(t0 + r) * a.ldd + e] = rows[r * pitch + e];
        }
    }
    wave_sync();
  }
#endif  // SG_DEVICE_PASS
}

template <int VPL, bool F64, bool BF16>
static void launch_route_rows(const RouteArgs& a, hipStream_t st) {
  const int64_t tokens = 4 * RT_WAVES;
  const unsigned grid = grid_for(a.T, tokens, 1024);
  const size_t lds = a.n_group > 1 ? (size_t)RT_WAVES * VPL * 36 * sizeof(double) : 0;
  const int vec = a.E % 4 == 0 && a.ldl % 4 == 0 && aligned(a.logits, BF16 ? 8 : 16);
  if (a.k <= 10) k_moe_route_rows<VPL, VPL < 12 ? VPL : 12, F64, BF16><<<grid, 64 * RT_WAVES, lds, st>>>(a, vec);
  else k_moe_route_rows<VPL, VPL, F64, BF16><<<grid, 64 * RT_WAVES, lds, st>>>(a, vec);
}

// VPL: the smallest of 1, 2, 4, 8, 16 that holds E experts in 64 lanes.
template <bool F64, bool BF16>
static void launch_route(const RouteArgs& a, hipStream_t st) {
  if (a.T >= RT_ROWS_MIN && a.E <= 256 && a.k <= 16 && a.n_group <= 16) {
    if (a.E <= 64) launch_route_rows<4, F64, BF16>(a, st);
    else if (a.E <= 128) launch_route_rows<8, F64, BF16>(a, st);
    else launch_route_rows<16, F64, BF16>(a, st);
    return;
  }
  const unsigned grid = grid_for(a.T, RT_WAVES, 2048);
  const int vpl = a.E <= 64 ? 1 : a.E <= 128 ? 2 : a.E <= 256 ? 4 : a.E <= 512 ? 8 : 16;
  const size_t lds = a.n_group > 1 ? (size_t)RT_WAVES * vpl * 64 * sizeof(double) : 0;
  switch (vpl) {
    case 1: k_moe_route<1, F64, BF16><<<grid, 64 * RT_WAVES, lds, st>>>(a); break;
    case 2: k_moe_route<2, F64, BF16><<<grid, 64 * RT_WAVES, lds, st>>>(a); break;
    case 4: k_moe_route<4, F64, BF16><<<grid, 64 * RT_WAVES, lds, st>>>(a); break;
    case 8: k_moe_route<8, F64, BF16><<<grid, 64 * RT_WAVES, lds, st>>>(a); break;
    default: k_moe_route<16, F64, BF16><<<grid, 64 * RT_WAVES, lds, st>>>(a); break;
  }
}

template <bool ALL, bool BF16>
static void launch_route_grad(const RouteGradArgs& a, hipStream_t st) {
  if (!ALL && a.k <= 16 && a.E <= 512) {
    const int pitch = (a.E + 3) & ~3;
    const int vec = a.E % 4 == 0 && a.ldd % 4 == 0 && aligned(a.out, BF16 ? 8 : 16);
    k_moe_route_grad_rows<BF16><<<grid_for(a.T, 4 * RT_WAVES, 2048), 64 * RT_WAVES, (size_t)RT_WAVES * 4 * pitch * 4, st>>>(
        a, vec);
    return;
  }
  const unsigned grid = grid_for(a.T, RT_WAVES, 2048);
  const int vpl = a.E <= 64 ? 1 : a.E <= 128 ? 2 : a.E <= 256 ? 4 : a.E <= 512 ? 8 : 16;
  const size_t lds = (size_t)RT_WAVES * vpl * 64 * sizeof(float);
  switch (vpl) {
    case 1: k_moe_route_grad<1, ALL, BF16><<<grid, 64 * RT_WAVES, lds, st>>>(a); break;
    case 2: k_moe_route_grad<2, ALL, BF16><<<grid, 64 * RT_WAVES, lds, st>>>(a); break;
    case 4: k_moe_route_grad<4, ALL, BF16><<<grid, 64 * RT_WAVES, lds, st>>>(a); break;
    case 8: k_moe_route_grad<8, ALL, BF16><<<grid, 64 * RT_WAVES, lds, st>>>(a); break;
    default: k_moe_route_grad<16, ALL, BF16><<<grid, 64 * RT_WAVES, lds, st>>>(a); break;
  }
}

}  // namespace sg

using namespace sg;

extern "C" sg_status sg_moe_route(const void* logits, sg_dtype l_dt, int64_t T, int64_t E, int64_t ldl,
                                  const float* bias, int k, sg_score score, int n_group, int topk_group,
                                  sg_group_score group_score, int renormalize, float scale, int32_t* ids,
                                  float* weights, hipStream_t stream) {
  if (!logits || !ids || !weights) return SG_ERR_NULL;
  if (l_dt != SG_F32 && l_dt != SG_BF16) return SG_ERR_UNSUPPORTED;
  if (score != SG_SCORE_SOFTMAX && score != SG_SCORE_SIGMOID) return SG_ERR_UNSUPPORTED;
  if (group_score != SG_GROUP_MAX && group_score != SG_GROUP_TOP2) return SG_ERR_UNSUPPORTED;
  if (T <= 0 || E <= 0 || E > RT_EMAX || ldl < E || k < 1 || k > RT_KMAX || k > E) return SG_ERR_SHAPE;
  if (n_group < 1 || n_group > RT_GMAX || E % n_group || topk_group < 1 || topk_group > n_group) return SG_ERR_SHAPE;
  if (k > topk_group * (E / n_group)) return SG_ERR_SHAPE;
  if (!aligned(logits, dtype_size(l_dt)) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
    return SG_ERR_ALIGN;
  RouteArgs a;
  a.logits = logits; a.ldl = ldl; a.T = T; a.E = (int)E; a.k = k; a.bias = bias;
  a.n_group = n_group; a.per = (int)(E / n_group); a.topk_group = topk_group;
  a.top2 = group_score == SG_GROUP_TOP2; a.sigmoid = score == SG_SCORE_SIGMOID; a.renorm = renormalize != 0;
  a.scale = scale; a.ids = ids; a.weights = weights;
  clear_hip_error();
  const bool f64 = bias || (n_group > 1 && a.top2);
  if (l_dt == SG_BF16) {
    if (f64) launch_route<true, true>(a, stream);
    else launch_route<false, true>(a, stream);
  } else {
    if (f64) launch_route<true, false>(a, stream);
    else launch_route<false, false>(a, stream);
  }
  return launch_status();
}

extern "C" sg_status sg_moe_route_backward(const float* grad, const void* logits, sg_dtype l_dt, int64_t T, int64_t E,
                                           int64_t ldl, const int32_t* ids, int k, sg_score score, int renormalize,
                                           float scale, void* dlogits, int64_t ldd, hipStream_t stream) {
  if (!grad || !logits || !ids || !dlogits) return SG_ERR_NULL;
  if (l_dt != SG_F32 && l_dt != SG_BF16) return SG_ERR_UNSUPPORTED;
  if (score != SG_SCORE_SOFTMAX && score != SG_SCORE_SIGMOID) return SG_ERR_UNSUPPORTED;
  if (T <= 0 || E <= 0 || E > RT_EMAX || ldl < E || ldd < E || k < 1 || k > RT_KMAX || k > E) return SG_ERR_SHAPE;
  if (!aligned(grad, 4) || !aligned(logits, dtype_size(l_dt)) || !aligned(ids, 4) ||
      !aligned(dlogits, dtype_size(l_dt)))
    return SG_ERR_ALIGN;
  RouteGradArgs a;
  a.grad = grad; a.logits = logits; a.ldl = ldl; a.T = T; a.E = (int)E; a.k = k; a.ids = ids;
  a.sigmoid = score == SG_SCORE_SIGMOID; a.renorm = renormalize != 0; a.scale = scale;
  a.out = dlogits; a.ldd = ldd;
  clear_hip_error();
  const bool all = score == SG_SCORE_SOFTMAX && !renormalize;
  if (l_dt == SG_BF16) {
    if (all) launch_route_grad<true, true>(a, stream);
    else launch_route_grad<false, true>(a, stream);
  } else {
    if (all) launch_route_grad<true, false>(a, stream);
    else launch_route_grad<false, false>(a, stream);
  }
  return launch_status();
}
