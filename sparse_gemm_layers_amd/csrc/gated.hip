// Gated projections, H = a(X . Wg^T + gate_add) * (X . Wu^T + up_add), and their
// backward pass
//   dG = dH * U * a'(G), dU = dH * a(G), dX = dG . Wg + dU . Wu,
//   dWg = dG^T . X, dWu = dU^T . X.
// One product of X with the rows of both weights (a workgroup's tile holds as many
// gate as up rows, of the same f), activation and product on its fp32 sums.  The
// backward pass has the same product with another epilogue where G and U were not
// kept, a pass over [T, F] where they were; then dX sums over both weights' rows in
// one product (2 F long, split over workgroups where its tiles are few), and dW is one
// product whose left rows are those of dWg and dWu.
#include "bf16_tile.h"
#include "sg_gated.h"
#include <stdlib.h>

namespace sg {

struct GatedArgs {
  int64_t T;
  int F, D;
  const uint16_t *x, *gate, *up;
  int64_t ldx, ldg, ldu;
  int act;
  const uint16_t *gate_add, *up_add;
  int64_t ld_add;
  // forward
  void* h;
  int64_t ldh;
  int h_f32;
  uint16_t *g, *u;       // NULL: not kept
  int64_t ld_gu;
  // backward
  const uint16_t* dh;
  int64_t ld_dh;
  uint16_t *dg, *du;
  int64_t ld_dgu;
};

#if SG_DEVICE_PASS
__device__ __forceinline__ float sigmoid_(float v) { return 1.0f / (1.0f + __expf(-v)); }

// a(g) and a'(g).  erfc, not 1 + erf: the latter loses all digits of the left tail.
template <bool SLOPE>
__device__ __forceinline__ float act_of(int act, float g, float& slope) {
  constexpr float C = 0.7978845608028654f;   // sqrt(2 / pi)
  if (act == SG_ACT_SILU) {
    const float s = sigmoid_(g);
    if (SLOPE) slope = s * (1.0f + g * (1.0f - s));
    return g * s;
  }
  if (act == SG_ACT_GELU) {
    const float phi = 0.5f * erfcf(-0.7071067811865476f * g);
    if (SLOPE) slope = phi + g * (0.3989422804014327f * __expf(-0.5f * g * g));
    return g * phi;
  }
  if (act == SG_ACT_GELU_TANH) {
    const float s = sigmoid_(2.0f * C * (g + 0.044715f * g * g * g));
    if (SLOPE) {
      const float t = g * s * (1.0f - s);
      // the factor overflows where the sigmoid has long reached 0 or 1
      slope = s + (t == 0.0f ? t : t * (2.0f * C) * (1.0f + 0.134145f * g * g));
    }
    return g * s;
  }
  if (SLOPE) slope = g > 0.0f ? 1.0f : g <= 0.0f ? 0.0f : g;
  return g > 0.0f ? g : g <= 0.0f ? 0.0f : g;   // NaN stays
}

__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const uint4 t = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]),
                                            f32x2_to_bf16x2(v[4], v[5]), f32x2_to_bf16x2(v[6], v[7]));
}

// Token m, hidden values f .. f + 7: from the sums of both products to what is stored.
template <bool BACK>
__device__ __forceinline__ void gated_finish(const GatedArgs& a, int64_t m, int f, float (&g)[8], float (&u)[8]) {
  float t[8];
  if (a.gate_add) {
    load8(a.gate_add + m * a.ld_add + f, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] += t[i];
  }
  if (a.up_add) {
    load8(a.up_add + m * a.ld_add + f, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] += t[i];
  }
  float s = 0.0f;
  if (!BACK) {
    if (a.g) {
      store8(a.g + m * a.ld_gu + f, g);
      store8(a.u + m * a.ld_gu + f, u);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = act_of<false>(a.act, g[i], s) * u[i];
    if (a.h_f32) {
      float* const h = reinterpret_cast<float*>(a.h) + m * a.ldh + f;
      *reinterpret_cast<float4*>(h) = make_float4(t[0], t[1], t[2], t[3]);
      *reinterpret_cast<float4*>(h + 4) = make_float4(t[4], t[5], t[6], t[7]);
    } else {
      store8(reinterpret_cast<uint16_t*>(a.h) + m * a.ldh + f, t);
    }
  } else {
    load8(a.dh + m * a.ld_dh + f, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = act_of<true>(a.act, g[i], s);
      g[i] = t[i] * u[i] * s;
      u[i] = t[i] * v;
    }
    store8(a.dg + m * a.ld_dgu + f, g);
    store8(a.du + m * a.ld_dgu + f, u);
  }
}
#endif  // SG_DEVICE_PASS

// Left rows of a tile: a wave's first NI / 2 sub-tiles are gate rows, the others up rows
// of the same f.
template <int NI, int NW>
struct GatedRow {
  // the waves of an instruction cover NW / 2 sub-tiles: half of a wave's at most, or all of them
  static constexpr int HALF = NI / 2, MATS = NW / 2 <= HALF ? 2 : 1;
  static_assert(NW / 2 <= HALF || NW / 2 == NI, "sub-tiles of an instruction");
#if SG_DEVICE_PASS
  __device__ static __forceinline__ int row(int u, int wave, int l) {
    const int s = (NW * u + wave) >> 1, r = 8 * (wave & 1) + (l >> 3);
    return s / NI * (16 * HALF) + tile_n(s % HALF, r);
  }
  __device__ static constexpr int sel(int u) { return MATS == 1 ? 0 : NW / 2 * u / HALF & 1; }
  __device__ static __forceinline__ int sel_wave(int wave) { return MATS == 1 ? (wave >> 1) / HALF : 0; }
#endif
};

// Many rows: tiles of BN / 2 rows of each weight x BM tokens (bf16_tile.h).
template <typename T, bool BACK>
__global__ void __launch_bounds__(T::NW * 64) k_gated_tile(GatedArgs a, int tiles_m, int tiles_n) {
#if SG_DEVICE_PASS
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::LDS];
  int tn, tm;
  tile_coords(tiles_m, tiles_n, tn, tm);
  const int l = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int f0 = tn * (T::BN / 2);
  const int64_t m0 = (int64_t)tm * T::BM;
  const int rows = (int)min((int64_t)T::BM, a.T - m0), wrows = min(T::BN / 2, a.F - f0);
  const int KB = (a.D + 63) >> 6;
  typename T::L lo;
  typename T::R ro;
  lo.p[0] = a.gate + f0 * a.ldg;
  lo.p[1] = a.up + f0 * a.ldu;
  lo.bytes[0] = (uint32_t)(((wrows - 1) * a.ldg + a.D) * 2);
  lo.bytes[1] = (uint32_t)(((wrows - 1) * a.ldu + a.D) * 2);
  lo.ld[0] = a.ldg;
  lo.ld[1] = a.ldu;
  lo.K = ro.K = a.D;
  ro.p[0] = ro.p[1] = a.x + m0 * a.ldx;
  ro.ld[0] = ro.ld[1] = a.ldx;
  ro.bytes[0] = ro.bytes[1] = (uint32_t)(((rows - 1) * a.ldx + a.D) * 2);
  v4f acc[T::NI][T::MJ];
  T::run(lds, lo, ro, 0, KB, KB, wave, l, acc);
  const int g = l >> 4, lr = l & 15, wn = wave / T::WM, wm = wave % T::WM, half = T::NI / 2;
#pragma unroll
  for (int j = 0; j < T::MJ; ++j) {
    const int m = 16 * (wm * T::MJ + j) + lr;
#pragma unroll
    for (int p = 0; p < half / 2; ++p) {
      const int f = wn * (16 * half) + 32 * p + 8 * g;
      if (m < rows && f < wrows) {
        float vg[8], vu[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          vg[e] = acc[2 * p + (e >> 2)][j][e & 3];
          vu[e] = acc[half + 2 * p + (e >> 2)][j][e & 3];
        }
        gated_finish<BACK>(a, m0 + m, f0 + f, vg, vu);
      }
    }
  }
#endif  // SG_DEVICE_PASS
}

// Few rows: a workgroup takes RB blocks of 16 rows of each weight and 16 MT tokens;
// its 8 waves split K and add their partial tiles in LDS.  Weights come from HBM and
// are all that counts: a wave asks for the next K block's while it multiplies one.
template <int RB, int MT, bool BACK>
__global__ void __launch_bounds__(512) k_gated_rows(GatedArgs a) {
#if SG_DEVICE_PASS
  __shared__ __attribute__((aligned(1024))) float red[8][RB * 2 * MT][64][4];
  const int t = threadIdx.x, l = t & 63, g = l >> 4, lr = l & 15;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int f0 = blockIdx.x * (16 * RB);
  const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
  const int rows = (int)min((int64_t)(16 * MT), a.T - m0), wrows = min(16 * RB, a.F - f0);
  const int KB = (a.D + 127) >> 7;
  const __amdgpu_buffer_rsrc_t rx = w4_rsrc(a.x + m0 * a.ldx, (uint32_t)(((rows - 1) * a.ldx + a.D) * 2));
  const __amdgpu_buffer_rsrc_t rg = w4_rsrc(a.gate + f0 * a.ldg, (uint32_t)(((wrows - 1) * a.ldg + a.D) * 2));
  const __amdgpu_buffer_rsrc_t ru = w4_rsrc(a.up + f0 * a.ldu, (uint32_t)(((wrows - 1) * a.ldu + a.D) * 2));
  uint32_t xo[MT], wo[RB][2];
#pragma unroll
  for (int j = 0; j < MT; ++j) xo[j] = 16 * j + lr < rows ? (uint32_t)(((16 * j + lr) * a.ldx + 8 * g) * 2) : W4_OUT;
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const int f = 16 * b + lr;
    wo[b][0] = f < wrows ? (uint32_t)((f * a.ldg + 8 * g) * 2) : W4_OUT;
    wo[b][1] = f < wrows ? (uint32_t)((f * a.ldu + 8 * g) * 2) : W4_OUT;
  }
  v4f acc[RB][2][MT];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[b][h][j] = (v4f){0.f, 0.f, 0.f, 0.f};
  v4i w[2][RB][2][4], x[2][MT][4];
  const auto load = [&](int s, int kb) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bool in = kb * 128 + 32 * q + 8 * g < a.D;
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        w[s][b][0][q] = w4_ld16(rg, in ? wo[b][0] + 64 * q : W4_OUT, kb * 256);
        w[s][b][1][q] = w4_ld16(ru, in ? wo[b][1] + 64 * q : W4_OUT, kb * 256);
      }
#pragma unroll
      for (int j = 0; j < MT; ++j) x[s][j][q] = w4_ld16(rx, in ? xo[j] + 64 * q : W4_OUT, kb * 256);
    }
  };
  const auto compute = [&](int s) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < MT; ++j) acc[b][h][j] = w4_mfma(w[s][b][h][q], x[s][j][q], acc[b][h][j]);
  };
  if (wave < KB) load(0, wave);
  for (int kb = wave; kb < KB; kb += 16) {
    if (kb + 8 < KB) load(1, kb + 8);
    compute(0);
    if (kb + 8 < KB) {
      if (kb + 16 < KB) load(0, kb + 16);
      compute(1);
    }
  }
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < MT; ++j) *reinterpret_cast<v4f*>(&red[wave][(b * 2 + h) * MT + j][l][0]) = acc[b][h][j];
  __syncthreads();
  // token 16 j + i, values 8 o .. 8 o + 7 of the workgroup's
  for (int q = t; q < 32 * RB * MT; q += 512) {
    const int i = q & 15, o = (q >> 4) % (2 * RB), j = q / (32 * RB);
    if (16 * j + i >= rows || 8 * o >= wrows) continue;
    float v[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        v4f s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 8; ++k)
          s += *reinterpret_cast<const v4f*>(&red[k][((o >> 1) * 2 + h) * MT + j][16 * (2 * (o & 1) + (e >> 2)) + i][0]);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[h][e + k] = s[k];
      }
    gated_finish<BACK>(a, m0 + 16 * j + i, f0 + 8 * o, v[0], v[1]);
  }
#endif  // SG_DEVICE_PASS
}

// dG and dU from G and U that were kept: one pass over [T, F], 8 values a thread.
struct GatedKept {
  const uint16_t *g, *u;
  int64_t ld;
};
__global__ void __launch_bounds__(256) k_gated_slopes(GatedArgs a, GatedKept k) {
#if SG_DEVICE_PASS
  a.gate_add = a.up_add = nullptr;   // G and U hold them
  const int per = a.F / 8;
  const int64_t all = a.T * per, step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += step) {
    const int64_t m = i / per;
    const int f = 8 * (int)(i - m * per);
    float g[8], u[8];
    load8(k.g + m * k.ld + f, g);
    load8(k.u + m * k.ld + f, u);
    gated_finish<true>(a, m, f, g, u);
  }
#endif
}

struct GatedGradArgs {
  int64_t T;
  int F, D;
  const uint16_t *x, *gate, *up, *dg, *du;
  int64_t ldx, ldg, ldu, ld_dgu;
  uint16_t* dx;
  int64_t ld_dx;
  uint16_t *dgate, *dup;
  int64_t ld_dw;
  float* part;      // split sums [splits][T][D]
  int splits;
};

// dX [T, D]: left the weights' columns (k across rows), right dG and dU; the sum runs
// over dG . Wg, then dU . Wu.
template <typename T>
__global__ void __launch_bounds__(T::NW * 64) k_gated_dx(GatedGradArgs a, int tiles_m, int tiles_n) {
#if SG_DEVICE_PASS
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::LDS];
  int tn, tm;
  const int tiles = tiles_m * tiles_n, b = xcd_order(blockIdx.x, tiles * a.splits);
  const int split = b / tiles;
  tile_of(b - split * tiles, tiles_m, tiles_n, tn, tm);
  const int l = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = tn * T::BN;
  const int64_t m0 = (int64_t)tm * T::BM;
  const int rows = (int)min((int64_t)T::BM, a.T - m0), cols = min(T::BN, a.D - n0);
  const int KB = (a.F + 63) >> 6;
  const int kb0 = (int)((int64_t)2 * KB * split / a.splits), kb1 = (int)((int64_t)2 * KB * (split + 1) / a.splits);
  typename T::L lo;
  typename T::R ro;
  lo.p[0] = a.gate + n0;
  lo.p[1] = a.up + n0;
  lo.ld[0] = a.ldg;
  lo.ld[1] = a.ldu;
  lo.width = (uint32_t)((a.D - n0) * 2);
  lo.K = ro.K = a.F;
  ro.p[0] = a.dg + m0 * a.ld_dgu;
  ro.p[1] = a.du + m0 * a.ld_dgu;
  ro.ld[0] = ro.ld[1] = a.ld_dgu;
  ro.bytes[0] = ro.bytes[1] = (uint32_t)(((rows - 1) * a.ld_dgu + a.F) * 2);
  v4f acc[T::NI][T::MJ];
  T::run(lds, lo, ro, kb0, kb1, KB, wave, l, acc);
  const int g = l >> 4, lr = l & 15, wn = wave / T::WM, wm = wave % T::WM;
#pragma unroll
  for (int j = 0; j < T::MJ; ++j) {
    const int m = 16 * (wm * T::MJ + j) + lr;
#pragma unroll
    for (int p = 0; p < T::NI / 2; ++p) {
      const int n = wn * (16 * T::NI) + 32 * p + 8 * g;
      if (m >= rows || n >= cols) continue;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = acc[2 * p + (e >> 2)][j][e & 3];
      if (a.splits == 1) {
        store8(a.dx + (m0 + m) * a.ld_dx + n0 + n, v);
      } else {
        float* const o = a.part + ((int64_t)split * a.T + m0 + m) * a.D + n0 + n;
        *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
  }
#endif  // SG_DEVICE_PASS
}

// The split sums of dX, added in order.
__global__ void __launch_bounds__(256) k_gated_dx_join(GatedGradArgs a) {
#if SG_DEVICE_PASS
  const int per = a.D / 8;
  const int64_t all = a.T * per, step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += step) {
    const int64_t m = i / per;
    const int n = 8 * (int)(i - m * per);
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < a.splits; ++s) {
      float t[8];
      load4(a.part + ((int64_t)s * a.T + m) * a.D + n, t);
      load4(a.part + ((int64_t)s * a.T + m) * a.D + n + 4, t + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += t[e];
    }
    store8(a.dx + m * a.ld_dx + n, v);
  }
#endif
}

// dWg and dWu [F, D]: left the columns of X, right those of dG (the first half of the
// tiles along m) or dU; the sum runs over tokens, across the rows of both.
template <typename T>
__global__ void __launch_bounds__(T::NW * 64) k_gated_dw(GatedGradArgs a, int tiles_m, int tiles_n) {
#if SG_DEVICE_PASS
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::LDS];
  int tn, tm;
  tile_coords(tiles_m, tiles_n, tn, tm);
  const int l = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool up = 2 * tm >= tiles_m;
  const int n0 = tn * T::BN, m0 = (up ? tm - tiles_m / 2 : tm) * T::BM;
  const int rows = min(T::BM, a.F - m0), cols = min(T::BN, a.D - n0);
  const int K = (int)a.T, KB = (K + 63) >> 6;
  typename T::L lo;
  typename T::R ro;
  lo.p[0] = lo.p[1] = a.x + n0;
  lo.ld[0] = lo.ld[1] = a.ldx;
  lo.width = (uint32_t)((a.D - n0) * 2);
  lo.K = ro.K = K;
  ro.p[0] = ro.p[1] = (up ? a.du : a.dg) + m0;
  ro.ld[0] = ro.ld[1] = a.ld_dgu;
  ro.width = (uint32_t)((a.F - m0) * 2);
  v4f acc[T::NI][T::MJ];
  T::run(lds, lo, ro, 0, KB, KB, wave, l, acc);
  uint16_t* const out = up ? a.dup : a.dgate;
  const int g = l >> 4, lr = l & 15, wn = wave / T::WM, wm = wave % T::WM;
#pragma unroll
  for (int j = 0; j < T::MJ; ++j) {
    const int m = 16 * (wm * T::MJ + j) + lr;
#pragma unroll
    for (int p = 0; p < T::NI / 2; ++p) {
      const int n = wn * (16 * T::NI) + 32 * p + 8 * g;
      if (m >= rows || n >= cols) continue;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = acc[2 * p + (e >> 2)][j][e & 3];
      store8(out + (int64_t)(m0 + m) * a.ld_dw + n0 + n, v);
    }
  }
#endif  // SG_DEVICE_PASS
}

// Tiles of n x m, their waves, and blocks of k in LDS.
template <bool L, bool R, typename Row = PlainRow<8>> using TileA = Bf16Tile<L, R, 2, 4, 8, 4, 3, 2, Row>;   // 256 x 256
template <bool L, bool R, typename Row = PlainRow<8>> using TileC = Bf16Tile<L, R, 2, 4, 4, 4, 3, 3, Row>;   // 128 x 256
template <bool L, bool R, typename Row = PlainRow<8>> using TileB = Bf16Tile<L, R, 2, 4, 4, 2, 5, 5, Row>;   // 128 x 128
template <bool L, bool R, typename Row = PlainRow<8>> using TileB2 = Bf16Tile<L, R, 2, 4, 4, 2, 3, 2, Row>;   // 128 x 128
template <bool L, bool R, typename Row = PlainRow<4>> using TileD = Bf16Tile<L, R, 1, 4, 4, 1, 5, 5, Row>;   // 64 x 64

template <bool BACK, int MT>
static void launch_gated_rows(const GatedArgs& a, hipStream_t st) {
  k_gated_rows<1, MT, BACK><<<dim3((unsigned)cdiv(a.F, 16), (unsigned)cdiv(a.T, 16 * MT)), 512, 0, st>>>(a);
}

template <typename T, bool BACK>
static void launch_gated_tile(const GatedArgs& a, hipStream_t st) {
  const int tm = (int)cdiv(a.T, T::BM), tn = (int)cdiv(a.F, T::BN / 2);
  k_gated_tile<T, BACK><<<(unsigned)tm * tn, T::NW * 64, 0, st>>>(a, tm, tn);
}

template <bool BACK>
static void launch_gated(const GatedArgs& a, hipStream_t st) {
  static const int few = getenv("FEW") ? atoi(getenv("FEW")) : 64;
  if (a.T <= few) {
    switch ((a.T + 15) / 16) {
      case 1: launch_gated_rows<BACK, 1>(a, st); break;
      case 2: launch_gated_rows<BACK, 2>(a, st); break;
      case 3: launch_gated_rows<BACK, 3>(a, st); break;
      default: launch_gated_rows<BACK, 4>(a, st); break;
    }
    return;
  }
  static const int way = getenv("WAY") ? atoi(getenv("WAY")) : 0;
  if (way == 1) launch_gated_tile<TileA<false, false, GatedRow<8, 8>>, BACK>(a, st);
  else if (way == 2) launch_gated_tile<TileB<false, false, GatedRow<4, 8>>, BACK>(a, st);
  else if (way == 3) launch_gated_tile<TileC<false, false, GatedRow<4, 8>>, BACK>(a, st);
  else if (way == 5) launch_gated_tile<TileB2<false, false, GatedRow<4, 8>>, BACK>(a, st);
  else if (way == 4) launch_gated_tile<TileD<false, false, GatedRow<4, 4>>, BACK>(a, st);
  else if (cdiv(a.T, 256) * cdiv(a.F, 128) >= 256) launch_gated_tile<TileA<false, false, GatedRow<8, 8>>, BACK>(a, st);
  else launch_gated_tile<TileB<false, false, GatedRow<4, 8>>, BACK>(a, st);
}

// How dX is computed: tiles of 256 or 128, parts of its sum over 2 F.
struct DxPlan {
  bool big;
  int splits;
  DxPlan(int64_t T, int64_t F, int64_t D) {
    const int64_t steps = 2 * cdiv(F, 64);
    big = cdiv(T, 256) * cdiv(D, 256) >= 64;
    const int64_t tiles = big ? cdiv(T, 256) * cdiv(D, 256) : cdiv(T, 128) * cdiv(D, 128);
    int64_t s = (big ? 256 : 512) / tiles;
    if (s > steps / 8) s = steps / 8;
    splits = (int)(s < 1 ? 1 : s > 64 ? 64 : s);
  }
  int64_t bytes(int64_t T, int64_t D) const { return splits == 1 ? 0 : 4 * splits * T * D; }
};

static bool gated_shape_ok(int64_t T, int64_t F, int64_t D) {
  if (T < 1 || F < 8 || D < 8 || F % 8 || D % 8 || T >= (1LL << 31) || F >= (1LL << 22) || D >= (1LL << 22)) return false;
  return cdiv(T, 128) * cdiv(F, 64) < (1LL << 22);
}
static bool gated_back_ok(int64_t T, int64_t F, int64_t D) {
  return gated_shape_ok(T, F, D) && cdiv(F, 128) * cdiv(D, 128) < (1LL << 22) &&
         cdiv(T, 128) * cdiv(D, 128) < (1LL << 22);
}
static bool ld_ok(int64_t ld, int64_t cols) { return ld >= cols && ld < (1LL << 22); }

}  // namespace sg

using namespace sg;

extern "C" sg_status sg_gated_gemm(int64_t T, int64_t F, int64_t D, const uint16_t* x, int64_t ldx,
                                   const uint16_t* gate, int64_t ldg, const uint16_t* up, int64_t ldu, sg_act act,
                                   const uint16_t* gate_add, const uint16_t* up_add, int64_t ld_add, void* h,
                                   sg_dtype h_dt, int64_t ldh, uint16_t* g, uint16_t* u, int64_t ld_gu,
                                   hipStream_t stream) {
  if (!x || !gate || !up || !h || !g != !u) return SG_ERR_NULL;
  if (act < SG_ACT_SILU || act > SG_ACT_RELU || (h_dt != SG_F32 && h_dt != SG_BF16)) return SG_ERR_UNSUPPORTED;
  const bool add = gate_add || up_add;
  if (!gated_shape_ok(T, F, D) || !ld_ok(ldx, D) || !ld_ok(ldg, D) || !ld_ok(ldu, D) || !ld_ok(ldh, F) ||
      (add && !ld_ok(ld_add, F)) || (g && !ld_ok(ld_gu, F)))
    return SG_ERR_SHAPE;
  if (ldx % 8 || ldg % 8 || ldu % 8 || ldh % 8 || (add && ld_add % 8) || (g && ld_gu % 8) || !aligned(x, 16) ||
      !aligned(gate, 16) || !aligned(up, 16) || !aligned(h, 16) || !aligned(gate_add, 16) || !aligned(up_add, 16) ||
      !aligned(g, 16) || !aligned(u, 16))
    return SG_ERR_ALIGN;
  GatedArgs a = {};
  a.T = T; a.F = (int)F; a.D = (int)D; a.x = x; a.gate = gate; a.up = up; a.ldx = ldx; a.ldg = ldg; a.ldu = ldu;
  a.act = act; a.gate_add = gate_add; a.up_add = up_add; a.ld_add = ld_add;
  a.h = h; a.ldh = ldh; a.h_f32 = h_dt == SG_F32; a.g = g; a.u = u; a.ld_gu = ld_gu;
  clear_hip_error();
  launch_gated<false>(a, stream);
  return launch_status();
}

extern "C" int64_t sg_gated_gemm_backward_workspace(int64_t T, int64_t F, int64_t D) {
  if (!gated_back_ok(T, F, D)) return -1;
  return DxPlan(T, F, D).bytes(T, D);
}

extern "C" sg_status sg_gated_gemm_backward(int64_t T, int64_t F, int64_t D, const uint16_t* dh, int64_t ld_dh,
                                            const uint16_t* x, int64_t ldx, const uint16_t* gate, int64_t ldg,
                                            const uint16_t* up, int64_t ldu, sg_act act, const uint16_t* g,
                                            const uint16_t* u, int64_t ld_gu, const uint16_t* gate_add,
                                            const uint16_t* up_add, int64_t ld_add, uint16_t* dg, uint16_t* du,
                                            int64_t ld_dgu, uint16_t* dx, int64_t ld_dx, uint16_t* dgate,
                                            uint16_t* dup, int64_t ld_dw, void* workspace, int64_t workspace_bytes,
                                            hipStream_t stream) {
  if (!dh || !x || !gate || !up || !dg || !du || !g != !u || !dgate != !dup) return SG_ERR_NULL;
  if (act < SG_ACT_SILU || act > SG_ACT_RELU) return SG_ERR_UNSUPPORTED;
  const bool add = gate_add || up_add;
  if (!gated_back_ok(T, F, D) || !ld_ok(ld_dh, F) || !ld_ok(ldx, D) || !ld_ok(ldg, D) || !ld_ok(ldu, D) ||
      (g && !ld_ok(ld_gu, F)) || (add && !ld_ok(ld_add, F)) || !ld_ok(ld_dgu, F) || (dx && !ld_ok(ld_dx, D)) ||
      (dgate && !ld_ok(ld_dw, D)))
    return SG_ERR_SHAPE;
  const DxPlan plan(T, F, D);
  const int64_t need = dx ? plan.bytes(T, D) : 0;
  if (need && !workspace) return SG_ERR_NULL;
  if (need > workspace_bytes) return SG_ERR_SHAPE;
  if (ld_dh % 8 || ldx % 8 || ldg % 8 || ldu % 8 || (g && ld_gu % 8) || (add && ld_add % 8) || ld_dgu % 8 ||
      (dx && ld_dx % 8) || (dgate && ld_dw % 8) || !aligned(dh, 16) || !aligned(x, 16) || !aligned(gate, 16) ||
      !aligned(up, 16) || !aligned(g, 16) || !aligned(u, 16) || !aligned(gate_add, 16) || !aligned(up_add, 16) ||
      !aligned(dg, 16) || !aligned(du, 16) || !aligned(dx, 16) || !aligned(dgate, 16) || !aligned(dup, 16) ||
      (need && !aligned(workspace, 256)))
    return SG_ERR_ALIGN;
  clear_hip_error();
  GatedArgs a = {};
  a.T = T; a.F = (int)F; a.D = (int)D; a.x = x; a.gate = gate; a.up = up; a.ldx = ldx; a.ldg = ldg; a.ldu = ldu;
  a.act = act; a.gate_add = gate_add; a.up_add = up_add; a.ld_add = ld_add;
  a.dh = dh; a.ld_dh = ld_dh; a.dg = dg; a.du = du; a.ld_dgu = ld_dgu;
  if (g) k_gated_slopes<<<grid_for(T * (F / 8), 256, 8192), 256, 0, stream>>>(a, GatedKept{g, u, ld_gu});
  else launch_gated<true>(a, stream);
  GatedGradArgs b = {};
  b.T = T; b.F = (int)F; b.D = (int)D; b.x = x; b.gate = gate; b.up = up; b.dg = dg; b.du = du;
  b.ldx = ldx; b.ldg = ldg; b.ldu = ldu; b.ld_dgu = ld_dgu; b.dx = dx; b.ld_dx = ld_dx;
  b.dgate = dgate; b.dup = dup; b.ld_dw = ld_dw; b.part = reinterpret_cast<float*>(workspace); b.splits = plan.splits;
  if (dx) {
    if (plan.big) {
      const int tm = (int)cdiv(T, 256), tn = (int)cdiv(D, 256);
      k_gated_dx<TileA<true, false>><<<(unsigned)(tm * tn * plan.splits), TileA<true, false>::NW * 64, 0, stream>>>(b, tm, tn);
    } else {
      const int tm = (int)cdiv(T, 128), tn = (int)cdiv(D, 128);
      k_gated_dx<TileB<true, false>><<<(unsigned)(tm * tn * plan.splits), TileB<true, false>::NW * 64, 0, stream>>>(b, tm, tn);
    }
    if (plan.splits > 1) k_gated_dx_join<<<grid_for(T * (D / 8), 256, 8192), 256, 0, stream>>>(b);
  }
  if (dgate) {
    if (2 * cdiv(F, 256) * cdiv(D, 256) >= 256) {
      const int tm = 2 * (int)cdiv(F, 256), tn = (int)cdiv(D, 256);
      k_gated_dw<TileA<true, true>><<<(unsigned)tm * tn, TileA<true, true>::NW * 64, 0, stream>>>(b, tm, tn);
    } else {
      const int tm = 2 * (int)cdiv(F, 128), tn = (int)cdiv(D, 128);
      k_gated_dw<TileB<true, true>><<<(unsigned)tm * tn, TileB<true, true>::NW * 64, 0, stream>>>(b, tm, tn);
    }
  }
  return launch_status();
}
