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
// BACK: dG and dU are rounded to bf16 here, once, and as such are what is returned, what an adapter's
// backward pass takes for its dy, and the operands of dX and dW.  The matrix core takes 8 bits a value;
// two parts of each, as in lora.hip, would double its instructions, which are what the large
// gradients wait for (2048 x 11008 x 4096 540 us of 600).  Over the whole output dX and dW are off
// by 0.0023 then, where rounding them alone gives 0.0017 (tests/test_gpu_gated_formula.py).
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

// Up to 16 tokens: a workgroup takes 16 rows of each weight; its 8 waves split K and add
// their partial tiles in LDS.  Weights come from HBM and are all that counts: a wave asks
// for the next K block's while it multiplies one.  (One token, 14336 x 4096: 44 us, 5.3
// TB/s.)
template <bool BACK>
__global__ void __launch_bounds__(512) k_gated_rows(GatedArgs a) {
#if SG_DEVICE_PASS
  __shared__ __attribute__((aligned(1024))) float red[8][2][64][4];
  const int t = threadIdx.x, l = t & 63, g = l >> 4, lr = l & 15;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int f0 = blockIdx.x * 16, rows = (int)a.T, wrows = min(16, a.F - f0);
  const int KB = (a.D + 127) >> 7;
  const __amdgpu_buffer_rsrc_t rx = w4_rsrc(a.x, (uint32_t)(((rows - 1) * a.ldx + a.D) * 2));
  const __amdgpu_buffer_rsrc_t rg = w4_rsrc(a.gate + f0 * a.ldg, (uint32_t)(((wrows - 1) * a.ldg + a.D) * 2));
  const __amdgpu_buffer_rsrc_t ru = w4_rsrc(a.up + f0 * a.ldu, (uint32_t)(((wrows - 1) * a.ldu + a.D) * 2));
  const uint32_t xo = lr < rows ? (uint32_t)((lr * a.ldx + 8 * g) * 2) : W4_OUT;
  const uint32_t go = lr < wrows ? (uint32_t)((lr * a.ldg + 8 * g) * 2) : W4_OUT;
  const uint32_t uo = lr < wrows ? (uint32_t)((lr * a.ldu + 8 * g) * 2) : W4_OUT;
  v4f acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  v4i w[2][2][4], x[2][4];
  const auto load = [&](int s, int kb) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bool in = kb * 128 + 32 * q + 8 * g < a.D;
      w[s][0][q] = w4_ld16(rg, in ? go + 64 * q : W4_OUT, kb * 256);
      w[s][1][q] = w4_ld16(ru, in ? uo + 64 * q : W4_OUT, kb * 256);
      x[s][q] = w4_ld16(rx, in ? xo + 64 * q : W4_OUT, kb * 256);
    }
  };
  const auto compute = [&](int s) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int h = 0; h < 2; ++h) acc[h] = w4_mfma(w[s][h][q], x[s][q], acc[h]);
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
  for (int h = 0; h < 2; ++h) *reinterpret_cast<v4f*>(&red[wave][h][l][0]) = acc[h];
  __syncthreads();
  // token t % 16, values 8 o .. 8 o + 7 of the workgroup's
  const int i = t & 15, o = t >> 4;
  if (o >= 2 || i >= rows || 8 * o >= wrows) return;
  float v[2][8];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      v4f s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < 8; ++k) s += *reinterpret_cast<const v4f*>(&red[k][h][16 * (2 * o + (e >> 2)) + i][0]);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[h][e + k] = s[k];
    }
  gated_finish<BACK>(a, i, f0 + 8 * o, v[0], v[1]);
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
  int dx_m, dx_n, dw_m, dw_n;   // tiles of either; none of what is not asked for
};

// dX [T, D]: left the weights' columns (k across rows), right dG and dU; the sum runs
// over dG . Wg, then dU . Wu.
#if SG_DEVICE_PASS
template <typename T>
__device__ __forceinline__ void gated_dx(const GatedGradArgs& a, uint8_t* lds, int block) {
  const int tiles_m = a.dx_m, tiles_n = a.dx_n;
  int tn, tm;
  const int tiles = tiles_m * tiles_n, b = xcd_order(block, tiles * a.splits);
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
}
#endif  // SG_DEVICE_PASS

// dWg and dWu [F, D]: left the columns of X, right those of dG (the first half of the
// tiles along m) or dU; the sum runs over tokens, across the rows of both.
#if SG_DEVICE_PASS
template <typename T>
__device__ __forceinline__ void gated_dw(const GatedGradArgs& a, uint8_t* lds, int block) {
  const int tiles_m = a.dw_m, tiles_n = a.dw_n;
  int tn, tm;
  tile_of(xcd_order(block, tiles_m * tiles_n), tiles_m, tiles_n, tn, tm);
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
}
#endif  // SG_DEVICE_PASS

// Both in one launch, dX's workgroups first: theirs are the longer ones, and the others fill
// the card behind them.
template <typename TX, typename TW>
__global__ void __launch_bounds__(512) k_gated_grads(GatedGradArgs a) {
#if SG_DEVICE_PASS
  __shared__ __attribute__((aligned(1024))) uint8_t lds[TX::LDS > TW::LDS ? TX::LDS : TW::LDS];
  const int first = a.dx_m * a.dx_n * a.splits;
  if ((int)blockIdx.x < first) gated_dx<TX>(a, lds, blockIdx.x);
  else gated_dw<TW>(a, lds, blockIdx.x - first);
#endif
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

// Tiles of n x m, their waves, and blocks of k in LDS.
template <bool L, bool R, typename Row = PlainRow<8>> using TileA = Bf16Tile<L, R, true, 2, 4, 8, 4, 3, 2, Row>;   // 256 x 256
template <bool L, bool R, typename Row = PlainRow<8>> using TileC = Bf16Tile<L, R, true, 2, 4, 4, 4, 3, 3, Row>;   // 128 x 256
template <bool L, bool R, typename Row = PlainRow<8>> using TileB = Bf16Tile<L, R, false, 2, 4, 4, 2, 5, 5, Row>;   // 128 x 128
template <bool L, bool R, typename Row = PlainRow<8>> using TileE = Bf16Tile<L, R, false, 2, 4, 4, 2, 3, 2, Row>;   // 128 x 128, two a unit
template <bool L, bool R, typename Row = PlainRow<4>> using TileD = Bf16Tile<L, R, false, 1, 4, 4, 1, 5, 5, Row>;   // 64 x 64, two a unit

template <bool BACK>
static void launch_gated_rows(const GatedArgs& a, hipStream_t st) {
  k_gated_rows<BACK><<<(unsigned)cdiv(a.F, 16), 512, 0, st>>>(a);
}

template <typename T, bool BACK>
static void launch_gated_tile(const GatedArgs& a, hipStream_t st) {
  const int tm = (int)cdiv(a.T, T::BM), tn = (int)cdiv(a.F, T::BN / 2);
  k_gated_tile<T, BACK><<<(unsigned)tm * tn, T::NW * 64, 0, st>>>(a, tm, tn);
}

// Which tiles: a block of 64 k takes a workgroup about as long however many others there
// are, until they take turns.  us a block, in hundredths: 256 x 256 127, 128 x 256 93,
// 128 x 128 75, 64 x 64 50 (one a compute unit) or 73 (two).  Measured, us, tiles in
// that order, one launch after another from a graph with other weights each time (a program whose other
// data goes through the caches too sees up to 70 for the 63 of 256 tokens): 128 x 11008 x 4096 81 / 59 /
// 51 / 60; 256 tokens 81 / 63 / 85 / 96; 512 93 / 114 / 124 / 165; 1024 x 4096 x 4096 82 / 66 / 82 / 120; 333 x
// 2760 x 1032 31 / 20 / 16 / 18; 200 x 2000 x 3000 58 / 41 / 31 / 19; 64 x 5512 x 2040 53 / 33 / 30 / 21; 64 x
// 14336 x 4096 80 / 59 / 52 / 54 (the rule takes the last).
enum GatedWay { GATED_ROWS, GATED_A, GATED_B, GATED_C, GATED_D };
static GatedWay gated_way(int64_t T, int64_t F) {
  if (T <= 16) return GATED_ROWS;
  const auto tiles = [&](int bm, int bf) { return cdiv(T, bm) * cdiv(F, bf); };
  const int64_t A = 127 * cdiv(tiles(256, 128), 256), C = 93 * cdiv(tiles(256, 64), 256);
  const int64_t B = 75 * cdiv(tiles(128, 64), 256), d = tiles(64, 32), D = d <= 256 ? 50 : 73 * cdiv(d, 512);
  return A <= B && A <= C && A <= D ? GATED_A : C <= B && C <= D ? GATED_C : B <= D ? GATED_B : GATED_D;
}
template <bool BACK>
static void launch_gated(const GatedArgs& a, hipStream_t st) {
  switch (gated_way(a.T, a.F)) {
    case GATED_ROWS: return launch_gated_rows<BACK>(a, st);
    case GATED_A: return launch_gated_tile<TileA<false, false, GatedRow<8, 8>>, BACK>(a, st);
    case GATED_B: return launch_gated_tile<TileB<false, false, GatedRow<4, 8>>, BACK>(a, st);
    case GATED_C: return launch_gated_tile<TileC<false, false, GatedRow<4, 8>>, BACK>(a, st);
    case GATED_D: return launch_gated_tile<TileD<false, false, GatedRow<4, 4>>, BACK>(a, st);
  }
}

// How dX and dW are computed: tiles of 256 (one a compute unit) or 128 (two), and parts of
// dX's sum over 2 F.  By the time until all workgroups are through, the longest one's at
// least (us a block of 64 k as above and for a tile's start and end), and that of writing,
// reading and adding the parts.  With the many shorter workgroups of dW behind them, dX's
// need no parts to fill the card: 2048 x 11008 x 4096, 2 parts and their sum 591 us, none 560.
// Over 23 sizes with and without dW (20 x 512 x 1000 to 2048 x 11008 x 4096, plans in turn) the choice is 2.9%
// off the best one measured on average; furthest with dW at few tokens of wide projections: 64 x 11008 x
// 4096 125 us for 96, 128 tokens 135 for 107, 256 160 for 136, all with tiles of 256 and 8 parts; 1200 x 7168 x
// 2048 157 for 145.  333 x 2760 x 1032, whole call: 128 with 6 or 8 parts 34 us, with 16 36;
// 2048 x 4096 x 1024: 256 with 4 parts 83, 128 with 2 97.
struct GradPlan {
  bool big;
  int splits;
  GradPlan(int64_t T, int64_t F, int64_t D, bool dw) {
    const int64_t blocks = 2 * cdiv(F, 64);
    double best = 1e30;
    for (int b = 0; b < 2; ++b) {
      const int64_t t = b ? 256 : 128, nx = cdiv(T, t) * cdiv(D, t), nw = dw ? 2 * cdiv(F, t) * cdiv(D, t) : 0;
      for (int s = 1; s <= 32 && (s == 1 || 4 * s <= blocks); ++s) {
        const int64_t all = nx * s + nw, slots = b ? 256 : 512;
        const double block = b ? 1.2 : all <= 256 ? 0.8 : 1.0, ends = b ? 12.0 : 5.0;
        const double x = cdiv(blocks, s) * block + ends, w = dw ? cdiv(T, 64) * block + ends : 0.0;
        double us = x > w ? x : w;
        if (all > slots) {
          const double shared = (nx * s * x + nw * w) / slots + 0.6 * (dw ? w : x);
          if (shared > us) us = shared;
        }
        if (s > 1) us += 3.0 + 8.0 * s * T * D / 4e6;
        if (us < best) best = us, big = b, splits = s;
      }
    }
  }
  int64_t bytes(int64_t T, int64_t D) const { return splits == 1 ? 0 : 4 * splits * T * D; }
};

static bool gated_shape_ok(int64_t T, int64_t F, int64_t D) {
  if (T < 1 || F < 8 || D < 8 || F % 8 || D % 8 || T >= (1LL << 31) || F >= (1LL << 22) || D >= (1LL << 22)) return false;
  return cdiv(T, 128) * cdiv(F, 64) < (1LL << 22);
}
static bool gated_back_ok(int64_t T, int64_t F, int64_t D) {
  // tiles of both in one launch; parts are only where there are few
  return gated_shape_ok(T, F, D) && 2 * cdiv(F, 128) * cdiv(D, 128) + cdiv(T, 128) * cdiv(D, 128) < (1LL << 22);
}
static bool ld_ok(int64_t ld, int64_t cols) { return ld >= cols && ld < (1LL << 22); }

}  // namespace sg

using namespace sg;

extern "C" sg_status sg_gated_gemm_plan(int64_t T, int64_t F, int64_t D, int32_t* tokens, int32_t* values) {
  if (!tokens || !values) return SG_ERR_NULL;
  if (!gated_shape_ok(T, F, D)) return SG_ERR_SHAPE;
  const GatedWay way = gated_way(T, F);
  *tokens = way == GATED_ROWS ? 16 : way == GATED_D ? 64 : way == GATED_B ? 128 : 256;
  *values = way == GATED_ROWS ? 16 : way == GATED_D ? 32 : way == GATED_A ? 128 : 64;
  return SG_OK;
}

extern "C" sg_status sg_gated_gemm_backward_plan(int64_t T, int64_t F, int64_t D, int with_dw, int32_t* tile,
                                                 int32_t* parts) {
  if (!tile || !parts) return SG_ERR_NULL;
  if (!gated_back_ok(T, F, D)) return SG_ERR_SHAPE;
  const GradPlan plan(T, F, D, with_dw != 0);
  *tile = plan.big ? 256 : 128;
  *parts = plan.splits;
  return SG_OK;
}

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
  const int64_t with = GradPlan(T, F, D, true).bytes(T, D), without = GradPlan(T, F, D, false).bytes(T, D);
  return with > without ? with : without;
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
  const GradPlan plan(T, F, D, dgate != nullptr);
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
  const int t = plan.big ? 256 : 128;
  if (dx) b.dx_m = (int)cdiv(T, t), b.dx_n = (int)cdiv(D, t);
  if (dgate) b.dw_m = 2 * (int)cdiv(F, t), b.dw_n = (int)cdiv(D, t);
  const unsigned grid = (unsigned)(b.dx_m * b.dx_n * b.splits + b.dw_m * b.dw_n);
  if (grid && plan.big) k_gated_grads<TileA<true, false>, TileA<true, true>><<<grid, 512, 0, stream>>>(b);
  else if (grid) k_gated_grads<TileE<true, false>, TileE<true, true>><<<grid, 512, 0, stream>>>(b);
  if (dx && plan.splits > 1) k_gated_dx_join<<<grid_for(T * (D / 8), 256, 8192), 256, 0, stream>>>(b);
  return launch_status();
}
