// Linear layers on dense 4-bit weights: Y = X . W^T + bias with X in bf16 and
// W as int4 codes with one fp32 scale per row and group of 32, 64 or 128
// columns (w4.h has the packed layout),
//   y[m, n] = sum_g s[n, g] sum_{k in g} x[m, k] c[n, k].
// Codes are widened to bf16 in registers (exact) and multiplied on the matrix
// core with fp32 sums; each group's partial sum is scaled in fp32, so the
// weight is never rounded.  W is the left operand: lane 16 g + r of a result
// tile holds columns n = 4 g .. 4 g + 3 of row m = r.
#include "w4_rows.h"
#include "w4_tile.h"
#include "sg_moe.h"

namespace sg {

struct W4PackArgs {
  const uint8_t* wq;
  int64_t ldw, w_bs;
  const float* s;
  int64_t s_sn, s_sk, s_bs;
  int64_t N, K;
  int KB, gc, chunk;
  int64_t RB, per;   // row blocks, bytes of one packed weight
  int64_t chunks;    // chunks of all weights
  uint8_t* out;
};

// One wave per chunk, grid-striding: a launch has threads for 2^26 of them.
__global__ void __launch_bounds__(256) k_w4_pack(W4PackArgs a) {
  const int l = threadIdx.x & 63, g = l >> 4, r = l & 15;
  const int ng = 128 / a.gc;
  const int64_t one = a.RB * a.KB;
  for (int64_t c = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); c < a.chunks; c += (int64_t)gridDim.x * 4) {
    const int64_t e = c / one, rest = c - e * one;
    const int64_t R = rest / a.KB;
    const int kb = (int)(rest - R * a.KB);
    const int64_t n = R * 16 + r;
    uint8_t* const out = a.out + e * a.per + rest * a.chunk;
    uint32_t d[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t k = (int64_t)kb * 128 + 32 * q + 8 * g;
      d[q] = n < a.N && k < a.K ? *reinterpret_cast<const uint32_t*>(a.wq + e * a.w_bs + n * a.ldw + k / 2) : 0u;
    }
    *reinterpret_cast<uint4*>(out + 16 * l) = make_uint4(d[0], d[1], d[2], d[3]);
    for (int i = l; i < 16 * ng; i += 64) {   // [group][row]
      const int64_t nr = R * 16 + (i & 15), k = (int64_t)kb * 128 + (int64_t)(i >> 4) * a.gc;
      reinterpret_cast<float*>(out + W4_CODES)[i] =
          nr < a.N && k < a.K ? a.s[e * a.s_bs + nr * a.s_sn + k / a.gc * a.s_sk] : 0.0f;
    }
  }
}

struct W4Args {
  int64_t M, N, K;
  const uint16_t* x;
  int64_t ldx;
  const uint8_t* w;
  const float* bias;
  void* y;
  int64_t ldy;
  int vec_store;
};

// Few rows: a workgroup owns RB blocks of 16 W rows and 4 XI X rows; its 8
// waves split the K blocks (w4_rows.h) and add their partial tiles in LDS.
template <int GC, int RB, int XI>
__global__ void __launch_bounds__(512) k_w4_rows(W4Args a, int out_bf16) {
#if SG_DEVICE_PASS
  using T = W4Rows<GC, RB, XI>;
  constexpr int MT = T::MT;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::LDS];
  const int t = threadIdx.x, l = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int64_t rb0 = (int64_t)blockIdx.x * RB, m0 = (int64_t)blockIdx.y * (4 * XI);
  const int xrows = (int)min((int64_t)(4 * XI), a.M - m0);
  typename T::Src s;
  s.K = (int)a.K;
  s.KB = (int)((a.K + 127) >> 7);
  s.x = a.x + m0 * a.ldx;
  s.x_bytes = (uint32_t)(((xrows - 1) * a.ldx + a.K) * 2);
#pragma unroll
  for (int rb = 0; rb < RB; ++rb)   // past N the last one again: nothing of it is stored
    s.w[rb] = a.w + min(rb0 + rb, (a.N - 1) >> 4) * s.KB * T::P::CHUNK;
#pragma unroll
  for (int i = 0; i < XI; ++i) {
    const int r = 4 * i + (l >> 4);
    s.xoff[i] = r < xrows ? (uint32_t)(r * a.ldx * 2) : W4_OUT;
  }
  v4f acc[RB][MT];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[rb][j] = (v4f){0.f, 0.f, 0.f, 0.f};
  T::multiply(lds + wave * T::WAVE_LDS, s, wave, W4_WAVES, l, acc);

  __syncthreads();
  float(*const red)[RB * MT][64][4] = reinterpret_cast<float(*)[RB * MT][64][4]>(lds);
#pragma unroll
  for (int rb = 0; rb < RB; ++rb)
#pragma unroll
    for (int j = 0; j < MT; ++j) *reinterpret_cast<v4f*>(&red[wave][rb * MT + j][l][0]) = acc[rb][j];
  __syncthreads();
  for (int q = t; q < RB * MT * 64; q += 512) {
    const int s2 = q >> 6, ll = q & 63, rb = s2 / MT, j = s2 % MT;
    if (16 * j + (ll & 15) >= xrows) continue;
    v4f v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < W4_WAVES; ++w) v += *reinterpret_cast<const v4f*>(&red[w][s2][ll][0]);
    const int64_t n = (rb0 + rb) * 16 + 4 * (ll >> 4);
    v *= W4_UNIT;
    if (a.bias) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += a.bias[min(n + e, a.N - 1)];
    }
    if (out_bf16) store_quad<true, false>(a, m0 + 16 * j + (ll & 15), n, v);
    else store_quad<false, false>(a, m0 + 16 * j + (ll & 15), n, v);
  }
#endif  // SG_DEVICE_PASS
}

// Many rows: tiles of 128 IW W rows x 128 X rows (w4_tile.h).
template <int GC, int IW>
__global__ void __launch_bounds__(512) k_w4_gemm(W4Args a, int tiles_m, int tiles_n, int out_bf16) {
#if SG_DEVICE_PASS
  using T = W4Tile<GC, IW>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::LDS];
  int tn, tm;
  tile_coords(tiles_m, tiles_n, tn, tm);
  const int64_t n0 = (int64_t)tn * T::BN, m0 = (int64_t)tm * T::BM;
  const int l = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int xrows = (int)min((int64_t)T::BM, a.M - m0);
  typename T::Src s;
  s.K = (int)a.K;
  s.KB = (int)((a.K + 127) >> 7);
  s.x = a.x + m0 * a.ldx;
  s.x_bytes = (uint32_t)(((xrows - 1) * a.ldx + a.K) * 2);
#pragma unroll
  for (int i = 0; i < IW; ++i)   // past N the last row block again: nothing of it is stored
    s.w[i] = a.w + min((n0 >> 4) + IW * wave + i, (a.N - 1) >> 4) * s.KB * T::P::CHUNK;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = T::x_row(u, wave, l);
    s.xoff[u] = r < xrows ? (uint32_t)(r * a.ldx * 2) : W4_OUT;
  }
  v4f acc[IW][8];
  T::template multiply<4>(lds, s, wave, l, acc);
  const int g = l >> 4, lr = l & 15;
#pragma unroll
  for (int i = 0; i < IW; ++i) {
    const int64_t n = n0 + (IW * wave + i) * 16 + 4 * g;
    float b[4] = {0.f, 0.f, 0.f, 0.f};
    if (a.bias) {
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = a.bias[min(n + e, a.N - 1)];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v4f v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = fmaf(acc[i][j][e], W4_UNIT, b[e]);
      if (out_bf16) store_quad<true, false>(a, m0 + j * 16 + lr, n, v);
      else store_quad<false, false>(a, m0 + j * 16 + lr, n, v);
    }
  }
#endif  // SG_DEVICE_PASS
}

template <int GC, int RB, int XI>
static void launch_w4_rows(const W4Args& a, bool b16, hipStream_t st) {
  k_w4_rows<GC, RB, XI><<<dim3((unsigned)cdiv(a.N, 16 * RB), (unsigned)cdiv(a.M, 4 * XI)), 512, 0, st>>>(a, b16);
}

// Time of the busiest compute unit per K block of 128, in units of 0.02 us at K =
// 4096: rb blocks of W rows and 4 xi X rows each (w4_rows.h), or tiles (w4_tile.h).
// 4096 x 4096, us: 64 rows: xi 8, rb 2 (308) 7.0; 12, 2 (372) 7.9; 16, 2 (436) 9.1;
// 16, 4 (616) 13.2.  16, 4 / tiles: 256 rows 14.2 / 29.3, 512 26.7 / 30.2, 600 37.7 /
// 30.7, 1024 50.9 / 37.4.  xi 6 and 10, for 8 and 12: 17 rows 5.3 / 5.4, 33 rows 6.8 /
// 6.9.  Left out, since they gave 2 % at most when they were tried: 10, 4 (40 x 14336 x
// 4096 14.0 for 12, 4's 14.1) and 14, 4 (56 x 14336 x 4096 16.2 for 16, 4's 16.5).
// The costs are those of groups of 128 (32: 64 rows 7.6, 256 rows 16.8 / 37.6), and K
// is left out of them: neither way splits it over workgroups, so sizes that fill few
// compute units are far from what memory allows (682 x 1621 x 12224 63 us, 262 x 5090 x
// 5632 30), and so is a size just past a full round of tiles (2048 x 4096 x 4096 61 us,
// 2049 rows 111).
static int64_t w4_rows_cost(int64_t M, int64_t N, int rb, int xi) {
  return cdiv(cdiv(N, 16 * rb) * cdiv(M, 4 * xi), 256) * (16 * xi + 90 * rb);
}
// Half tiles (128 W rows) where they do not fill the card: 1024 rows 38.4 us for 56.
static bool w4_half_tiles(int64_t M, int64_t N) { return cdiv(N, 128) * cdiv(M, 128) <= 256; }
static int64_t w4_tile_cost(int64_t M, int64_t N) {
  if (w4_half_tiles(M, N)) return 1300 + cdiv(N, 128) * cdiv(M, 128) * 8 / 5;
  const int64_t tiles = cdiv(N, 256) * cdiv(M, 128);
  return tiles < 256 ? 1600 + tiles * 32 / 5 : cdiv(tiles, 256) * 3240;
}

template <int GC>
static void launch_w4(const W4Args& a, bool b16, hipStream_t st) {
  int rb = 1, xi = a.M <= 4 ? 1 : a.M <= 8 ? 2 : 4;
  if (a.M > 8)
    for (int x = 4; x <= 16 && 4 * x < a.M + 16; x += x == 12 ? 4 : 2)
      // 16, 1 costs more than 8, 2 everywhere; 6, 4 more than 12, 2
      for (int r = x == 16 ? 2 : 1; r <= (x <= 6 || x == 10 ? 2 : 4); r *= 2)
        if (w4_rows_cost(a.M, a.N, r, x) < w4_rows_cost(a.M, a.N, rb, xi)) rb = r, xi = x;
  if (cdiv(a.M, 4 * xi) > 65535 || w4_tile_cost(a.M, a.N) < w4_rows_cost(a.M, a.N, rb, xi)) {
    const int64_t tm = cdiv(a.M, 128), tn = cdiv(a.N, 256), tn1 = cdiv(a.N, 128);
    if (w4_half_tiles(a.M, a.N)) k_w4_gemm<GC, 1><<<(unsigned)(tm * tn1), 512, 0, st>>>(a, (int)tm, (int)tn1, b16);
    else k_w4_gemm<GC, 2><<<(unsigned)(tm * tn), 512, 0, st>>>(a, (int)tm, (int)tn, b16);
    return;
  }
  switch (10 * xi + rb) {
    case 11: launch_w4_rows<GC, 1, 1>(a, b16, st); break;
    case 21: launch_w4_rows<GC, 1, 2>(a, b16, st); break;
    case 41: launch_w4_rows<GC, 1, 4>(a, b16, st); break;
    case 42: launch_w4_rows<GC, 2, 4>(a, b16, st); break;
    case 61: launch_w4_rows<GC, 1, 6>(a, b16, st); break;
    case 62: launch_w4_rows<GC, 2, 6>(a, b16, st); break;
    case 81: launch_w4_rows<GC, 1, 8>(a, b16, st); break;
    case 82: launch_w4_rows<GC, 2, 8>(a, b16, st); break;
    case 84: launch_w4_rows<GC, 4, 8>(a, b16, st); break;
    case 101: launch_w4_rows<GC, 1, 10>(a, b16, st); break;
    case 102: launch_w4_rows<GC, 2, 10>(a, b16, st); break;
    case 121: launch_w4_rows<GC, 1, 12>(a, b16, st); break;
    case 122: launch_w4_rows<GC, 2, 12>(a, b16, st); break;
    case 124: launch_w4_rows<GC, 4, 12>(a, b16, st); break;
    case 162: launch_w4_rows<GC, 2, 16>(a, b16, st); break;
    default: launch_w4_rows<GC, 4, 16>(a, b16, st); break;
  }
}

}  // namespace sg

using namespace sg;

extern "C" int64_t sg_w4_packed_bytes(int64_t N, int64_t K, int gc) {
  if (gc != 32 && gc != 64 && gc != 128) return -1;
  if (N < 1 || K < 1 || K % gc || N > (1LL << 31) || K > (1LL << 24)) return -1;
  return cdiv(N, 16) * cdiv(K, 128) * w4_chunk(gc);
}

extern "C" sg_status sg_w4_pack(int64_t L, const uint8_t* wq, int64_t ldw, int64_t w_bs, const float* s, int64_t s_sn,
                                int64_t s_sk, int64_t s_bs, int64_t N, int64_t K, int gc, uint8_t* packed,
                                hipStream_t stream) {
  if (!wq || !s || !packed) return SG_ERR_NULL;
  if (gc != 32 && gc != 64 && gc != 128) return SG_ERR_UNSUPPORTED;
  const int64_t per = sg_w4_packed_bytes(N, K, gc);
  if (L < 1 || per < 0 || ldw < K / 2 || w_bs < 0 || s_sn < 0 || s_sk < 0 || s_bs < 0) return SG_ERR_SHAPE;
  W4PackArgs a;
  a.KB = (int)cdiv(K, 128);
  a.RB = cdiv(N, 16);
  if (L > (1LL << 40) / (a.RB * a.KB)) return SG_ERR_SHAPE;   // 64-bit sizes
  if (!aligned(wq, 4) || ldw % 4 || w_bs % 4 || !aligned(s, 4) || !aligned(packed, 16)) return SG_ERR_ALIGN;
  a.wq = wq; a.ldw = ldw; a.w_bs = w_bs; a.s = s; a.s_sn = s_sn; a.s_sk = s_sk; a.s_bs = s_bs;
  a.N = N; a.K = K; a.gc = gc; a.chunk = w4_chunk(gc); a.per = per; a.chunks = L * a.RB * a.KB; a.out = packed;
  clear_hip_error();
  k_w4_pack<<<grid_for(a.chunks, 4, 1 << 20), 256, 0, stream>>>(a);
  return launch_status();
}

extern "C" sg_status sg_w4a16_gemm_groupwise_packed(int64_t M, int64_t N, int64_t K, const uint16_t* x, int64_t ldx,
                                                    const uint8_t* wpacked, int gc, const float* bias, void* y,
                                                    sg_dtype y_dt, int64_t ldy, hipStream_t stream) {
  if (!x || !wpacked || !y) return SG_ERR_NULL;
  if (gc != 32 && gc != 64 && gc != 128) return SG_ERR_UNSUPPORTED;
  if (y_dt != SG_F32 && y_dt != SG_BF16) return SG_ERR_UNSUPPORTED;
  if (M <= 0 || sg_w4_packed_bytes(N, K, gc) < 0 || ldx < K || ldy < N) return SG_ERR_SHAPE;
  // 32-bit buffer offsets: 256 X rows, and a tile's 8 row blocks of chunks; a launch's threads
  if (ldx >= (1LL << 22) || cdiv(K, 128) * 8 * w4_chunk(gc) >= (1LL << 31)) return SG_ERR_SHAPE;
  if (M >= (1LL << 31) || !launch_fits(cdiv(N, 16), 512) || !launch_fits(cdiv(M, 128) * cdiv(N, 256), 512))
    return SG_ERR_SHAPE;
  if (!aligned(x, 16) || (ldx * 2) % 16 || !aligned(wpacked, 16) || !aligned(bias, 4) || !aligned(y, dtype_size(y_dt)))
    return SG_ERR_ALIGN;
  W4Args a;
  a.M = M; a.N = N; a.K = K; a.x = x; a.ldx = ldx; a.w = wpacked; a.bias = bias; a.y = y; a.ldy = ldy;
  a.vec_store = (ldy % 4 == 0) && aligned(y, 4 * dtype_size(y_dt));
  clear_hip_error();
  const bool b16 = y_dt == SG_BF16;
  switch (gc) {
    case 32: launch_w4<32>(a, b16, stream); break;
    case 64: launch_w4<64>(a, b16, stream); break;
    default: launch_w4<128>(a, b16, stream); break;
  }
  return launch_status();
}
