// Linear layers on dense 4-bit weights: Y = X . W^T + bias with X in bf16 and
// W as int4 codes with one fp32 scale per row and group of 32, 64 or 128
// columns (w4.h has the packed layout),
//   y[m, n] = sum_g s[n, g] sum_{k in g} x[m, k] c[n, k].
// Codes are widened to bf16 in registers (exact) and multiplied on the matrix
// core with fp32 sums; each group's partial sum is scaled in fp32, so the
// weight is never rounded.  W is the left operand: lane 16 g + r of a result
// tile holds columns n = 4 g .. 4 g + 3 of row m = r.
#include "w4.h"
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

// One wave per chunk.
__global__ void __launch_bounds__(256) k_w4_pack(W4PackArgs a) {
  const int l = threadIdx.x & 63, g = l >> 4, r = l & 15;
  const int64_t c = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (c >= a.chunks) return;
  const int64_t one = a.RB * a.KB, e = c / one, rest = c - e * one;
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
  const int ng = 128 / a.gc;
  for (int i = l; i < 16 * ng; i += 64) {   // [group][row]
    const int64_t nr = R * 16 + (i & 15), k = (int64_t)kb * 128 + (int64_t)(i >> 4) * a.gc;
    reinterpret_cast<float*>(out + W4_CODES)[i] =
        nr < a.N && k < a.K ? a.s[e * a.s_bs + nr * a.s_sn + k / a.gc * a.s_sk] : 0.0f;
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

// Few rows (M <= 64 per grid row): a workgroup owns RB blocks of 16 W rows and
// 16 MT X rows; its 8 waves split the K blocks and add their partial tiles in
// LDS.  Operands come straight into registers: the packed codes are one
// 16-byte load per lane, X rows come from L2.
template <int GC, int RB, int MT, bool OUT_BF16>
__global__ void __launch_bounds__(512) k_w4_rows(W4Args a) {
#if SG_DEVICE_PASS
  using P = W4<GC>;
  __shared__ __attribute__((aligned(16))) float red[W4_WAVES][RB * MT][64][4];
  const int t = threadIdx.x, l = t & 63, g = l >> 4, lr = l & 15;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int KB = (int)((a.K + 127) >> 7);
  const int64_t rb0 = (int64_t)blockIdx.x * RB, m0 = (int64_t)blockIdx.y * (16 * MT);
  const int nrb = (int)min((int64_t)RB, ((a.N + 15) >> 4) - rb0);
  const int xrows = (int)min((int64_t)(16 * MT), a.M - m0);
  const __amdgpu_buffer_rsrc_t rw = w4_rsrc(a.w + rb0 * KB * P::CHUNK, (uint32_t)(nrb * KB * P::CHUNK));
  const __amdgpu_buffer_rsrc_t rx = w4_rsrc(a.x + m0 * a.ldx, (uint32_t)(((xrows - 1) * a.ldx + a.K) * 2));

  v4f acc[RB][MT];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[rb][j] = (v4f){0.f, 0.f, 0.f, 0.f};

  for (int kb = wave; kb < KB; kb += W4_WAVES) {
    v4i cw[RB], bx[MT][4];
    v4f sw[RB][P::NG];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      cw[rb] = w4_ld16(rw, (uint32_t)(rb * KB * P::CHUNK + 16 * l), kb * P::CHUNK);
#pragma unroll
      for (int u = 0; u < P::NG; ++u)
        sw[rb][u] = __builtin_bit_cast(
            v4f, w4_ld16(rw, (uint32_t)(rb * KB * P::CHUNK + W4_CODES + 64 * u + 16 * g), kb * P::CHUNK));
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bool in = kb * 128 + 32 * q + 8 * g < a.K;
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const int r = 16 * j + lr;
        bx[j][q] = w4_ld16(rx, in && r < xrows ? (uint32_t)(r * a.ldx * 2 + 64 * q + 16 * g) : W4_OUT, kb * 256);
      }
    }
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      v4i aw[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) aw[q] = w4_widen(cw[rb][q]);
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int u = 0; u < P::NG; ++u) {
          v4f p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = u * P::QPG; q < (u + 1) * P::QPG; ++q) p = w4_mfma(aw[q], bx[j][q], p);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[rb][j][e] = fmaf(p[e], sw[rb][u][e], acc[rb][j][e]);
        }
    }
  }

#pragma unroll
  for (int rb = 0; rb < RB; ++rb)
#pragma unroll
    for (int j = 0; j < MT; ++j) *reinterpret_cast<v4f*>(&red[wave][rb * MT + j][l][0]) = acc[rb][j];
  __syncthreads();
  for (int q = t; q < RB * MT * 64; q += 512) {
    const int s = q >> 6, ll = q & 63, rb = s / MT, j = s % MT;
    v4f v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < W4_WAVES; ++w) v += *reinterpret_cast<const v4f*>(&red[w][s][ll][0]);
    const int64_t n = (rb0 + rb) * 16 + 4 * (ll >> 4);
    v *= W4_UNIT;
    if (a.bias) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += a.bias[min(n + e, a.N - 1)];
    }
    store_quad<OUT_BF16, false>(a, m0 + 16 * j + (ll & 15), n, v);
  }
#endif  // SG_DEVICE_PASS
}

// Many rows: tiles of 256 W rows x 128 X rows (w4_tile.h).
template <int GC, bool OUT_BF16>
__global__ void __launch_bounds__(512) k_w4_gemm(W4Args a, int tiles_m, int tiles_n) {
#if SG_DEVICE_PASS
  using T = W4Tile<GC>;
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
  for (int i = 0; i < 2; ++i) {
    const int64_t rb = (n0 >> 4) + 2 * wave + i;
    s.w[i] = a.w + rb * s.KB * T::P::CHUNK;
    s.w_bytes[i] = rb * 16 < a.N ? (uint32_t)(s.KB * T::P::CHUNK) : 0u;
    const int r = T::x_row(i, wave, l);
    s.xoff[i] = r < xrows ? (uint32_t)(r * a.ldx * 2) : W4_OUT;
  }
  v4f acc[2][8];
  T::template multiply<4>(lds, s, wave, l, acc);
  const int g = l >> 4, lr = l & 15;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t n = n0 + (2 * wave + i) * 16 + 4 * g;
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
      store_quad<OUT_BF16, false>(a, m0 + j * 16 + lr, n, v);
    }
  }
#endif  // SG_DEVICE_PASS
}

template <int GC, int MT, bool OUT_BF16>
static void launch_w4_mt(const W4Args& a, hipStream_t st) {
  const int64_t rows16 = cdiv(a.N, 16);
  const unsigned gy = (unsigned)cdiv(a.M, 16 * MT);
  if (MT > 1 && rows16 * gy >= 2 * 224)
    k_w4_rows<GC, 2, MT, OUT_BF16><<<dim3((unsigned)cdiv(rows16, 2), gy), 512, 0, st>>>(a);
  else
    k_w4_rows<GC, 1, MT, OUT_BF16><<<dim3((unsigned)rows16, gy), 512, 0, st>>>(a);
}

template <int GC, bool OUT_BF16>
static void launch_w4(const W4Args& a, hipStream_t st) {
  if (a.M > 256) {
    using T = W4Tile<GC>;
    const int64_t tm = cdiv(a.M, T::BM), tn = cdiv(a.N, T::BN);
    k_w4_gemm<GC, OUT_BF16><<<(unsigned)(tm * tn), 512, 0, st>>>(a, (int)tm, (int)tn);
    return;
  }
  if (a.M <= 16) launch_w4_mt<GC, 1, OUT_BF16>(a, st);
  else if (a.M <= 32) launch_w4_mt<GC, 2, OUT_BF16>(a, st);
  else if (a.M <= 48) launch_w4_mt<GC, 3, OUT_BF16>(a, st);
  else launch_w4_mt<GC, 4, OUT_BF16>(a, st);
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
  if (L > (1LL << 33) / (a.RB * a.KB)) return SG_ERR_SHAPE;   // workgroups: a quarter of the chunks
  if (!aligned(wq, 4) || ldw % 4 || w_bs % 4 || !aligned(s, 4) || !aligned(packed, 16)) return SG_ERR_ALIGN;
  a.wq = wq; a.ldw = ldw; a.w_bs = w_bs; a.s = s; a.s_sn = s_sn; a.s_sk = s_sk; a.s_bs = s_bs;
  a.N = N; a.K = K; a.gc = gc; a.chunk = w4_chunk(gc); a.per = per; a.chunks = L * a.RB * a.KB; a.out = packed;
  clear_hip_error();
  k_w4_pack<<<(unsigned)cdiv(a.chunks, 4), 256, 0, stream>>>(a);
  return launch_status();
}

extern "C" sg_status sg_w4a16_gemm_groupwise_packed(int64_t M, int64_t N, int64_t K, const uint16_t* x, int64_t ldx,
                                                    const uint8_t* wpacked, int gc, const float* bias, void* y,
                                                    sg_dtype y_dt, int64_t ldy, hipStream_t stream) {
  if (!x || !wpacked || !y) return SG_ERR_NULL;
  if (gc != 32 && gc != 64 && gc != 128) return SG_ERR_UNSUPPORTED;
  if (y_dt != SG_F32 && y_dt != SG_BF16) return SG_ERR_UNSUPPORTED;
  if (M <= 0 || sg_w4_packed_bytes(N, K, gc) < 0 || ldx < K || ldy < N) return SG_ERR_SHAPE;
  // 32-bit buffer offsets: 256 X rows, and a tile's 8 row blocks of chunks; a 32-bit tile count
  if (ldx >= (1LL << 22) || cdiv(K, 128) * 8 * w4_chunk(gc) >= (1LL << 31)) return SG_ERR_SHAPE;
  if (M >= (1LL << 31) || cdiv(M, 128) * cdiv(N, 256) > 0x7fffffffLL) return SG_ERR_SHAPE;
  if (!aligned(x, 16) || (ldx * 2) % 16 || !aligned(wpacked, 16) || !aligned(bias, 4) || !aligned(y, dtype_size(y_dt)))
    return SG_ERR_ALIGN;
  W4Args a;
  a.M = M; a.N = N; a.K = K; a.x = x; a.ldx = ldx; a.w = wpacked; a.bias = bias; a.y = y; a.ldy = ldy;
  a.vec_store = (ldy % 4 == 0) && aligned(y, 4 * dtype_size(y_dt));
  clear_hip_error();
  const bool b16 = y_dt == SG_BF16;
  switch (gc) {
    case 32: b16 ? launch_w4<32, true>(a, stream) : launch_w4<32, false>(a, stream); break;
    case 64: b16 ? launch_w4<64, true>(a, stream) : launch_w4<64, false>(a, stream); break;
    default: b16 ? launch_w4<128, true>(a, stream) : launch_w4<128, false>(a, stream); break;
  }
  return launch_status();
}
