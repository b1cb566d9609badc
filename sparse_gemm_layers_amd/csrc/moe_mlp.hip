// The routed gated MLP on 4-bit expert weights:
//   y[t] = sum_j w[t, j] Wd_e (silu(Wg_e x_t) * (Wu_e x_t)),  e = ids[t, j].
//
// Four launches.  (1) The pairs (t, j) are sorted by expert.  (2) Gate and up
// products of each expert's pairs, x rows gathered by token, silu(g) u in the
// epilogue, h in bf16 (the down product's operand on the matrix core: one
// rounding of half a step, at most 2^-8 of the value).  (3) Down products, one fp32 row
// per pair.  (4) Each token's k rows are weighted and summed in fp32 in slot
// order, so results do not depend on the order of pairs within an expert.
#include "sg_moe.h"
#include "w4.h"
#include "w4_tile.h"

namespace sg {

constexpr int MOE_EMAX = 1024;
constexpr int MOE_BM = 128;   // pairs per tile

struct MoeArgs {
  int64_t T, P;           // tokens, pairs
  int k, E, D, F;
  const uint16_t* x;
  int64_t ldx;
  const int32_t* ids;
  const float* weights;
  const uint8_t *gate, *up, *down;
  int64_t gu_bytes, d_bytes;   // one packed expert
  void* y;
  int64_t ldy;
  // workspace
  int* off;       // [E + 1] first sorted pair of each expert
  int* list;      // [P] pairs sorted by expert
  int* act;       // [E + 1] number of experts with pairs, then those
  int* tile;      // [2 * max_tiles + 1] number of tiles, then expert and first sorted pair of each
  uint16_t* h;    // [P, F], in sorted order
  float* o;       // [P, D], by pair
};

// One workgroup counts, sums and places the pairs.
__global__ void __launch_bounds__(1024) k_moe_plan(MoeArgs a) {
  __shared__ int cnt[MOE_EMAX], off[MOE_EMAX], tiles[MOE_EMAX], act[MOE_EMAX];
  const int t = threadIdx.x;
  cnt[t] = 0;
  __syncthreads();
  for (int64_t p = t; p < a.P; p += 1024) {
    const int e = a.ids[p];
    if (e >= 0 && e < a.E) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  const int c = t < a.E ? cnt[t] : 0, nt = (c + MOE_BM - 1) / MOE_BM, on = c > 0;
  off[t] = c;
  tiles[t] = nt;
  act[t] = on;
  __syncthreads();
  for (int d = 1; d < 1024; d <<= 1) {
    const int u = t >= d ? off[t - d] : 0, v = t >= d ? tiles[t - d] : 0, w = t >= d ? act[t - d] : 0;
    __syncthreads();
    off[t] += u;
    tiles[t] += v;
    act[t] += w;
    __syncthreads();
  }
  const int first = off[t] - c;
  if (t < a.E) a.off[t] = first;
  if (t == a.E - 1) {
    a.off[a.E] = off[t];
    a.tile[0] = tiles[t];
    a.act[0] = act[t];
  }
  if (on) a.act[act[t]] = t;
  for (int i = 0; i < nt; ++i) {
    a.tile[1 + 2 * (tiles[t] - nt + i)] = t;
    a.tile[2 + 2 * (tiles[t] - nt + i)] = first + i * MOE_BM;
  }
  cnt[t] = first;
  __syncthreads();
  for (int64_t p = t; p < a.P; p += 1024) {
    const int e = a.ids[p];
    if (e >= 0 && e < a.E) a.list[atomicAdd(&cnt[e], 1)] = (int)p;
  }
}

#if SG_DEVICE_PASS
__device__ __forceinline__ float silu(float g) { return g / (1.0f + __expf(-g)); }

// Adds 8 waves' partial tiles (each lane 4 floats) and gives the sum to the first wave.
template <int TILES>
__device__ __forceinline__ void join_waves(float (*red)[TILES][64][4], const v4f (&acc)[TILES], int wave, int l,
                                           v4f (&sum)[TILES]) {
#pragma unroll
  for (int i = 0; i < TILES; ++i) *reinterpret_cast<v4f*>(&red[wave][i][l][0]) = acc[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < TILES; ++i) {
    v4f v = {0.f, 0.f, 0.f, 0.f};
    if (wave == 0) {
#pragma unroll
      for (int w = 0; w < W4_WAVES; ++w) v += *reinterpret_cast<const v4f*>(&red[w][i][l][0]);
    }
    sum[i] = v;
  }
  __syncthreads();
}

// acc += the K block's product of one row block (chunk at 0 of rw) with 16 X rows.
template <int GC>
__device__ __forceinline__ void block_product(__amdgpu_buffer_rsrc_t rw, const v4i (&bx)[4], int kb, int l, v4f& acc) {
  using P = W4<GC>;
  const int g = l >> 4;
  const v4i cw = w4_ld16(rw, (uint32_t)(16 * l), kb * P::CHUNK);
  v4f sw[P::NG];
#pragma unroll
  for (int u = 0; u < P::NG; ++u)
    sw[u] = __builtin_bit_cast(v4f, w4_ld16(rw, (uint32_t)(W4_CODES + 64 * u + 16 * g), kb * P::CHUNK));
#pragma unroll
  for (int u = 0; u < P::NG; ++u) {
    v4f p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = u * P::QPG; q < (u + 1) * P::QPG; ++q) p = w4_mfma(w4_widen(cw[q]), bx[q], p);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = fmaf(p[e], sw[u][e], acc[e]);
  }
}
#endif  // SG_DEVICE_PASS

// Few pairs per expert: a workgroup takes one block of 16 rows of one active
// expert's gate and up weights; its waves split the K blocks.
template <int GC>
__global__ void __launch_bounds__(512) k_moe_gate_up_rows(MoeArgs a) {
#if SG_DEVICE_PASS
  using P = W4<GC>;
  __shared__ __attribute__((aligned(16))) float red[W4_WAVES][2][64][4];
  if ((int)blockIdx.y >= a.act[0]) return;
  const int e = a.act[1 + blockIdx.y], first = a.off[e], last = a.off[e + 1];
  const int t = threadIdx.x, l = t & 63, g = l >> 4, lr = l & 15;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int KB = (a.D + 127) >> 7;
  const int64_t at = (int64_t)e * a.gu_bytes + (int64_t)blockIdx.x * KB * P::CHUNK;
  const __amdgpu_buffer_rsrc_t rg = w4_rsrc(a.gate + at, (uint32_t)(KB * P::CHUNK));
  const __amdgpu_buffer_rsrc_t ru = w4_rsrc(a.up + at, (uint32_t)(KB * P::CHUNK));
  for (int m0 = first; m0 < last; m0 += 16) {
    const bool row = m0 + lr < last;
    const int64_t tok = row ? a.list[m0 + lr] / a.k : 0;
    const __amdgpu_buffer_rsrc_t rx = w4_rsrc(a.x, (uint32_t)(((a.T - 1) * a.ldx + a.D) * 2));
    v4f acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    for (int kb = wave; kb < KB; kb += W4_WAVES) {
      v4i bx[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        bx[q] = w4_ld16(rx, row && kb * 128 + 32 * q + 8 * g < a.D ? (uint32_t)(tok * a.ldx * 2 + 64 * q + 16 * g) + kb * 256 : 0xffffffffu, 0);
      block_product<GC>(rg, bx, kb, l, acc[0]);
      block_product<GC>(ru, bx, kb, l, acc[1]);
    }
    v4f s[2];
    join_waves<2>(red, acc, wave, l, s);
    const int f = blockIdx.x * 16 + 4 * g;
    if (wave == 0 && row && f < a.F) {   // F is a multiple of 32
      float h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = silu(s[0][i] * W4_UNIT) * (s[1][i] * W4_UNIT);
      *reinterpret_cast<uint2*>(a.h + (int64_t)(m0 + lr) * a.F + f) =
          make_uint2(f32x2_to_bf16x2(h[0], h[1]), f32x2_to_bf16x2(h[2], h[3]));
    }
  }
#endif  // SG_DEVICE_PASS
}

template <int GC>
__global__ void __launch_bounds__(512) k_moe_down_rows(MoeArgs a) {
#if SG_DEVICE_PASS
  using P = W4<GC>;
  __shared__ __attribute__((aligned(16))) float red[W4_WAVES][1][64][4];
  if ((int)blockIdx.y >= a.act[0]) return;
  const int e = a.act[1 + blockIdx.y], first = a.off[e], last = a.off[e + 1];
  const int t = threadIdx.x, l = t & 63, g = l >> 4, lr = l & 15;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int KB = (a.F + 127) >> 7;
  const __amdgpu_buffer_rsrc_t rw =
      w4_rsrc(a.down + (int64_t)e * a.d_bytes + (int64_t)blockIdx.x * KB * P::CHUNK, (uint32_t)(KB * P::CHUNK));
  for (int m0 = first; m0 < last; m0 += 16) {
    const bool row = m0 + lr < last;
    const __amdgpu_buffer_rsrc_t rx = w4_rsrc(a.h + (int64_t)m0 * a.F, (uint32_t)(min(16, last - m0) * a.F * 2));
    v4f acc[1] = {{0.f, 0.f, 0.f, 0.f}};
    for (int kb = wave; kb < KB; kb += W4_WAVES) {
      v4i bx[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        bx[q] = w4_ld16(rx, row && kb * 128 + 32 * q + 8 * g < a.F ? (uint32_t)(lr * a.F * 2 + 64 * q + 16 * g) : W4_OUT, kb * 256);
      block_product<GC>(rw, bx, kb, l, acc[0]);
    }
    v4f s[1];
    join_waves<1>(red, acc, wave, l, s);
    const int n = blockIdx.x * 16 + 4 * g;
    if (wave == 0 && row && n < a.D)
      *reinterpret_cast<v4f*>(a.o + (int64_t)a.list[m0 + lr] * a.D + n) = s[0] * W4_UNIT;
  }
#endif  // SG_DEVICE_PASS
}

#if SG_DEVICE_PASS
// The tile's product over its first `rows` pairs, in steps of 32.
template <int GC>
__device__ __forceinline__ void multiply_rows(uint8_t* lds, const typename W4Tile<GC>::Src& s, int rows, int wave,
                                              int l, v4f (&acc)[2][8]) {
  using T = W4Tile<GC>;
  if (rows > 96) T::template multiply<4>(lds, s, wave, l, acc);
  else if (rows > 64) T::template multiply<3>(lds, s, wave, l, acc);
  else if (rows > 32) T::template multiply<2>(lds, s, wave, l, acc);
  else T::template multiply<1>(lds, s, wave, l, acc);
}
#endif  // SG_DEVICE_PASS

// Many pairs per expert: tiles of MOE_BM pairs of one expert.  Gate and up: 128
// rows of each, a wave's first slot is gate's row block, its second the same of up's.
template <int GC>
__global__ void __launch_bounds__(512) k_moe_gate_up(MoeArgs a, int tiles_n) {
#if SG_DEVICE_PASS
  using T = W4Tile<GC>;
  static_assert(T::BM == MOE_BM, "tile");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::LDS];
  const int tile = blockIdx.x / tiles_n, tn = blockIdx.x % tiles_n;
  if (tile >= a.tile[0]) return;
  const int e = a.tile[1 + 2 * tile], m0 = a.tile[2 + 2 * tile], rows = min(T::BM, a.off[e + 1] - m0);
  const int l = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  typename T::Src s;
  s.K = a.D;
  s.KB = (a.D + 127) >> 7;
  const int fb = tn * 8 + wave;
  const int64_t at = (int64_t)e * a.gu_bytes + (int64_t)fb * s.KB * T::P::CHUNK;
  s.w[0] = a.gate + at;
  s.w[1] = a.up + at;
  s.w_bytes[0] = s.w_bytes[1] = fb * 16 < a.F ? (uint32_t)(s.KB * T::P::CHUNK) : 0u;
  s.x = a.x;
  s.x_bytes = (uint32_t)(((a.T - 1) * a.ldx + a.D) * 2);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = T::x_row(u, wave, l);
    s.xoff[u] = r < rows ? (uint32_t)((int64_t)(a.list[m0 + r] / a.k) * a.ldx * 2) : W4_OUT;
  }
  v4f acc[2][8];
  multiply_rows<GC>(lds, s, rows, wave, l, acc);
  const int f = fb * 16 + 4 * (l >> 4), lr = l & 15;
  if (f >= a.F) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (16 * j + lr >= rows) continue;
    float h[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) h[q] = silu(acc[0][j][q] * W4_UNIT) * (acc[1][j][q] * W4_UNIT);
    *reinterpret_cast<uint2*>(a.h + (int64_t)(m0 + 16 * j + lr) * a.F + f) =
        make_uint2(f32x2_to_bf16x2(h[0], h[1]), f32x2_to_bf16x2(h[2], h[3]));
  }
#endif  // SG_DEVICE_PASS
}

template <int GC>
__global__ void __launch_bounds__(512) k_moe_down(MoeArgs a, int tiles_n) {
#if SG_DEVICE_PASS
  using T = W4Tile<GC>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::LDS];
  const int tile = blockIdx.x / tiles_n, tn = blockIdx.x % tiles_n;
  if (tile >= a.tile[0]) return;
  const int e = a.tile[1 + 2 * tile], m0 = a.tile[2 + 2 * tile], rows = min(T::BM, a.off[e + 1] - m0);
  const int l = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  typename T::Src s;
  s.K = a.F;
  s.KB = (a.F + 127) >> 7;
  s.x = a.h + (int64_t)m0 * a.F;
  s.x_bytes = (uint32_t)(rows * a.F * 2);
  const int rb0 = tn * 16 + 2 * wave;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    s.w[i] = a.down + (int64_t)e * a.d_bytes + (int64_t)(rb0 + i) * s.KB * T::P::CHUNK;
    s.w_bytes[i] = (rb0 + i) * 16 < a.D ? (uint32_t)(s.KB * T::P::CHUNK) : 0u;
    const int r = T::x_row(i, wave, l);
    s.xoff[i] = r < rows ? (uint32_t)(r * a.F * 2) : W4_OUT;
  }
  v4f acc[2][8];
  multiply_rows<GC>(lds, s, rows, wave, l, acc);
  const int g = l >> 4, lr = l & 15;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (16 * j + lr >= rows) continue;
    float* const row = a.o + (int64_t)a.list[m0 + 16 * j + lr] * a.D;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int n = (rb0 + i) * 16 + 4 * g;
      if (n < a.D) *reinterpret_cast<v4f*>(row + n) = acc[i][j] * W4_UNIT;
    }
  }
#endif  // SG_DEVICE_PASS
}

// y[t] = sum_j w[t, j] o[t k + j], 4 columns a thread, in slot order.
template <bool OUT_BF16>
__global__ void __launch_bounds__(256) k_moe_combine(MoeArgs a) {
  const int per = a.D / 4;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.T * per; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / per;
    const int n = (int)(i - t * per) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < a.k; ++j) {
      const int64_t p = t * a.k + j;
      const int e = a.ids[p];
      if (e < 0 || e >= a.E) continue;
      const float w = a.weights[p];
      const float4 o = *reinterpret_cast<const float4*>(a.o + p * a.D + n);
      v.x = fmaf(w, o.x, v.x); v.y = fmaf(w, o.y, v.y); v.z = fmaf(w, o.z, v.z); v.w = fmaf(w, o.w, v.w);
    }
    if (OUT_BF16)
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.y) + t * a.ldy + n) =
          make_uint2(f32x2_to_bf16x2(v.x, v.y), f32x2_to_bf16x2(v.z, v.w));
    else
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.y) + t * a.ldy + n) = v;
  }
}

static int64_t moe_tiles(int64_t P, int64_t E) { return cdiv(P, MOE_BM) + (P < E ? P : E); }

// Offsets of the workspace's parts; `bytes` its size.
struct MoeSpace {
  int64_t off, list, act, tile, h, o, bytes;
  MoeSpace(int64_t P, int64_t E, int64_t D, int64_t F) {
    int64_t at = 0;
    const auto part = [&](int64_t n) { const int64_t was = at; at += cdiv(n, 256) * 256; return was; };
    off = part(4 * (E + 1));
    list = part(4 * P);
    act = part(4 * (E + 1));
    tile = part(4 * (2 * moe_tiles(P, E) + 1));
    h = part(2 * P * F);
    o = part(4 * P * D);
    bytes = at;
  }
};

template <int GC>
static void launch_moe(const MoeArgs& a, bool bf16, hipStream_t st) {
  k_moe_plan<<<1, 1024, 0, st>>>(a);
  if (a.P <= 16LL * a.E) {
    const unsigned gy = (unsigned)(a.P < a.E ? a.P : a.E);
    k_moe_gate_up_rows<GC><<<dim3((unsigned)cdiv(a.F, 16), gy), 512, 0, st>>>(a);
    k_moe_down_rows<GC><<<dim3((unsigned)cdiv(a.D, 16), gy), 512, 0, st>>>(a);
  } else {
    const int tm = (int)moe_tiles(a.P, a.E), ng = (int)cdiv(a.F, 128), nd = (int)cdiv(a.D, 256);
    k_moe_gate_up<GC><<<(unsigned)(tm * ng), 512, 0, st>>>(a, ng);
    k_moe_down<GC><<<(unsigned)(tm * nd), 512, 0, st>>>(a, nd);
  }
  const unsigned grid = grid_for(a.T * (a.D / 4), 256, 8192);
  if (bf16) k_moe_combine<true><<<grid, 256, 0, st>>>(a);
  else k_moe_combine<false><<<grid, 256, 0, st>>>(a);
}

// The limits shared by the call and its workspace size.
static bool moe_shape_ok(int64_t T, int k, int64_t E, int64_t D, int64_t F) {
  if (T < 1 || k < 1 || E < 1 || E > MOE_EMAX || D < 32 || F < 32 || D % 32 || F % 32) return false;
  if (D >= (1LL << 22) || F >= (1LL << 22) || T > (1LL << 30) / k) return false;
  return (moe_tiles(T * k, E) + 1) * cdiv(D > F ? D : F, 64) < (1LL << 31);
}

}  // namespace sg

using namespace sg;

extern "C" int64_t sg_w4a16_moe_mlp_workspace(int64_t T, int k, int64_t E, int64_t D, int64_t F) {
  if (!moe_shape_ok(T, k, E, D, F)) return -1;
  return MoeSpace(T * k, E, D, F).bytes;
}

extern "C" sg_status sg_w4a16_moe_mlp(int64_t T, int k, int64_t E, int64_t D, int64_t F, const uint16_t* x,
                                      int64_t ldx, const int32_t* ids, const float* weights, const uint8_t* gate,
                                      const uint8_t* up, const uint8_t* down, int gc, void* y, sg_dtype y_dt,
                                      int64_t ldy, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  if (!x || !ids || !weights || !gate || !up || !down || !y || !workspace) return SG_ERR_NULL;
  if (gc != 32 && gc != 64 && gc != 128) return SG_ERR_UNSUPPORTED;
  if (y_dt != SG_F32 && y_dt != SG_BF16) return SG_ERR_UNSUPPORTED;
  if (!moe_shape_ok(T, k, E, D, F) || D % gc || F % gc || ldx < D || ldy < D || ldy % 4) return SG_ERR_SHAPE;
  if (T > (1LL << 30) / ldx) return SG_ERR_SHAPE;   // 32-bit buffer offsets into x
  const MoeSpace ws(T * k, E, D, F);
  if (workspace_bytes < ws.bytes) return SG_ERR_SHAPE;
  if (!aligned(x, 16) || ldx % 8 || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(gate, 16) ||
      !aligned(up, 16) || !aligned(down, 16) || !aligned(y, 4 * dtype_size(y_dt)) || !aligned(workspace, 256))
    return SG_ERR_ALIGN;
  uint8_t* const w = reinterpret_cast<uint8_t*>(workspace);
  MoeArgs a;
  a.T = T; a.P = T * k; a.k = k; a.E = (int)E; a.D = (int)D; a.F = (int)F;
  a.x = x; a.ldx = ldx; a.ids = ids; a.weights = weights; a.gate = gate; a.up = up; a.down = down;
  a.gu_bytes = sg_w4_packed_bytes(F, D, gc); a.d_bytes = sg_w4_packed_bytes(D, F, gc);
  a.y = y; a.ldy = ldy;
  a.off = reinterpret_cast<int*>(w + ws.off); a.list = reinterpret_cast<int*>(w + ws.list);
  a.act = reinterpret_cast<int*>(w + ws.act); a.tile = reinterpret_cast<int*>(w + ws.tile);
  a.h = reinterpret_cast<uint16_t*>(w + ws.h); a.o = reinterpret_cast<float*>(w + ws.o);
  clear_hip_error();
  const bool b16 = y_dt == SG_BF16;
  switch (gc) {
    case 32: launch_moe<32>(a, b16, stream); break;
    case 64: launch_moe<64>(a, b16, stream); break;
    default: launch_moe<128>(a, b16, stream); break;
  }
  return launch_status();
}
