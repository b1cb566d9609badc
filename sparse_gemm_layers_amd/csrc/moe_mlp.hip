// The routed gated MLP on 4-bit expert weights:
//   y[t] = sum_j w[t, j] Wd_e (silu(Wg_e x_t) * (Wu_e x_t)),  e = ids[t, j].
//
// Many pairs per expert, four launches.  (1) The pairs (t, j) are sorted by
// expert.  (2) Gate and up products of each expert's pairs, x rows gathered by
// token, silu(g) u in the epilogue, h in bf16 (the down product's operand on the
// matrix core: one rounding of half a step, at most 2^-8 of the value).  (3) Down
// products, one fp32 row per pair.  (4) Each token's k rows are weighted and
// summed in fp32 in slot order, so results do not depend on the order of pairs
// within an expert.
// Few pairs per expert: no sorting, the products' workgroups find their pairs; a
// handful of pairs: no fourth launch either, the down kernel adds up each token's
// experts.
#include "sg_moe.h"
#include "w4_rows.h"
#include "w4_tile.h"

namespace sg {

constexpr int MOE_EMAX = 1024;
constexpr int MOE_BM = 128;   // pairs per tile
constexpr int MOE_FEW = 16;   // pairs of the shortest calls: a wave holds them all

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
  int* tile;      // [2 * max_tiles + 1] number of tiles, then expert and first sorted pair of each
  uint16_t* h;    // [P, F], in sorted order; with few pairs by pair
  float* o;       // [P, D], by pair
};

// One workgroup counts, sums and places the pairs.  Up to 16 pairs a thread stay
// in registers between counting and placing, each with its rank in its expert.
// (16384 pairs: 18 us when the ids were read and counted twice, 12 so; beyond, they are.)
constexpr int PLAN_KEEP = 16;
__global__ void __launch_bounds__(1024) k_moe_plan(MoeArgs a) {
  __shared__ int cnt[MOE_EMAX], wsum[16], wtiles[16];
  const int t = threadIdx.x, l = t & 63, wave = t >> 6;
  const bool keep = a.P <= 1024 * PLAN_KEEP;
  int id[PLAN_KEEP], rank[PLAN_KEEP];
  cnt[t] = 0;
  if (keep) {
#pragma unroll
    for (int i = 0; i < PLAN_KEEP; ++i) {
      const int p = i * 1024 + t;
      const int e = p < a.P ? a.ids[p] : -1;
      id[i] = e >= 0 && e < a.E ? e : -1;
    }
  }
  __syncthreads();
  if (keep) {
#pragma unroll
    for (int i = 0; i < PLAN_KEEP; ++i)
      if (id[i] >= 0) rank[i] = atomicAdd(&cnt[id[i]], 1);
  } else {
    for (int64_t p = t; p < a.P; p += 1024) {
      const int e = a.ids[p];
      if (e >= 0 && e < a.E) atomicAdd(&cnt[e], 1);
    }
  }
  __syncthreads();
  const int c = t < a.E ? cnt[t] : 0, nt = (c + MOE_BM - 1) / MOE_BM;
  int off = c, tiles = nt;   // sums up to this expert
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(off, d, 64), v = __shfl_up(tiles, d, 64);
    if (l >= d) off += u, tiles += v;
  }
  if (l == 63) wsum[wave] = off, wtiles[wave] = tiles;
  __syncthreads();
  for (int w = 0; w < wave; ++w) off += wsum[w], tiles += wtiles[w];
  const int first = off - c;
  if (t < a.E) a.off[t] = first;
  if (t == a.E - 1) {
    a.off[a.E] = off;
    a.tile[0] = tiles;
  }
  for (int i = 0; i < nt; ++i) {
    a.tile[1 + 2 * (tiles - nt + i)] = t;
    a.tile[2 + 2 * (tiles - nt + i)] = first + i * MOE_BM;
  }
  cnt[t] = first;
  __syncthreads();
  if (keep) {
#pragma unroll
    for (int i = 0; i < PLAN_KEEP; ++i)
      if (id[i] >= 0) a.list[cnt[id[i]] + rank[i]] = i * 1024 + t;
  } else {
    for (int64_t p = t; p < a.P; p += 1024) {
      const int e = a.ids[p];
      if (e >= 0 && e < a.E) a.list[atomicAdd(&cnt[e], 1)] = (int)p;
    }
  }
}

#if SG_DEVICE_PASS
__device__ __forceinline__ float silu(float g) { return g / (1.0f + __expf(-g)); }

// This wave's LDS accesses before are done before those after.
__device__ __forceinline__ void wave_order() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// The pairs of expert e, in order: their number; the first one; list (this
// wave's LDS) holds those of rank m0 .. m0 + n - 1.  v: ids[l], -1 past the end.
__device__ __forceinline__ int find_pairs(const int32_t* ids, int P, int v, int e, int m0, int n, int* list, int l,
                                          int& first) {
  int cnt = 0;
  first = P;
  for (int c0 = 0; c0 < P; c0 += 512) {
    int id[8];   // all on their way before the first is looked at
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int p = c0 + 64 * i + l;
      id[i] = p == l ? v : p < P ? ids[p] : -1;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool hit = id[i] == e;
      const uint64_t m = __ballot(hit);
      const int rank = cnt + __builtin_popcountll(m & ((1ull << l) - 1)) - m0;
      if (hit && rank >= 0 && rank < n) list[rank] = c0 + 64 * i + l;
      if (cnt == 0 && m) first = c0 + 64 * i + __builtin_ctzll(m);
      cnt += __builtin_popcountll(m);
    }
  }
  wave_order();
  return cnt;
}

// The expert of workgroup row y: with fewer pairs than experts the one of pair
// y, otherwise expert y; -1 where the pair is empty.
__device__ __forceinline__ int row_expert(const MoeArgs& a, int v, int y) {
  const int e = a.P > a.E ? y : y < 64 ? __builtin_amdgcn_readlane(v, y) : a.ids[y];
  return __builtin_amdgcn_readfirstlane(e >= 0 && e < a.E ? e : -1);
}

// Adds 8 waves' partial tile i (each lane 4 floats), for the lanes of one wave.
template <int TILES>
__device__ __forceinline__ v4f join_waves(const uint8_t* lds, int i, int l) {
  const float(*const red)[TILES][64][4] = reinterpret_cast<const float(*)[TILES][64][4]>(lds);
  v4f v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < W4_WAVES; ++w) v += *reinterpret_cast<const v4f*>(&red[w][i][l][0]);
  return v;
}
template <int TILES>
__device__ __forceinline__ void give_tile(uint8_t* lds, int wave, int i, int l, const v4f& v) {
  float(*const red)[TILES][64][4] = reinterpret_cast<float(*)[TILES][64][4]>(lds);
  *reinterpret_cast<v4f*>(&red[wave][i][l][0]) = v;
}
#endif  // SG_DEVICE_PASS

// A handful of pairs (P <= MOE_FEW): a workgroup takes one block of 16 rows of one
// expert's gate and up weights, finds that expert's pairs by itself (no sorting
// launch before it: 5 us) and takes 4 XI of them a pass; its waves split the K
// blocks.  One token of 64 experts (4096, 1024, k 8): 12 us for 36 MB, of which
// 2.5 are the launch and 1.5 the ids' way from memory; the down product 8.
template <int GC, int XI>
__global__ void __launch_bounds__(512) k_moe_gate_up_rows(MoeArgs a) {
#if SG_DEVICE_PASS
  using T = W4Rows<GC, 2, XI>;
  static_assert(T::MT == 1, "one sub-tile");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::LDS];
  const int t = threadIdx.x, l = t & 63, g = l >> 4, lr = l & 15;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6), P = (int)a.P;
  const int v = l < P ? a.ids[l] : -1;
  const int e = row_expert(a, v, blockIdx.y);
  if (e < 0) return;
  uint8_t* const mine = lds + wave * T::WAVE_LDS;
  int* const list = reinterpret_cast<int*>(mine);
  typename T::Src s;
  s.K = a.D;
  s.KB = (a.D + 127) >> 7;
  s.x = a.x;
  s.x_bytes = (uint32_t)(((a.T - 1) * a.ldx + a.D) * 2);
  const int64_t at = (int64_t)e * a.gu_bytes + (int64_t)blockIdx.x * s.KB * T::P::CHUNK;
  s.w[0] = a.gate + at;
  s.w[1] = a.up + at;
  int first, cnt = 1;
  for (int m0 = 0; m0 < cnt; m0 += 4 * XI) {
    cnt = find_pairs(a.ids, P, v, e, m0, 4 * XI, list, l, first);
    if (cnt == 0 || (a.P <= a.E && first != (int)blockIdx.y)) return;   // the same for every wave
    const int n = min(4 * XI, cnt - m0);
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const int r = 4 * i + g;
      s.xoff[i] = r < n ? (uint32_t)((int64_t)(list[r] / a.k) * a.ldx * 2) : W4_OUT;
    }
    const int pair = lr < n ? list[lr] : -1;
    wave_order();
    v4f acc[2][1] = {{{0.f, 0.f, 0.f, 0.f}}, {{0.f, 0.f, 0.f, 0.f}}};
    T::multiply(mine, s, wave, W4_WAVES, l, acc);
    __syncthreads();
    give_tile<2>(lds, wave, 0, l, acc[0][0]);
    give_tile<2>(lds, wave, 1, l, acc[1][0]);
    __syncthreads();
    const int f = blockIdx.x * 16 + 4 * g;
    if (wave == 0 && pair >= 0 && f < a.F) {   // F is a multiple of 32
      const v4f gs = join_waves<2>(lds, 0, l) * W4_UNIT, us = join_waves<2>(lds, 1, l) * W4_UNIT;
      float h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = silu(gs[i]) * us[i];
      *reinterpret_cast<uint2*>(a.h + (int64_t)pair * a.F + f) =
          make_uint2(f32x2_to_bf16x2(h[0], h[1]), f32x2_to_bf16x2(h[2], h[3]));
    }
    __syncthreads();
  }
#endif  // SG_DEVICE_PASS
}

// Its down product: a workgroup takes 16 rows of every active expert's down weight and adds up their weighted products itself.  X row t is
// token t's; waves take whole experts, or parts of one's K blocks where there
// are fewer than 8.  Duplicates of an expert in a token share a row: their
// weights are added.
template <int GC, int XI>
__global__ void __launch_bounds__(512) k_moe_down_join(MoeArgs a, int out_bf16) {
#if SG_DEVICE_PASS
  using T = W4Rows<GC, 1, XI>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::LDS];
  const int t = threadIdx.x, l = t & 63, g = l >> 4, lr = l & 15;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6), P = (int)a.P;
  const int v = l < P ? a.ids[l] : -1;
  const float wl = l < P ? a.weights[l] : 0.f;
  const bool live = v >= 0 && v < a.E;
  bool again = false;   // an earlier pair has this expert
  for (int p = 0; p < P; ++p) again = again || (p < l && __builtin_amdgcn_readlane(v, p) == v);
  uint64_t lead = __ballot(live && !again);
  const int na = __builtin_popcountll(lead), parts = na >= W4_WAVES ? 1 : na > 0 ? W4_WAVES / na : 1;
  typename T::Src s;
  s.K = a.F;
  s.KB = (a.F + 127) >> 7;
  s.x = a.h;
  s.x_bytes = (uint32_t)(a.P * a.F * 2);
  v4f sum = {0.f, 0.f, 0.f, 0.f};
  int at = 0;   // rank of the expert in hand
  for (; lead; lead &= lead - 1, ++at) {
    const int turn = at % W4_WAVES;   // wave of its first part; at < na <= 16
    if (parts == 1 ? turn != wave : wave % na != at || wave / na >= parts) continue;
    const int e = __builtin_amdgcn_readlane(v, __builtin_ctzll(lead));
    const uint64_t m = __ballot(v == e);
    const auto row_pair = [&](int r) {   // token r's first pair with e
      const uint64_t b = r < (int)a.T ? (m >> (r * a.k)) & ((1ull << a.k) - 1) : 0;
      return b ? r * a.k + (int)__builtin_ctzll(b) : -1;
    };
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const int p = row_pair(4 * i + g);
      s.xoff[i] = p >= 0 ? (uint32_t)p * (a.F * 2) : W4_OUT;
    }
    float w = 0.f;
    bool mine = false;   // token lr has this expert: another's infinities stay out of its sum
    for (int j = 0; j < a.k; ++j) {
      const int p = min(lr * a.k + j, 63);
      const float u = __shfl(wl, p, 64);
      const bool in = lr < (int)a.T && ((m >> p) & 1);
      w += in ? u : 0.f;
      mine = mine || in;
    }
    s.w[0] = a.down + (int64_t)e * a.d_bytes + (int64_t)blockIdx.x * s.KB * T::P::CHUNK;
    v4f acc[1][1] = {{{0.f, 0.f, 0.f, 0.f}}};
    T::multiply(lds + wave * T::WAVE_LDS, s, parts == 1 ? 0 : wave / na, parts, l, acc);
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] = mine ? fmaf(w, acc[0][0][i], sum[i]) : sum[i];
  }
  __syncthreads();
  give_tile<1>(lds, wave, 0, l, sum);
  __syncthreads();
  const int d = blockIdx.x * 16 + 4 * g;
  if (wave == 0 && lr < (int)a.T && d < a.D) {
    const v4f r = join_waves<1>(lds, 0, l) * W4_UNIT;
    if (out_bf16)
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.y) + lr * a.ldy + d) =
          make_uint2(f32x2_to_bf16x2(r[0], r[1]), f32x2_to_bf16x2(r[2], r[3]));
    else
      *reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.y) + lr * a.ldy + d) = r;
  }
#endif  // SG_DEVICE_PASS
}

// Few pairs, many row blocks: a workgroup keeps R pairs' rows of one expert in LDS
// and its waves stream row blocks of that expert's weights past them (W4Stream).
// Dynamic LDS: 8 lists of 16 pairs, then the rows.
template <int GC, bool DOWN>
__global__ void __launch_bounds__(512) k_moe_stream(MoeArgs a, int R) {
#if SG_DEVICE_PASS
  using S = W4Stream<GC>;
  extern __shared__ __attribute__((aligned(1024))) uint8_t moe_lds[];
  const int t = threadIdx.x, l = t & 63, g = l >> 4, lr = l & 15;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6), P = (int)a.P;
  const int v = l < P ? a.ids[l] : -1;
  const int e = row_expert(a, v, blockIdx.y);
  if (e < 0) return;
  int* const list = reinterpret_cast<int*>(moe_lds) + 16 * wave;
  uint8_t* const xs = moe_lds + 512;
  const int K = DOWN ? a.F : a.D, N = DOWN ? a.D : a.F, KB = (K + 127) >> 7, blocks = N / 16;
  const int rb0 = blockIdx.x * W4_WAVES + wave, step = gridDim.x * W4_WAVES;
  const int mine = rb0 < blocks ? (blocks - rb0 + step - 1) / step : 0;
  const int64_t bytes = (int64_t)KB * S::P::CHUNK;
  const uint8_t* const w0 = (DOWN ? a.down + e * a.d_bytes : a.gate + e * a.gu_bytes) + rb0 * bytes;
  const uint8_t* const w1 = DOWN ? w0 : a.up + e * a.gu_bytes + rb0 * bytes;
  int first, cnt = 1;
  for (int m0 = 0; m0 < cnt; m0 += R) {
    cnt = find_pairs(a.ids, P, v, e, m0, R, list, l, first);
    if (cnt == 0 || (a.P <= a.E && first != (int)blockIdx.y)) return;   // the same for every wave
    const int n = min(R, cnt - m0);
    const int pair = lr < n ? list[lr] : -1;
    if (DOWN)
      S::load_x(xs, a.h, (uint32_t)(a.P * a.F * 2), K, R, n, wave, l,
                [&](int r) { return (uint32_t)list[r] * (a.F * 2); });
    else
      S::load_x(xs, a.x, (uint32_t)(((a.T - 1) * a.ldx + a.D) * 2), K, R, n, wave, l,
                [&](int r) { return (uint32_t)((int64_t)(list[r] / a.k) * a.ldx * 2); });
    w4_wait<0>();
    __syncthreads();
    if (DOWN) {
      S::run(xs, KB, R, mine, l, [&](int u) { return w0 + (int64_t)u * step * bytes; },
             [&](int u, const v4f& acc) {
               if (pair >= 0)
                 *reinterpret_cast<v4f*>(a.o + (int64_t)pair * a.D + (rb0 + u * step) * 16 + 4 * g) = acc * W4_UNIT;
             });
    } else {
      v4f gate;
      S::run(xs, KB, R, 2 * mine, l, [&](int u) { return ((u & 1) ? w1 : w0) + (int64_t)(u >> 1) * step * bytes; },
             [&](int u, const v4f& acc) {
               if ((u & 1) == 0) {
                 gate = acc;
               } else if (pair >= 0) {
                 float h[4];
#pragma unroll
                 for (int i = 0; i < 4; ++i) h[i] = silu(gate[i] * W4_UNIT) * (acc[i] * W4_UNIT);
                 *reinterpret_cast<uint2*>(a.h + (int64_t)pair * a.F + (rb0 + (u >> 1) * step) * 16 + 4 * g) =
                     make_uint2(f32x2_to_bf16x2(h[0], h[1]), f32x2_to_bf16x2(h[2], h[3]));
               }
             });
    }
    __syncthreads();
  }
#endif  // SG_DEVICE_PASS
}

#if SG_DEVICE_PASS
// The tile's product over its first `rows` pairs, in steps of 32.
template <int GC, int IW>
__device__ __forceinline__ void multiply_rows(uint8_t* lds, const typename W4Tile<GC, IW>::Src& s, int rows, int wave,
                                              int l, v4f (&acc)[IW][8]) {
  using T = W4Tile<GC, IW>;
  if (rows > 96) T::template multiply<4>(lds, s, wave, l, acc);
  else if (rows > 64) T::template multiply<3>(lds, s, wave, l, acc);
  else if (rows > 32) T::template multiply<2>(lds, s, wave, l, acc);
  else T::template multiply<1>(lds, s, wave, l, acc);
}
#endif  // SG_DEVICE_PASS

// Many pairs per expert: tiles of MOE_BM pairs of one expert.  Gate and up, 64 IW
// rows of each.  IW = 2: a wave's first slot is gate's row block, its second the
// same of up's; IW = 1: waves 0 .. 3 have gate's row blocks, 4 .. 7 up's, and
// hand their sums over in LDS.
template <int GC, int IW>
__global__ void __launch_bounds__(512) k_moe_gate_up(MoeArgs a, int tiles_n) {
#if SG_DEVICE_PASS
  using T = W4Tile<GC, IW>;
  static_assert(T::BM == MOE_BM, "tile");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::LDS];
  const int tile = blockIdx.x / tiles_n, tn = blockIdx.x % tiles_n;
  if (tile >= a.tile[0]) return;
  const int e = a.tile[1 + 2 * tile], m0 = a.tile[2 + 2 * tile], rows = min(T::BM, a.off[e + 1] - m0);
  const int l = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  typename T::Src s;
  s.K = a.D;
  s.KB = (a.D + 127) >> 7;
  const int fb = tn * 4 * IW + (IW == 2 ? wave : wave & 3);
  // past F the last row block again: nothing of it is stored
  const int64_t at = (int64_t)e * a.gu_bytes + (int64_t)min(fb, (a.F - 1) >> 4) * s.KB * T::P::CHUNK;
#pragma unroll
  for (int i = 0; i < IW; ++i) s.w[i] = ((IW == 2 ? i : wave >> 2) ? a.up : a.gate) + at;
  s.x = a.x;
  s.x_bytes = (uint32_t)(((a.T - 1) * a.ldx + a.D) * 2);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = T::x_row(u, wave, l);
    s.xoff[u] = r < rows ? (uint32_t)((int64_t)(a.list[m0 + r] / a.k) * a.ldx * 2) : W4_OUT;
  }
  v4f acc[IW][8];
  multiply_rows<GC, IW>(lds, s, rows, wave, l, acc);
  if (IW == 1) {
    lds_barrier();   // every wave is done with the stages
    if (wave >= 4) {
#pragma unroll
      for (int j = 0; j < 8; ++j) *reinterpret_cast<v4f*>(lds + ((wave - 4) * 8 + j) * 1024 + 16 * l) = acc[0][j];
    }
    __syncthreads();
    if (wave >= 4) return;
  }
  const int f = fb * 16 + 4 * (l >> 4), lr = l & 15;
  if (f >= a.F) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (16 * j + lr >= rows) continue;
    const v4f up = IW == 2 ? acc[IW - 1][j] : *reinterpret_cast<const v4f*>(lds + (wave * 8 + j) * 1024 + 16 * l);
    float h[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) h[q] = silu(acc[0][j][q] * W4_UNIT) * (up[q] * W4_UNIT);
    *reinterpret_cast<uint2*>(a.h + (int64_t)(m0 + 16 * j + lr) * a.F + f) =
        make_uint2(f32x2_to_bf16x2(h[0], h[1]), f32x2_to_bf16x2(h[2], h[3]));
  }
#endif  // SG_DEVICE_PASS
}

template <int GC, int IW>
__global__ void __launch_bounds__(512) k_moe_down(MoeArgs a, int tiles_n) {
#if SG_DEVICE_PASS
  using T = W4Tile<GC, IW>;
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
  const int rb0 = (tn * 8 + wave) * IW;
#pragma unroll
  for (int i = 0; i < IW; ++i)
    s.w[i] = a.down + (int64_t)e * a.d_bytes + (int64_t)min(rb0 + i, (a.D - 1) >> 4) * s.KB * T::P::CHUNK;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = T::x_row(u, wave, l);
    s.xoff[u] = r < rows ? (uint32_t)(r * a.F * 2) : W4_OUT;
  }
  v4f acc[IW][8];
  multiply_rows<GC, IW>(lds, s, rows, wave, l, acc);
  const int g = l >> 4, lr = l & 15;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (16 * j + lr >= rows) continue;
    float* const row = a.o + (int64_t)a.list[m0 + 16 * j + lr] * a.D;
#pragma unroll
    for (int i = 0; i < IW; ++i) {
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
  int64_t off, list, tile, h, o, bytes;
  MoeSpace(int64_t P, int64_t E, int64_t D, int64_t F) {
    int64_t at = 0;
    const auto part = [&](int64_t n) { const int64_t was = at; at += cdiv(n, 256) * 256; return was; };
    off = part(4 * (E + 1));
    list = part(4 * P);
    tile = part(4 * (2 * moe_tiles(P, E) + 1));
    h = part(2 * P * F);
    o = part(4 * P * D);
    bytes = at;
  }
};

template <int GC, int XI>
static void launch_moe_few(const MoeArgs& a, bool bf16, hipStream_t st) {
  const unsigned gy = (unsigned)(a.P < a.E ? a.P : a.E);
  k_moe_gate_up_rows<GC, XI><<<dim3((unsigned)cdiv(a.F, 16), gy), 512, 0, st>>>(a);
  k_moe_down_join<GC, XI><<<(unsigned)cdiv(a.D, 16), 512, 0, st>>>(a, bf16);
}

// One product by streaming: the most X rows of 16, 8, 4 that leave LDS to two
// workgroups of a compute unit; workgroups as many as stay busy.
static int moe_stream_rows(int64_t K) {
  const int64_t row = cdiv(K, 128) * 256;
  return 16 * row <= 79 * 1024 ? 16 : 8 * row <= 79 * 1024 ? 8 : 4 * row <= 79 * 1024 ? 4 : 0;
}
template <int GC, bool DOWN>
static void launch_moe_stream(const MoeArgs& a, hipStream_t st) {
  const int64_t K = DOWN ? a.F : a.D, blocks = (DOWN ? a.D : a.F) / 16, gy = a.P < a.E ? a.P : a.E;
  const int R = moe_stream_rows(K);
  int64_t gx = cdiv(blocks, W4_WAVES);
  if (gx * gy > 1024) gx = cdiv(1024, gy) < gx ? cdiv(1024, gy) : gx;
  k_moe_stream<GC, DOWN><<<dim3((unsigned)gx, (unsigned)gy), 512, 512 + R * cdiv(K, 128) * 256, st>>>(a, R);
}

// Which way: us of 64 experts (4096, 1024), k 8 / 60 experts (2048, 1408), k 4 / 9
// experts (2016, 1216), k 2, the same four routings in turn for each way.
//   pairs       few            stream            tiles
//   16      34 / 38 / 24     49 /  34 / 35     48 / 38 / 32
//   32                       58 /  53 / 37     72 / 54 / 32
//   64                       80 /  61 / 53     83 / 67 / 32
//   128                     104 /  68 / 77    101 / 70 / 36
//   256                     131 /  94         109 / 77
//   512                     216 / 135         123 / 92
// Streaming passes over an expert's weights once for every R of its pairs (R is 8, 16
// and 16 here), so it is taken while an expert has R / 4 on average (some have several
// times that).  With as few experts as 9 its workgroups are too few: the tiles are
// faster by a seventh from 17 to 36 pairs, where the rule still streams.
template <int GC>
static void launch_moe(const MoeArgs& a, bool bf16, hipStream_t st) {
  if (a.P <= MOE_FEW) {
    if (a.T <= 4) launch_moe_few<GC, 1>(a, bf16, st);
    else if (a.T <= 8) launch_moe_few<GC, 2>(a, bf16, st);
    else launch_moe_few<GC, 4>(a, bf16, st);
    return;
  }
  const int rd = moe_stream_rows(a.D), rf = moe_stream_rows(a.F), R = rd < rf ? rd : rf;
  if (4 * a.P <= (int64_t)R * a.E && a.P <= 2048) {   // every workgroup reads all ids
    launch_moe_stream<GC, false>(a, st);
    launch_moe_stream<GC, true>(a, st);
  } else {
    k_moe_plan<<<1, 1024, 0, st>>>(a);
    // tiles there may be, and about as many as there are: half an expert's last one is empty
    const int64_t tm = moe_tiles(a.P, a.E), about = cdiv(a.P, MOE_BM) + (a.P < a.E ? a.P : a.E) / 2;
    const int64_t ng = cdiv(a.F, 128), nd = cdiv(a.D, 256);
    if (about * ng <= 256) k_moe_gate_up<GC, 1><<<(unsigned)(tm * cdiv(a.F, 64)), 512, 0, st>>>(a, (int)cdiv(a.F, 64));
    else k_moe_gate_up<GC, 2><<<(unsigned)(tm * ng), 512, 0, st>>>(a, (int)ng);
    if (about * nd <= 256) k_moe_down<GC, 1><<<(unsigned)(tm * cdiv(a.D, 128)), 512, 0, st>>>(a, (int)cdiv(a.D, 128));
    else k_moe_down<GC, 2><<<(unsigned)(tm * nd), 512, 0, st>>>(a, (int)nd);
  }
  const unsigned grid = grid_for(a.T * (a.D / 4), 256, 8192);
  if (bf16) k_moe_combine<true><<<grid, 256, 0, st>>>(a);
  else k_moe_combine<false><<<grid, 256, 0, st>>>(a);
}

// The limits shared by the call and its workspace size.
static bool moe_shape_ok(int64_t T, int k, int64_t E, int64_t D, int64_t F) {
  if (T < 1 || k < 1 || E < 1 || E > MOE_EMAX || D < 32 || F < 32 || D % 32 || F % 32) return false;
  if (D >= (1LL << 22) || F >= (1LL << 22) || T > (1LL << 30) / k) return false;
  // the tiles' launches (the half tiles are of a few hundred workgroups)
  const int64_t nf = cdiv(F, 128), nd = cdiv(D, 256);
  return launch_fits(moe_tiles(T * k, E) * (nf > nd ? nf : nd), 512);
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
  a.tile = reinterpret_cast<int*>(w + ws.tile);
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
