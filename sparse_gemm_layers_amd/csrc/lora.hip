// Low-rank adapters of many requests, with e = ids[t]:
//   y[t] = base[t] + s_e (x[t] . A_e^T) . B_e^T
// and the backward pass
//   u = x . A_e^T, v = s_e dy . B_e, dx = base + v . A_e,
//   dA_e = sum_t v[t]^T x[t], dB_e = s_e sum_t dy[t]^T u[t].
// Three kinds of kernel, all bound by memory: "down" products [T, C] -> [T, r], the
// long side summed in up to LORA_PARTS parts over workgroups; "up" products [T, r] ->
// [T, C], which add up those parts as they read them; and the sums over an adapter's
// tokens [T, r]^T [T, C].
//
// The [T, r] values between two products stay fp32 in memory and enter the matrix
// core as a sum of NP bf16 parts (each the rounding of what the ones before leave):
// with so few ranks that costs matrix instructions only, which nothing waits for.
//
// Down and up go by blocks of 64 tokens, one to a lane.  The tokens of one adapter in
// a block are gathered, 16 TM at a time, into the columns of a matrix product (an
// "item"): a prompt's block is few items, a decoding batch's many, which the third
// dimension of the grid shares out, and either way an adapter is read once for
// all of them.  The sums over tokens gather the rows of one adapter likewise.
#include "bf16_tile.h"
#include "sg_lora.h"

namespace sg {

#if SG_DEVICE_PASS
// The adapter of token t, -1: none.
__device__ __forceinline__ int lora_id(const int32_t* ids, int64_t t, int64_t T, int L) {
  if (t >= T) return -1;
  const int e = ids ? ids[t] : 0;
  return e >= 0 && e < L ? e : -1;
}

// The items of a block of 64 tokens that are this workgroup's, the first-th and every
// step-th after it: adapter by adapter, of each 16 TM tokens at a time in their order.  Lane l
// holds the adapter of token t0 + l.  Every wave goes through all of the block's adapters, so
// that must be cheap: blocks of 256 tokens, whose items are fuller, made it four times as long
// (700 tokens of 100 adapters of rank 32, 4096 x 4096: 117 us for 60; 150 of 10, rank 16: 14.3 for
// 11.8; but 1000 of 16, rank 32, 4096 x 11008: 36 for 54).
template <int TM>
struct LoraItems {
  int id, e, all, at, step;   // the adapter, its tokens; the item, from its first on
  uint64_t left, m;           // tokens of this and the adapters to come, of this one
  int* list;                  // in LDS, this wave's own
  __device__ __forceinline__ void start(const int32_t* ids, int64_t t0, int64_t T, int L, int l, bool none, int first,
                                        int steps, int* lds) {
    id = lora_id(ids, t0 + l, T, L);
    left = __ballot(t0 + l < T && (none || id >= 0));
    m = 0;
    e = -1;
    all = 0;
    at = first;
    step = steps;
    list = lds;
  }
  // The next item: its adapter (-1: tokens without one) and number of tokens, whose places
  // in the block list then holds.
  __device__ __forceinline__ bool next(int l, int& adapter, int& n) {
    while (at * (16 * TM) >= all) {
      at -= (all + 16 * TM - 1) / (16 * TM);
      left &= ~m;
      if (!left) return false;
      e = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
      m = __ballot(id == e) & left;
      all = __builtin_popcountll(m);
    }
    const int before = at * (16 * TM), rank = __builtin_popcountll(m & ((1ull << l) - 1)) - before;
    n = min(all - before, 16 * TM);
    if (((m >> l) & 1) && rank >= 0 && rank < 16 * TM) list[rank] = l;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    adapter = e;
    at += step;
    return true;
  }
};

// NP bf16 parts of V fp32 values.  What an infinite part or a NaN leaves is nothing,
// not the NaN that subtracting it gives.
template <int NP, int V>
__device__ __forceinline__ void lora_parts(float (&v)[V], uint32_t (&p)[NP][V / 2]) {
#pragma unroll
  for (int n = 0; n < NP; ++n)
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const uint32_t w = f32x2_to_bf16x2(v[2 * i], v[2 * i + 1]);
      p[n][i] = w;
      if (n + 1 == NP) continue;
      v[2 * i] = (w & 0x7f80u) == 0x7f80u ? 0.0f : v[2 * i] - __uint_as_float(w << 16);
      v[2 * i + 1] = (w & 0x7f800000u) == 0x7f800000u ? 0.0f : v[2 * i + 1] - __uint_as_float(w & 0xffff0000u);
    }
}
// What the parts after the first are multiplied by: eight bf16 values, zero for an infinity or a NaN.
// The first part alone meets those, as the whole value would: the next ones may be zero or
// of the other sign, and their product with an infinity would make the sum a NaN.  (Costs, kernels:
// 2048 x 4096 x 4096, rank 16 18.1 us for 17.7; gradients of 4096 tokens, rank 16 51.4 for 49.8.)
__device__ __forceinline__ v4i lora_finite(const v4i& w) {
  typedef short v2s __attribute__((ext_vector_type(2)));
  v4i f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t top = ((uint32_t)w[i] & 0x7f807f80u) + 0x00800080u;   // a half's sign bit: its exponent is all ones
    f[i] = w[i] & ~__builtin_bit_cast(int, __builtin_bit_cast(v2s, top) >> 15);
  }
  return f;
}
__device__ __forceinline__ uint4 lora_pack(const uint32_t (&p)[4]) { return make_uint4(p[0], p[1], p[2], p[3]); }
#endif

constexpr int LORA_PARTS = 2;    // of a down product's sum, at most
constexpr int LORA_WAVES = 8;    // of a down workgroup

// ------------------------------------------------------------------ down

struct LoraDown {
  int64_t T;
  int C, r, L, splits;     // the sum runs over C, in `splits` parts
  const uint16_t *z, *w;   // z [T, C]; w [L][r][C], or KS: [L][C][r]
  int64_t ldz;
  const int32_t* ids;
  float* part;             // [splits][T][r]
};

// A workgroup's waves take every LORA_WAVES-th 64 columns of its part; the next ones are asked
// for while these are multiplied.  Rows come whole, 8 lanes to 128 bytes of one, and go
// through the wave's own LDS: as the matrix core wants them, neighbouring lanes in
// different rows, a load keeps the compute unit's address path busy four times as long
// (2048 x 4096, rank 16: 10.4 us).
template <bool KS, int TM, int RM>
struct LoraDownLds {
  static constexpr int PITCH = 32 * RM + 16;   // KS: one row's ranks
  static constexpr int WAVE = 2048 * TM + (KS ? 64 * PITCH : 2048 * RM), RED = LORA_WAVES * RM * TM * 1024;
  static constexpr int BYTES = RED > LORA_WAVES * WAVE ? RED : LORA_WAVES * WAVE;
};
#if SG_DEVICE_PASS
template <bool KS, int TM, int RM>
__device__ __forceinline__ void lora_down(const LoraDown& a, uint8_t* lds, int (*lists)[64], int by) {
  constexpr int PITCH = LoraDownLds<KS, TM, RM>::PITCH, WAVE = LoraDownLds<KS, TM, RM>::WAVE;
  const int t = threadIdx.x, l = t & 63, g = l >> 4, lr = l & 15;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int64_t t0 = (int64_t)blockIdx.x * 64;
  const int split = by % a.splits, rho0 = by / a.splits * 16 * RM;
  const int rows = (int)min((int64_t)64, a.T - t0);
  const int units = (a.C + 63) >> 6;   // of 64 columns
  const int u0 = (int)((int64_t)units * split / a.splits), u1 = (int)((int64_t)units * (split + 1) / a.splits);
  LoraItems<TM> items;
  items.start(a.ids, t0, a.T, a.L, l, false, blockIdx.z, gridDim.z, lists[wave]);
  const __amdgpu_buffer_rsrc_t rz = w4_rsrc(a.z + t0 * a.ldz, (uint32_t)(((rows - 1) * a.ldz + a.C) * 2));
  uint8_t *const zl = lds + wave * WAVE, *const wl = zl + 2048 * TM;
  const int put = (l >> 3) * 128 + (((l & 7) ^ swz8q(l >> 3)) << 4);   // of 8 rows of 128 bytes
  int e, n;
  while (items.next(l, e, n)) {
    const uint16_t* const w = a.w + (int64_t)e * a.r * a.C;
    // KC: rows of ranks past r are outside; KS: its rows hold all ranks
    const __amdgpu_buffer_rsrc_t rw =
        KS ? w4_rsrc(w, (uint32_t)(a.C * a.r * 2))
           : w4_rsrc(w + (int64_t)rho0 * a.C, (uint32_t)(min(a.r - rho0, 16 * RM) * a.C * 2));
    uint32_t zo[2 * TM];
#pragma unroll
    for (int i = 0; i < 2 * TM; ++i) {
      const int c = 8 * i + (l >> 3);
      zo[i] = c < n ? (uint32_t)(items.list[c] * a.ldz * 2) + 16 * (l & 7) : W4_OUT;
    }
    v4f acc[RM][TM];
#pragma unroll
    for (int m = 0; m < RM; ++m)
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[m][j] = (v4f){0.f, 0.f, 0.f, 0.f};
    v4i zv[2][2 * TM], wv[2][2 * RM];
    const auto load = [&](int s, int u) {
      const bool in = 64 * u + 8 * (l & 7) < a.C;
#pragma unroll
      for (int i = 0; i < 2 * RM; ++i) {
        if (KS) {   // 16 bytes c of row k; the 64 rows of 16 RM ranks are 2 RM loads
          const int k = (i * 64 + l) / (2 * RM), c = (i * 64 + l) % (2 * RM);
          wv[s][i] = w4_ld16(rw, rho0 + 8 * c < a.r ? ((uint32_t)(64 * u + k) * a.r + rho0 + 8 * c) * 2 : W4_OUT, 0);
        } else {
          wv[s][i] = w4_ld16(rw, in ? (uint32_t)((8 * i + (l >> 3)) * a.C * 2 + 16 * (l & 7)) : W4_OUT, u * 128);
        }
      }
#pragma unroll
      for (int i = 0; i < 2 * TM; ++i) zv[s][i] = w4_ld16(rz, in ? zo[i] : W4_OUT, u * 128);
    };
    const auto compute = [&](int s) {
#pragma unroll
      for (int i = 0; i < 2 * RM; ++i) {
        if (KS) *reinterpret_cast<v4i*>(wl + (i * 64 + l) / (2 * RM) * PITCH + 16 * ((i * 64 + l) % (2 * RM))) = wv[s][i];
        else *reinterpret_cast<v4i*>(wl + 1024 * i + put) = wv[s][i];
      }
#pragma unroll
      for (int i = 0; i < 2 * TM; ++i) *reinterpret_cast<v4i*>(zl + 1024 * i + put) = zv[s][i];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int at = lr * 128 + (((4 * q + g) ^ swz8q(lr)) << 4);
        v4i zf[TM];
#pragma unroll
        for (int j = 0; j < TM; ++j) zf[j] = *reinterpret_cast<const v4i*>(zl + 2048 * j + at);
#pragma unroll
        for (int m = 0; m < RM; ++m) {
          v4i wf;
          if (KS) {
            const uint8_t* const from = wl + (32 * q + 8 * g + (lr >> 2)) * PITCH + 32 * m + 8 * (lr & 3);
            const uint2 x = lds_tr4(from), y = lds_tr4(from + 4 * PITCH);
            wf = (v4i){(int)x.x, (int)x.y, (int)y.x, (int)y.y};
          } else {
            wf = *reinterpret_cast<const v4i*>(wl + 2048 * m + at);
          }
#pragma unroll
          for (int j = 0; j < TM; ++j) acc[m][j] = w4_mfma(wf, zf[j], acc[m][j]);
        }
      }
    };
    int u = u0 + wave;
    if (u < u1) load(0, u);
    for (; u < u1; u += 2 * LORA_WAVES) {
      const bool more = u + LORA_WAVES < u1;
      if (more) load(1, u + LORA_WAVES);
      compute(0);
      if (more) {
        if (u + 2 * LORA_WAVES < u1) load(0, u + 2 * LORA_WAVES);
        compute(1);
      }
    }
    float(*const red)[RM * TM][64][4] = reinterpret_cast<float(*)[RM * TM][64][4]>(lds);
    __syncthreads();
#pragma unroll
    for (int m = 0; m < RM; ++m)
#pragma unroll
      for (int j = 0; j < TM; ++j) *reinterpret_cast<v4f*>(&red[wave][m * TM + j][l][0]) = acc[m][j];
    __syncthreads();
    for (int q = wave; q < RM * TM; q += LORA_WAVES) {
      const int m = q / TM, c = 16 * (q % TM) + lr, rho = rho0 + 16 * m + 4 * g;
      v4f s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < LORA_WAVES; ++k) s += *reinterpret_cast<const v4f*>(&red[k][q][l][0]);
      if (c < n && rho < a.r)
        *reinterpret_cast<float4*>(a.part + ((int64_t)split * a.T + t0 + items.list[c]) * a.r + rho) =
            make_float4(s[0], s[1], s[2], s[3]);
    }
    __syncthreads();
  }
}
#endif  // SG_DEVICE_PASS

template <bool KS, int TM, int RM>
__global__ void __launch_bounds__(512) k_lora_down(LoraDown a) {
#if SG_DEVICE_PASS
  __shared__ __attribute__((aligned(16))) uint8_t lds[LoraDownLds<KS, TM, RM>::BYTES];
  __shared__ int lists[LORA_WAVES][64];
  lora_down<KS, TM, RM>(a, lds, lists, blockIdx.y);
#endif
}

// Both of the backward pass: v's workgroups come first along y, then u's.
template <int TM, int RM>
__global__ void __launch_bounds__(512) k_lora_down_two(LoraDown v, LoraDown u, int v_y) {
#if SG_DEVICE_PASS
  __shared__ __attribute__((aligned(16))) uint8_t lds[LoraDownLds<true, TM, RM>::BYTES];   // the larger
  __shared__ int lists[LORA_WAVES][64];
  if ((int)blockIdx.y < v_y) lora_down<true, TM, RM>(v, lds, lists, blockIdx.y);
  else lora_down<false, TM, RM>(u, lds, lists, blockIdx.y - v_y);
#endif
}

// ------------------------------------------------------------------ up

struct LoraUp {
  int64_t T;
  int C, r, L, splits;     // parts of p
  const float* part;       // [splits][T][r]
  const float* scale;
  const int32_t* ids;
  const uint16_t* w;       // [L][C][r], or KS: [L][r][C]
  const void* base;
  int64_t ld_base;
  int base_f32;
  void* y;
  int64_t ldy;
  int y_f32;
};

#if SG_DEVICE_PASS
// Ranks rho .. rho + 7 of token t's [T, r] value: its parts, all asked for at once;
// lora_total adds them in order and scales.
struct LoraValue {
  float4 x[LORA_PARTS][2];
  __device__ __forceinline__ void load(const float* part, int splits, int64_t T, int r, int64_t t, int rho, bool there) {
#pragma unroll
    for (int s = 0; s < LORA_PARTS; ++s) {
      x[s][0] = x[s][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s < splits && there) {
        const float4* const p = reinterpret_cast<const float4*>(part + ((int64_t)s * T + t) * r + rho);
        x[s][0] = p[0];
        x[s][1] = p[1];
      }
    }
  }
  __device__ __forceinline__ void total(float scale, float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const auto at = [&](int s) {
        const float4 q = x[s][i >> 2];
        return (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
      };
      float t = at(0);
#pragma unroll
      for (int s = 1; s < LORA_PARTS; ++s) t += at(s);
      v[i] = t * scale;
    }
  }
};

// Columns n .. n + 7 of row t: v plus base, of which bf16 ones have been read.
__device__ __forceinline__ void lora_store(const LoraUp& a, int64_t t, int n, const uint4& base, float (&v)[8]) {
  if (a.base_f32) {
    float x[8];
    const float* const p = reinterpret_cast<const float*>(a.base) + t * a.ld_base + n;
    load4(p, x);
    load4(p + 4, x + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += x[i];
  } else if (a.base) {
    const uint32_t w[4] = {base.x, base.y, base.z, base.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += __uint_as_float((i & 1) ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
  if (a.y_f32) {
    float* const o = reinterpret_cast<float*>(a.y) + t * a.ldy + n;
    *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.y) + t * a.ldy + n) =
        make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]), f32x2_to_bf16x2(v[4], v[5]),
                   f32x2_to_bf16x2(v[6], v[7]));
  }
}
#endif

// A workgroup's four waves take 64 columns each.
template <bool KS>
struct LoraUpLds {
  static constexpr int PITCH = 128 + 16;   // KS: 64 columns of one rank
  uint8_t w[KS ? 4 * 32 * PITCH : 16];
  int lists[4][64];
};
#if SG_DEVICE_PASS
// bx, by, bz: the workgroup's block of tokens, its columns, its share gz-th of the items
template <bool KS, int NP>
__device__ __forceinline__ void lora_up(const LoraUp& a, LoraUpLds<KS>& shared, int bx, int by, int bz, int gz) {
  constexpr int TM = 1, PITCH = LoraUpLds<KS>::PITCH;
  uint8_t* const lds = shared.w;
  const int t = threadIdx.x, l = t & 63, g = l >> 4, lr = l & 15;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int64_t t0 = (int64_t)bx * 64;
  const int n0 = (by * 4 + wave) * 64;
  if (n0 >= a.C) return;   // no barrier follows
  LoraItems<TM> items;
  items.start(a.ids, t0, a.T, a.L, l, a.y != a.base, bz, gz, shared.lists[wave]);
  int e, count;
  while (items.next(l, e, count)) {
    int tok[TM];   // of column 16 j + lr, -1: none
    uint4 base[TM][2];
#pragma unroll
    for (int j = 0; j < TM; ++j) tok[j] = 16 * j + lr < count ? items.list[16 * j + lr] : -1;
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int n = n0 + 32 * q + 8 * g;
        base[j][q] = make_uint4(0, 0, 0, 0);
        if (a.base && !a.base_f32 && tok[j] >= 0 && n < a.C)
          base[j][q] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.base) +
                                                       (t0 + tok[j]) * a.ld_base + n);
      }
    v4f acc[4][TM];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
    const float scale = a.scale && e >= 0 ? a.scale[e] : 1.0f;
    const uint16_t* const w = a.w + (int64_t)e * a.r * a.C;
    for (int rho0 = 0; e >= 0 && rho0 < a.r; rho0 += 32) {
      const int rho = rho0 + 8 * g;
      v4i wf[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        wf[i] = (v4i){0, 0, 0, 0};
        if (!KS) {
          const int n = n0 + tile_n(i, lr);
          if (n < a.C && rho < a.r) wf[i] = *reinterpret_cast<const v4i*>(w + (int64_t)n * a.r + rho);
        } else {
          const int k = rho0 + 8 * i + (l >> 3), c = n0 + 8 * (l & 7);
          if (k < a.r && c < a.C) wf[i] = *reinterpret_cast<const v4i*>(w + (int64_t)k * a.C + c);
        }
      }
      LoraValue value[TM];
#pragma unroll
      for (int j = 0; j < TM; ++j)
        value[j].load(a.part, a.splits, a.T, a.r, t0 + tok[j], rho, tok[j] >= 0 && rho < a.r);
      if (KS) {
        uint8_t* const st = lds + wave * 32 * PITCH;
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<v4i*>(st + (8 * i + (l >> 3)) * PITCH + 16 * (l & 7)) = wf[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint8_t* const at = st + (8 * g + (lr >> 2)) * PITCH + 64 * (i >> 1) + 16 * (lr & 3) + 8 * (i & 1);
          const uint2 x = lds_tr4(at), y = lds_tr4(at + 4 * PITCH);
          wf[i] = (v4i){(int)x.x, (int)x.y, (int)y.x, (int)y.y};
        }
      }
      v4i finite[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) finite[i] = lora_finite(wf[i]);
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        float v[8];
        value[j].total(scale, v);
        uint32_t p[NP][4];
        lora_parts<NP>(v, p);
#pragma unroll
        for (int n = NP - 1; n >= 0; --n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[i][j] = w4_mfma(n ? finite[i] : wf[i], __builtin_bit_cast(v4i, lora_pack(p[n])), acc[i][j]);
      }
    }
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int n = n0 + 32 * q + 8 * g;
        if (tok[j] >= 0 && n < a.C) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = acc[2 * q + (i >> 2)][j][i & 3];
          lora_store(a, t0 + tok[j], n, base[j][q], v);
        }
      }
  }
}
#endif  // SG_DEVICE_PASS

template <bool KS, int NP>
__global__ void __launch_bounds__(256) k_lora_up(LoraUp a) {
#if SG_DEVICE_PASS
  __shared__ __attribute__((aligned(16))) LoraUpLds<KS> lds;
  lora_up<KS, NP>(a, lds, blockIdx.x, blockIdx.y, blockIdx.z, gridDim.z);
#endif
}

// ------------------------------------------------------------------ both at once

// Down and up in one launch, for few tokens with short adapters (lora_both), where a second
// launch costs more than that every workgroup goes through the whole of an adapter's
// down part: it takes an item of 16 tokens at a time and a slice of the columns.  Its
// waves split the long sum and add it in LDS, where it stays as the other product's
// operand; then they take 64 columns each.  (One token, 4096 x 4096, rank 16: 7.4 us, two
// launches 8.6 and a gap; but 2048 tokens 28 us for 20, and 37 of 16 adapters of rank 64
// beside 14336 columns 35 us for 19.)
struct LoraBoth {
  LoraDown d;
  LoraUp u;
  int slice;       // columns of one workgroup, a multiple of 64
};

template <int RM, int NP>
__global__ void __launch_bounds__(512) k_lora_both(LoraBoth b) {
#if SG_DEVICE_PASS
  constexpr int RC = 16 * RM, WL = 2 * RM, DEPTH = RM == 1 ? 4 : RM == 2 ? 2 : 1;
  constexpr int PP = 2 * RC + 16, OP = 256 + 16;           // pitches of ranks, of one token's results
  constexpr int D_BYTES = 2048 + 2048 * RM, U_BYTES = 64 * PP;
  constexpr int WAVE0 = D_BYTES > U_BYTES ? D_BYTES : U_BYTES, WAVE = WAVE0 > 16 * OP ? WAVE0 : 16 * OP;
  constexpr int RED = LORA_WAVES * RM * 1024;
  __shared__ __attribute__((aligned(16))) uint8_t lds[RED > LORA_WAVES * WAVE ? RED : LORA_WAVES * WAVE], pl[NP * 16 * PP];
  __shared__ int lists[LORA_WAVES][64];
  const LoraDown& a = b.d;
  const LoraUp& y = b.u;
  const int t = threadIdx.x, l = t & 63, g = l >> 4, lr = l & 15;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int64_t t0 = (int64_t)blockIdx.x * 64;
  const int rows = (int)min((int64_t)64, a.T - t0);
  const int units = (a.C + 63) >> 6;
  const int s0 = blockIdx.y * b.slice, s1 = min(s0 + b.slice, y.C);
  LoraItems<1> items;
  items.start(a.ids, t0, a.T, a.L, l, y.y != y.base, blockIdx.z, gridDim.z, lists[wave]);
  const __amdgpu_buffer_rsrc_t rz = w4_rsrc(a.z + t0 * a.ldz, (uint32_t)(((rows - 1) * a.ldz + a.C) * 2));
  uint8_t *const zl = lds + wave * WAVE, *const wl = zl + 2048;
  const int put = (l >> 3) * 128 + (((l & 7) ^ swz8q(l >> 3)) << 4);   // of 8 rows of 128 bytes
  int e, n;
  while (items.next(l, e, n)) {
    const int place0 = items.list[l >> 3], place1 = items.list[8 + (l >> 3)];   // of the lane's pieces of rows
    // what the second product reads of memory: adapter rows and base of 64 columns
    const __amdgpu_buffer_rsrc_t r2 = w4_rsrc(y.w + (int64_t)e * a.r * y.C, e >= 0 ? (uint32_t)(a.r * y.C * 2) : 0u);
    v4i uv[WL];
    uint4 base[2];
    const auto load_up = [&](int n0) {
      const int col = n0 + 8 * (l & 7);
#pragma unroll
      for (int i = 0; i < WL; ++i) {
        const int c = n0 + (64 * i + l) / WL, k = 8 * ((64 * i + l) % WL);
        uv[i] = w4_ld16(r2, c < s1 && k < a.r ? (uint32_t)((c * a.r + k) * 2) : W4_OUT, 0);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        base[i] = make_uint4(0, 0, 0, 0);
        if (y.base && !y.base_f32 && 8 * i + (l >> 3) < n && col < s1)
          base[i] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(y.base) +
                                                    (t0 + (i ? place1 : place0)) * y.ld_base + col);
      }
    };
    if (e >= 0) {
      const uint16_t* const w = a.w + (int64_t)e * a.r * a.C;
      const __amdgpu_buffer_rsrc_t rw = w4_rsrc(w, (uint32_t)(a.C * a.r * 2));   // rows of ranks past r are outside
      const uint32_t zo0 = (l >> 3) < n ? (uint32_t)(place0 * a.ldz * 2) + 16 * (l & 7) : W4_OUT;
      const uint32_t zo1 = 8 + (l >> 3) < n ? (uint32_t)(place1 * a.ldz * 2) + 16 * (l & 7) : W4_OUT;
      v4f acc[RM];
#pragma unroll
      for (int m = 0; m < RM; ++m) acc[m] = (v4f){0.f, 0.f, 0.f, 0.f};
      v4i zv[DEPTH][2], wv[DEPTH][2 * RM];
      const auto load = [&](int s, int u) {
        const bool in = 64 * u + 8 * (l & 7) < a.C;
#pragma unroll
        for (int i = 0; i < 2 * RM; ++i) {
          wv[s][i] = w4_ld16(rw, in ? (uint32_t)((8 * i + (l >> 3)) * a.C * 2 + 16 * (l & 7)) : W4_OUT, u * 128);
        }
        zv[s][0] = w4_ld16(rz, in ? zo0 : W4_OUT, u * 128);
        zv[s][1] = w4_ld16(rz, in ? zo1 : W4_OUT, u * 128);
      };
      const auto compute = [&](int s) {
#pragma unroll
        for (int i = 0; i < 2 * RM; ++i) {
          *reinterpret_cast<v4i*>(wl + 1024 * i + put) = wv[s][i];
        }
        *reinterpret_cast<v4i*>(zl + put) = zv[s][0];
        *reinterpret_cast<v4i*>(zl + 1024 + put) = zv[s][1];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int at = lr * 128 + (((4 * q + g) ^ swz8q(lr)) << 4);
          const v4i zf = *reinterpret_cast<const v4i*>(zl + at);
#pragma unroll
          for (int m = 0; m < RM; ++m) {
            acc[m] = w4_mfma(*reinterpret_cast<const v4i*>(wl + 2048 * m + at), zf, acc[m]);
          }
        }
      };
#pragma unroll
      for (int s = 0; s < DEPTH; ++s)
        if (wave + s * LORA_WAVES < units) load(s, wave + s * LORA_WAVES);
      for (int u = wave; u < units; u += DEPTH * LORA_WAVES) {
#pragma unroll
        for (int s = 0; s < DEPTH; ++s) {
          if (u + s * LORA_WAVES >= units) break;
          compute(s);
          if (u + (s + DEPTH) * LORA_WAVES < units) load(s, u + (s + DEPTH) * LORA_WAVES);
        }
      }
      if (s0 + 64 * wave < s1) load_up(s0 + 64 * wave);
      float(*const red)[RM][64][4] = reinterpret_cast<float(*)[RM][64][4]>(lds);
      __syncthreads();
#pragma unroll
      for (int m = 0; m < RM; ++m) *reinterpret_cast<v4f*>(&red[wave][m][l][0]) = acc[m];
      __syncthreads();
      if (wave < RM) {
        v4f s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < LORA_WAVES; ++k) s += *reinterpret_cast<const v4f*>(&red[k][wave][l][0]);
        const int rho = 16 * wave + 4 * g;
        const float scale = y.scale ? y.scale[e] : 1.0f;
        float v[4];
        // ranks past r are nothing, also where an infinity of x has met their zeros
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = rho < a.r ? s[k] * scale : 0.0f;
        uint32_t p[NP][2];
        lora_parts<NP>(v, p);
#pragma unroll
        for (int q = 0; q < NP; ++q) *reinterpret_cast<uint2*>(pl + (q * 16 + lr) * PP + 2 * rho) = make_uint2(p[q][0], p[q][1]);
      }
      __syncthreads();
    } else if (s0 + 64 * wave < s1) {
      load_up(s0 + 64 * wave);
    }
    for (int n0 = s0 + 64 * wave; n0 < s1; n0 += 64 * LORA_WAVES) {
      const int col = n0 + 8 * (l & 7);
      v4f acc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = (v4f){0.f, 0.f, 0.f, 0.f};
      const uint4 base0 = base[0], base1 = base[1];
      if (e >= 0) {
#pragma unroll
        for (int i = 0; i < WL; ++i) {
          *reinterpret_cast<v4i*>(zl + (64 * i + l) / WL * PP + 16 * ((64 * i + l) % WL)) = uv[i];
        }
      }
      if (n0 + 64 * LORA_WAVES < s1) load_up(n0 + 64 * LORA_WAVES);
      if (e >= 0) {
#pragma unroll
        for (int k = 0; k < RC; k += 32) {
          const bool in = k + 8 * g < RC;   // a step of 32 ranks, of which 16 may be all
          v4i pf[NP];
#pragma unroll
          for (int q = 0; q < NP; ++q) {
            pf[q] = (v4i){0, 0, 0, 0};
            if (in) pf[q] = *reinterpret_cast<const v4i*>(pl + (q * 16 + lr) * PP + 2 * (k + 8 * g));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v4i wf = {0, 0, 0, 0};
            if (in) wf = *reinterpret_cast<const v4i*>(zl + (16 * i + lr) * PP + 2 * (k + 8 * g));
#pragma unroll
            for (int q = NP - 1; q >= 0; --q) acc[i] = w4_mfma(q ? lora_finite(wf) : wf, pf[q], acc[i]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<v4f*>(zl + lr * OP + 4 * (16 * i + 4 * g)) = acc[i];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint8_t* const from = zl + (8 * i + (l >> 3)) * OP + 32 * (l & 7);
        const v4f x = *reinterpret_cast<const v4f*>(from), z = *reinterpret_cast<const v4f*>(from + 16);
        if (8 * i + (l >> 3) < n && col < s1) {
          float v[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = x[k], v[4 + k] = z[k];
          lora_store(y, t0 + (i ? place1 : place0), col, i ? base1 : base0, v);
        }
      }
    }
    __syncthreads();   // the next item's sum goes where the last results went
  }
#endif  // SG_DEVICE_PASS
}

// ------------------------------------------------------------------ sums over tokens

[[maybe_unused]] constexpr int LORA_LIST = 1024;   // tokens looked through at a time

struct LoraSum {
  int64_t T;
  int C, r, L, splits;     // parts of p
  const uint16_t* z;       // [T, C]
  int64_t ldz;
  const float* part;       // [splits][T][r]
  const float* scale;
  const int32_t* ids;
  int tsplits;             // parts of the tokens
  float* sums;             // [tsplits][L][r][C], or RC: [tsplits][L][C][r]; tsplits 1: NULL
  void* out;               // the same without the parts
  int out_f32;
};

// Adapter (and ranks) by's sum over its tokens in range bz, columns of 64 a wave.  32 tokens are
// asked for ahead; 64 are no faster (4096 x 4096 x 4096, rank 16 57 us for 58; two of rank 64 87 for
// 78, the registers of the larger).  CR:
// results are [C][r] (dB), else [r][C] (dA).
template <int RM, int NP>
struct LoraSumLds {
  static constexpr int PP = 32 * RM + 16, ZP = 128 + 16;   // pitches of one token's ranks and columns
  uint8_t pl[NP * 32 * PP], zl[4 * 32 * ZP];
  int list[LORA_LIST], count[4];
};
#if SG_DEVICE_PASS
template <bool CR, int RM, int NP>
__device__ __forceinline__ void lora_sum(const LoraSum& a, LoraSumLds<RM, NP>& lds, int bx, int by, int bz) {
  constexpr int PP = LoraSumLds<RM, NP>::PP, ZP = LoraSumLds<RM, NP>::ZP;
  uint8_t *const pl = lds.pl, *const zl = lds.zl;
  int *const list = lds.list, *const count = lds.count;
  const int t = threadIdx.x, l = t & 63, g = l >> 4, lr = l & 15;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int chunks = (a.r + 16 * RM - 1) / (16 * RM);
  const int e = by / chunks, rho0 = (int)(by % chunks) * 16 * RM;
  const int n0 = (bx * 4 + wave) * 64;
  const int64_t b0 = a.T * bz / a.tsplits, b1 = a.T * (bz + 1) / a.tsplits;
  const float scale = a.scale ? a.scale[e] : 1.0f;
  v4f acc[4][RM];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int m = 0; m < RM; ++m) acc[i][m] = (v4f){0.f, 0.f, 0.f, 0.f};
  for (int64_t c0 = b0; c0 < b1; c0 += LORA_LIST) {
    // this adapter's tokens among LORA_LIST, in order: each wave looks through a quarter
    __syncthreads();
    int n = 0;
    uint64_t hit[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hit[i] = __ballot(lora_id(a.ids, c0 + wave * 256 + 64 * i + l, b1, a.L) == e);
      n += __builtin_popcountll(hit[i]);
    }
    if (l == 0) count[wave] = n;
    __syncthreads();
    int at = 0, total = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k < wave) at += count[k];
      total += count[k];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((hit[i] >> l) & 1) list[at + __builtin_popcountll(hit[i] & ((1ull << l) - 1))] = wave * 256 + 64 * i + l;
      at += __builtin_popcountll(hit[i]);
    }
    __syncthreads();
    uint4 zv[4];
    const auto load_z = [&](int k0) {   // 32 tokens x 64 columns of this wave
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = k0 + 8 * i + (l >> 3), c = n0 + 8 * (l & 7);
        zv[i] = make_uint4(0, 0, 0, 0);
        if (k < total && c < a.C) zv[i] = *reinterpret_cast<const uint4*>(a.z + (c0 + list[k]) * a.ldz + c);
      }
    };
    LoraValue value;   // eight ranks of one token
    const int vk = t / (2 * RM), vrho = rho0 + 8 * (t % (2 * RM));
    const auto load_v = [&](int k0) {
      const bool there = t < 64 * RM && k0 + vk < total && vrho < a.r;
      value.load(a.part, a.splits, a.T, a.r, there ? c0 + list[k0 + vk] : 0, vrho, there);
    };
    load_z(0);
    load_v(0);
    for (int k0 = 0; k0 < total; k0 += 32) {
      if (t < 64 * RM) {
        float v[8];
        value.total(scale, v);
        uint32_t p[NP][4];
        lora_parts<NP>(v, p);
#pragma unroll
        for (int q = 0; q < NP; ++q) *reinterpret_cast<uint4*>(pl + (q * 32 + vk) * PP + 16 * (t % (2 * RM))) = lora_pack(p[q]);
      }
      uint8_t* const st = zl + wave * 32 * ZP;
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(st + (8 * i + (l >> 3)) * ZP + 16 * (l & 7)) = zv[i];
      __syncthreads();
      load_z(k0 + 32);
      load_v(k0 + 32);
      const auto z_at = [&](int i) {
        // CR: columns as they are; else dealt so that a lane's results are 8 neighbours
        const int col = CR ? 32 * i + 8 * (lr & 3) : 64 * (i >> 1) + 16 * (lr & 3) + 8 * (i & 1);
        const uint8_t* const from = st + (8 * g + (lr >> 2)) * ZP + col;
        const uint2 x = lds_tr4(from), y = lds_tr4(from + 4 * ZP);
        return (v4i){(int)x.x, (int)x.y, (int)y.x, (int)y.y};
      };
      const auto p_at = [&](int m, int q) {
        const uint8_t* const from = pl + (q * 32 + 8 * g + (lr >> 2)) * PP + 32 * m + 8 * (lr & 3);
        const uint2 x = lds_tr4(from), y = lds_tr4(from + 4 * PP);
        return (v4i){(int)x.x, (int)x.y, (int)y.x, (int)y.y};
      };
      // Parts after the first, then the first one: the operand is read for each.  With both held, two
      // waves fit a SIMD instead of three (two adapters of rank 64 90 us for 81).
      v4i zf[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) zf[i] = lora_finite(z_at(i));
#pragma unroll
      for (int m = 0; m < RM; ++m)
#pragma unroll
        for (int q = NP - 1; q > 0; --q) {
          const v4i pf = p_at(m, q);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i][m] = CR ? w4_mfma(pf, zf[i], acc[i][m]) : w4_mfma(zf[i], pf, acc[i][m]);
        }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 4; ++i) zf[i] = z_at(i);
#pragma unroll
      for (int m = 0; m < RM; ++m) {
        const v4i pf = p_at(m, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i][m] = CR ? w4_mfma(pf, zf[i], acc[i][m]) : w4_mfma(zf[i], pf, acc[i][m]);
      }
      __syncthreads();
    }
  }
  const int64_t one = (int64_t)a.r * a.C;
  const bool f32 = a.tsplits > 1 || a.out_f32;
  float* const of = (a.tsplits > 1 ? a.sums + (int64_t)bz * a.L * one : reinterpret_cast<float*>(a.out)) + e * one;
  uint16_t* const ob = reinterpret_cast<uint16_t*>(a.out) + e * one;
  if (CR) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int m = 0; m < RM; ++m) {
        const int n = n0 + 16 * i + lr, rho = rho0 + 16 * m + 4 * g;
        if (n >= a.C || rho >= a.r) continue;
        const v4f v = acc[i][m];
        if (f32) *reinterpret_cast<float4*>(of + (int64_t)n * a.r + rho) = make_float4(v[0], v[1], v[2], v[3]);
        else *reinterpret_cast<uint2*>(ob + (int64_t)n * a.r + rho) =
            make_uint2(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]));
      }
  } else {
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int m = 0; m < RM; ++m) {
        const int n = n0 + 32 * q + 8 * g, rho = rho0 + 16 * m + lr;
        if (n >= a.C || rho >= a.r) continue;
        const v4f v = acc[2 * q][m], w = acc[2 * q + 1][m];
        if (f32) {
          float* const o = of + (int64_t)rho * a.C + n;
          *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
          *reinterpret_cast<float4*>(o + 4) = make_float4(w[0], w[1], w[2], w[3]);
        } else {
          *reinterpret_cast<uint4*>(ob + (int64_t)rho * a.C + n) =
              make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]), f32x2_to_bf16x2(w[0], w[1]),
                         f32x2_to_bf16x2(w[2], w[3]));
        }
      }
  }
}
#endif  // SG_DEVICE_PASS

// dA's workgroups come first along x, then dB's; behind those of the sums, dx's, whose
// product needs v as dA does: a launch less.
struct LoraGrid {
  int x, y, z;
  __host__ __device__ int64_t all() const { return (int64_t)x * y * z; }
};
template <int RM, int NP>
__global__ void __launch_bounds__(256) k_lora_sum(LoraSum a, LoraSum b, int a_x, LoraGrid sums, LoraUp dx, LoraGrid ups) {
#if SG_DEVICE_PASS
  __shared__ __attribute__((aligned(16))) union {
    LoraSumLds<RM, NP> sum;
    LoraUpLds<true> up;
  } lds;
  unsigned i = blockIdx.x;
  if (i < sums.all()) {
    const int bx = i % sums.x, by = i / sums.x % sums.y, bz = i / sums.x / sums.y;
    if (bx < a_x) lora_sum<false, RM, NP>(a, lds.sum, bx, by, bz);
    else lora_sum<true, RM, NP>(b, lds.sum, bx - a_x, by, bz);
  } else {
    i -= (unsigned)sums.all();
    lora_up<true, 2>(dx, lds.up, i % ups.x, i / ups.x % ups.y, i / ups.x / ups.y, ups.z);
  }
#endif
}

// The parts of both gradients, added in order.  (With dx's workgroups here, behind these,
// and not beside the sums: 4096 x 4096 x 4096, rank 16 57 us for 58, but two of rank 64 92 for 77.)
// n: values of one part, of dA then dB.
struct LoraJoin {
  const float* sums[2];
  void* out[2];
  int64_t n[2];
  int parts, out_f32;
};
__global__ void __launch_bounds__(256) k_lora_join(LoraJoin a) {
#if SG_DEVICE_PASS
  const int64_t step = (int64_t)gridDim.x * 1024;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < a.n[0] + a.n[1]; i += step) {
    const int h = i >= a.n[0];
    const int64_t at = h ? i - a.n[0] : i, n = h ? a.n[1] : a.n[0];
    const float* const p = (h ? a.sums[1] : a.sums[0]) + at;
    void* const o = h ? a.out[1] : a.out[0];
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < a.parts; ++s) {
      float x[4];
      load4(p + s * n, x);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] += x[k];
    }
    if (a.out_f32) *reinterpret_cast<float4*>(reinterpret_cast<float*>(o) + at) = make_float4(v[0], v[1], v[2], v[3]);
    else *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(o) + at) =
        make_uint2(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]));
  }
#endif
}

// ------------------------------------------------------------------ sizes

// Times below are of the launches alone, one call after another from a graph, K = N = 4096 where not said.

// Workgroups that share the items of a block of 64 tokens: as many as it may have,
// while that does not come to more than 1024.  Limits of 256 / 512 / 1024 / 2048 / 4096, mixed order, us:
// 37 tokens of 16 adapters, rank 64, N = 14336 21 / 17 / 15.6 / 15.7 / 15.7; 300 of 16, rank 32 23 / 17.6 /
// 16.4 / 18.5 / 18.5; 700 of 100, rank 32 119 / 77 / 65 / 74 / 93, gradients 193 / 136 / 114 / 116 / 143;
// but 1000 of 16, rank 16, gradients 48 / 34.7 / 36.4 / 39 / 43.
static int lora_slots(int64_t T, int64_t L, int64_t groups, int tm) {
  const int64_t n = T < 64 ? T : 64, most = (L < n ? L : n) + n / (16 * tm);
  int64_t s = 1024 / (groups < 1 ? 1 : groups);
  return (int)(s < 1 ? 1 : s > most ? most : s);
}

// Parts of a down product's sum: 256 workgroups where 16-token items give fewer, and only where one
// part would give its waves more than two units of 64 columns (1032 columns, two parts: one unit a
// wave).  1 / 2 parts, us: 1 token, K = 14336, rank 16 15.4 / 11.1; 40, rank 16 9.9 / 8.6; 1000, rank 16 12.9 /
// 11.8; 1000, rank 64, K = 14336 36 / 30; nothing is gained at 1032 (1 token 7.3 / 7.2), and many ranks lose by it
// (500 tokens of rank 64 14.1 / 14.8; 2048, K = 1032 26 / 29).
static int lora_splits(int64_t T, int64_t C) {
  int64_t s = 256 / cdiv(T, 16);
  const int64_t most = cdiv(C, 64 * 2 * LORA_WAVES);
  s = s > most ? most : s;
  return (int)(s < 1 ? 1 : s > LORA_PARTS ? LORA_PARTS : s);
}

// Parts of the tokens in the sums over them: 256 workgroups, 256 tokens of an adapter each
// at least, so that small calls need no launch to join them.  Which adapters the tokens have is not
// known here; the rule takes them as even.  4096 tokens, rank 16, 1 / 2 / 4 / 8 parts, us: one adapter 157 / 91 /
// 58 / 47 (16, the rule: 52); 8, even 54 / 57 (the rule) / 59 / 65, all tokens of one 158 / 103 / 83 / 59; 32,
// even 58 (the rule) / 73 / 81 / 109, all of one 159 / 109 / 83 / 102.
static int lora_tsplits(int64_t T, int64_t C, int64_t L) {
  int64_t s = 256 / (cdiv(C, 256) * L);
  const int64_t most = T / (256 * L);
  s = s > most ? most : s;
  return (int)(s < 1 ? 1 : s > 32 ? 32 : s);
}

struct LoraSpace {
  int64_t u, v, sa, sb, bytes;
  int su, sv, ts;
  LoraSpace(int64_t T, int64_t K, int64_t N, int64_t r, int64_t L, bool back) {
    int64_t at = 0;
    const auto part = [&](int64_t n) { const int64_t was = at; at += cdiv(n, 256) * 256; return was; };
    su = lora_splits(T, K);
    sv = lora_splits(T, N);
    ts = lora_tsplits(T, K > N ? K : N, L);
    u = part(4 * su * T * r);
    v = sa = sb = 0;
    if (back) {
      v = part(4 * sv * T * r);
      if (ts > 1) {
        sa = part(4 * ts * L * r * K);
        sb = part(4 * ts * L * r * N);
      }
    }
    bytes = at;
  }
};

// Tokens of a down workgroup's item in 16s: an adapter read for 32 where there are many in a row.  16 / 32 at
// 64 ranks a workgroup, runs of 4 adapters, us: 2048 tokens, rank 64 37.6 / 34.0, rank 128 62.5 / 57.2; gradients
// of 4096, rank 256 283 / 245; 500, rank 64 15.9 / 17.0 (the edge: 600, rank 256 47.8 / 43.5).  In mixed order
// the items are not full and 32 lose: 1000 of 16 adapters, rank 48 41 / 50, 2048, rank 64 91 / 94.
static int lora_tm(int64_t T, int64_t r) { return T >= 512 && r > 32 ? 2 : 1; }
// Ranks of a down workgroup in 16s: more where there are many, so that z is read less often, fewer
// where more workgroups are wanted.  1 / 2 / 4, runs of 4 adapters, us: 300 tokens, rank 32 10.0 / 10.5 / 11.4, rank
// 128 18.1 / 17.2 / 19.4; 2048, rank 32 23.4 / 22.4 / 21.5; gradients of 4096, rank 32 73.4 / 70.9 / 73.0; with 32-token
// items 2 / 4: 600, rank 64 18.8 / 20.7, 2048, rank 64 36.6 / 34.0, gradients of 2048, rank 128 95.3 / 92.6.
// Off by most at the edges: gradients of 300, rank 64 (1: 23.2, 2: 19.1), 500, rank 256 (4: 39.3, 2: 36.2).
static int lora_rm(int64_t T, int64_t r, int splits) {
  const int64_t tiles = splits * cdiv(T, 16) * cdiv(r, 16);
  const int rm = r <= 16 || tiles <= 256 ? 1 : r <= 32 || tiles <= 512 ? 2 : 4;
  return rm == 1 && lora_tm(T, r) == 2 ? 2 : rm;
}
// Of a workgroup of the sums, of one launch for both products.
static int lora_rm(int64_t r) { return r <= 16 ? 1 : r <= 32 ? 2 : 4; }
template <int TM, int RM>
static void launch_down_tm(const LoraDown* v, const LoraDown* u, hipStream_t st) {
  const LoraDown& a = v ? *v : *u;
  const unsigned gx = (unsigned)cdiv(a.T, 64), chunks = (unsigned)cdiv(a.r, 16 * RM);
  const unsigned gv = v ? v->splits * chunks : 0, gu = u ? u->splits * chunks : 0;
  const dim3 grid(gx, gv + gu, (unsigned)lora_slots(a.T, a.L, (int64_t)gx * (gv + gu), TM));
  if (v && u) k_lora_down_two<TM, RM><<<grid, 512, 0, st>>>(*v, *u, (int)gv);
  else if (v) k_lora_down<true, TM, RM><<<grid, 512, 0, st>>>(*v);
  else k_lora_down<false, TM, RM><<<grid, 512, 0, st>>>(*u);
}
// dy . B (v) and x . A^T (u), either or both.
static void launch_down(const LoraDown* v, const LoraDown* u, hipStream_t st) {
  const LoraDown& a = v ? *v : *u;
  const int rm = lora_rm(a.T, a.r, a.splits);
  if (lora_tm(a.T, a.r) == 2) {
    if (rm == 2) launch_down_tm<2, 2>(v, u, st);
    else launch_down_tm<2, 4>(v, u, st);
  } else {
    if (rm == 1) launch_down_tm<1, 1>(v, u, st);
    else if (rm == 2) launch_down_tm<1, 2>(v, u, st);
    else launch_down_tm<1, 4>(v, u, st);
  }
}

static LoraGrid lora_up_grid(const LoraUp& a) {
  const int64_t gx = cdiv(a.T, 64), gy = cdiv(a.C, 256);
  return {(int)gx, (int)gy, lora_slots(a.T, a.L, gx * gy, 1)};
}
template <bool KS>
static void launch_up(const LoraUp& a, hipStream_t st) {
  const LoraGrid g = lora_up_grid(a);
  const dim3 grid(g.x, g.y, g.z);
  if (a.y_f32) k_lora_up<KS, 3><<<grid, 256, 0, st>>>(a);
  else k_lora_up<KS, 2><<<grid, 256, 0, st>>>(a);
}

// Both sums, and dx where it is not NULL.
template <int NP>
static void launch_sum(const LoraSum& a, const LoraSum& b, const LoraUp* dx, hipStream_t st) {
  const int ax = (int)cdiv(a.C, 256), bx = (int)cdiv(b.C, 256);
  const LoraUp none = {};
  const LoraGrid ups = dx ? lora_up_grid(*dx) : LoraGrid{0, 0, 0};
  const auto sums = [&](int rm) { return LoraGrid{ax + bx, (int)(a.L * cdiv(a.r, 16 * rm)), a.tsplits}; };
  const auto all = [&](int rm) { return (unsigned)(sums(rm).all() + ups.all()); };
  const LoraUp& u = dx ? *dx : none;
  const int rm = lora_rm(a.r);
  if (rm == 1) k_lora_sum<1, NP><<<all(1), 256, 0, st>>>(a, b, ax, sums(1), u, ups);
  else if (rm == 2) k_lora_sum<2, NP><<<all(2), 256, 0, st>>>(a, b, ax, sums(2), u, ups);
  else k_lora_sum<4, NP><<<all(4), 256, 0, st>>>(a, b, ax, sums(4), u, ups);
}

// Whether a call's two products go in one launch: up to 256 KB of an adapter's A, which every workgroup
// goes through.  Two launches / one, us, calls one after another from the host; from a graph: 1 token, rank 16
// 12.2 / 8.9; 7.8 / 7.1.  Rank 32 (the edge) 12.0 / 8.8; 7.7 / 8.1.  Rank 64 11.8 / 11.3; 8.9 / 10.9.  64 tokens, rank
// 32, N = 14336 11.7 / 11.1; 9.8 / 10.8.  37, rank 64 11.5 / 12.9; 10.3 / 13.0.  1, rank 8, K = 14336 11.8 / 12.8;
// 10.7 / 12.7.  From the host the second launch counts, so the edge is where a graph would already do
// better with two.  More than 64 tokens or ranks have no such kernel.
static bool lora_both(int64_t T, int64_t C, int64_t r) { return T <= 64 && r <= 64 && 2 * C * r <= 256 * 1024; }

template <int RM>
static void launch_both_rm(const LoraBoth& b, dim3 grid, hipStream_t st) {
  if (b.u.y_f32) k_lora_both<RM, 3><<<grid, 512, 0, st>>>(b);
  else k_lora_both<RM, 2><<<grid, 512, 0, st>>>(b);
}
static void launch_both(LoraBoth b, hipStream_t st) {
  const int64_t T = b.d.T, items = (b.d.L < T ? b.d.L : T) + T / 16;
  int64_t slices = 256 / items, most = cdiv(b.u.C, 64 * LORA_WAVES);
  slices = slices < 1 ? 1 : slices > most ? most : slices;
  b.slice = (int)cdiv(cdiv(b.u.C, 64), slices) * 64;
  const dim3 grid((unsigned)cdiv(T, 64), (unsigned)cdiv(b.u.C, b.slice), (unsigned)items);
  const int rm = lora_rm(b.d.r);
  if (rm == 1) launch_both_rm<1>(b, grid, st);
  else if (rm == 2) launch_both_rm<2>(b, grid, st);
  else launch_both_rm<4>(b, grid, st);
}

static bool lora_shape_ok(int64_t T, int64_t K, int64_t N, int64_t r, int64_t L) {
  if (T < 1 || K < 8 || N < 8 || r < 8 || L < 1 || K % 8 || N % 8 || r % 8) return false;
  return T < (1LL << 22) && K < (1LL << 22) && N < (1LL << 22) && r <= 256 && L <= 65535;
}
static bool lora_back_ok(int64_t T, int64_t K, int64_t N, int64_t r, int64_t L) {
  // workgroups of the sums and of dx, in one launch along x (parts of the tokens, and of a block's
  // items, are only where there are few)
  const int64_t c = K > N ? K : N;
  return lora_shape_ok(T, K, N, r, L) && launch_fits(cdiv(c, 256) * (2 * L * cdiv(r, 64) + cdiv(T, 64)) + 4096, 256);
}
static bool lora_ld_ok(int64_t ld, int64_t cols) { return ld >= cols && ld < (1LL << 22); }

}  // namespace sg

using namespace sg;

extern "C" int64_t sg_lora_gemm_workspace(int64_t T, int64_t K, int64_t N, int r, int64_t L) {
  if (!lora_shape_ok(T, K, N, r, L)) return -1;
  return lora_both(T, K, r) ? 0 : LoraSpace(T, K, N, r, L, false).bytes;
}

extern "C" int64_t sg_lora_gemm_backward_workspace(int64_t T, int64_t K, int64_t N, int r, int64_t L) {
  if (!lora_back_ok(T, K, N, r, L)) return -1;
  return LoraSpace(T, K, N, r, L, true).bytes;
}

extern "C" sg_status sg_lora_gemm_plan(int64_t T, int64_t K, int64_t N, int r, int64_t L, int32_t* plan) {
  if (!plan) return SG_ERR_NULL;
  if (!lora_shape_ok(T, K, N, r, L)) return SG_ERR_SHAPE;
  const bool both = lora_both(T, K, r);
  const int parts = both ? 1 : lora_splits(T, K);
  plan[0] = both ? 1 : 2;
  plan[1] = both ? 16 : 16 * lora_tm(T, r);
  plan[2] = 16 * (both ? lora_rm(r) : lora_rm(T, r, parts));
  plan[3] = parts;
  return SG_OK;
}

extern "C" sg_status sg_lora_gemm_backward_plan(int64_t T, int64_t K, int64_t N, int r, int64_t L, int32_t* plan) {
  if (!plan) return SG_ERR_NULL;
  if (!lora_back_ok(T, K, N, r, L)) return SG_ERR_SHAPE;
  const LoraSpace ws(T, K, N, r, L, true);
  plan[0] = 16 * lora_tm(T, r);
  plan[1] = 16 * lora_rm(T, r, ws.sv);
  plan[2] = ws.sv;
  plan[3] = ws.su;
  plan[4] = 16 * lora_rm(r);
  plan[5] = ws.ts;
  return SG_OK;
}

extern "C" sg_status sg_lora_gemm(int64_t T, int64_t K, int64_t N, int r, int64_t L, const uint16_t* x, int64_t ldx,
                                  const int32_t* ids, const uint16_t* a, const uint16_t* b, const float* scale,
                                  const void* base, sg_dtype base_dt, int64_t ld_base, void* y, sg_dtype y_dt,
                                  int64_t ldy, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  if (!x || !a || !b || !y) return SG_ERR_NULL;
  if ((y_dt != SG_F32 && y_dt != SG_BF16) || (base && base_dt != SG_F32 && base_dt != SG_BF16))
    return SG_ERR_UNSUPPORTED;
  if (!lora_shape_ok(T, K, N, r, L) || !lora_ld_ok(ldx, K) || !lora_ld_ok(ldy, N) ||
      (base && !lora_ld_ok(ld_base, N)) || (base == y && (base_dt != y_dt || ld_base != ldy)))
    return SG_ERR_SHAPE;
  const LoraSpace ws(T, K, N, r, L, false);
  const bool both = lora_both(T, K, r);
  if (!both && !workspace) return SG_ERR_NULL;
  if (!both && workspace_bytes < ws.bytes) return SG_ERR_SHAPE;
  if (ldx % 8 || ldy % 8 || (base && ld_base % 8) || !aligned(x, 16) || !aligned(ids, 4) || !aligned(a, 16) ||
      !aligned(b, 16) || !aligned(scale, 4) || !aligned(base, 16) || !aligned(y, 16) ||
      (!both && !aligned(workspace, 256)))
    return SG_ERR_ALIGN;
  clear_hip_error();
  float* const part = reinterpret_cast<float*>(workspace);
  LoraDown q = {T, (int)K, r, (int)L, ws.su, x, a, ldx, ids, part};
  LoraUp p = {};
  p.T = T; p.C = (int)N; p.r = r; p.L = (int)L; p.splits = ws.su; p.part = part; p.scale = scale; p.ids = ids; p.w = b;
  p.base = base; p.ld_base = ld_base; p.base_f32 = base && base_dt == SG_F32; p.y = y; p.ldy = ldy; p.y_f32 = y_dt == SG_F32;
  if (both) {
    launch_both(LoraBoth{q, p, 0}, stream);
  } else {
    launch_down(nullptr, &q, stream);
    launch_up<false>(p, stream);
  }
  return launch_status();
}

extern "C" sg_status sg_lora_gemm_backward(int64_t T, int64_t K, int64_t N, int r, int64_t L, const uint16_t* dy,
                                           int64_t ld_dy, const uint16_t* x, int64_t ldx, const int32_t* ids,
                                           const uint16_t* a, const uint16_t* b, const float* scale,
                                           const uint16_t* base, int64_t ld_base, uint16_t* dx, int64_t ld_dx,
                                           void* da, void* db, sg_dtype grad_dt, void* workspace,
                                           int64_t workspace_bytes, hipStream_t stream) {
  if (!dy || !x || !a || !b || !workspace || (!dx && !da) || !da != !db) return SG_ERR_NULL;
  if (da && grad_dt != SG_F32 && grad_dt != SG_BF16) return SG_ERR_UNSUPPORTED;
  if (!lora_back_ok(T, K, N, r, L) || !lora_ld_ok(ldx, K) || !lora_ld_ok(ld_dy, N) || (dx && !lora_ld_ok(ld_dx, K)) ||
      (dx && base && !lora_ld_ok(ld_base, K)) || (dx && base == dx && ld_base != ld_dx))
    return SG_ERR_SHAPE;
  const LoraSpace ws(T, K, N, r, L, true);
  if (workspace_bytes < ws.bytes) return SG_ERR_SHAPE;
  if (ldx % 8 || ld_dy % 8 || (dx && ld_dx % 8) || (dx && base && ld_base % 8) || !aligned(dy, 16) || !aligned(x, 16) ||
      !aligned(ids, 4) || !aligned(a, 16) || !aligned(b, 16) || !aligned(scale, 4) || !aligned(base, 16) ||
      !aligned(dx, 16) || !aligned(da, 16) || !aligned(db, 16) || !aligned(workspace, 256))
    return SG_ERR_ALIGN;
  clear_hip_error();
  uint8_t* const w = reinterpret_cast<uint8_t*>(workspace);
  float *const u = reinterpret_cast<float*>(w + ws.u), *const v = reinterpret_cast<float*>(w + ws.v);
  const LoraDown dv = {T, (int)N, r, (int)L, ws.sv, dy, b, ld_dy, ids, v}, du = {T, (int)K, r, (int)L, ws.su, x, a, ldx, ids, u};
  launch_down(&dv, da ? &du : nullptr, stream);
  LoraUp p = {};
  if (dx) {
    p.T = T; p.C = (int)K; p.r = r; p.L = (int)L; p.splits = ws.sv; p.part = v; p.scale = scale; p.ids = ids; p.w = a;
    p.base = base; p.ld_base = ld_base; p.y = dx; p.ldy = ld_dx;
    if (!da) launch_up<true>(p, stream);
  }
  if (da) {
    LoraSum s = {};
    s.T = T; s.C = (int)K; s.r = r; s.L = (int)L; s.splits = ws.sv; s.z = x; s.ldz = ldx; s.part = v; s.scale = scale;
    s.ids = ids; s.tsplits = ws.ts; s.sums = reinterpret_cast<float*>(w + ws.sa); s.out = da;
    s.out_f32 = grad_dt == SG_F32;
    LoraSum q = s;
    q.C = (int)N; q.splits = ws.su; q.z = dy; q.ldz = ld_dy; q.part = u; q.sums = reinterpret_cast<float*>(w + ws.sb);
    q.out = db;
    if (s.out_f32) launch_sum<3>(s, q, dx ? &p : nullptr, stream);
    else launch_sum<2>(s, q, dx ? &p : nullptr, stream);
    if (ws.ts > 1) {
      LoraJoin j = {};
      j.sums[0] = reinterpret_cast<float*>(w + ws.sa); j.sums[1] = reinterpret_cast<float*>(w + ws.sb);
      j.out[0] = da; j.out[1] = db; j.n[0] = L * r * K; j.n[1] = L * r * N; j.parts = ws.ts;
      j.out_f32 = grad_dt == SG_F32;
      k_lora_join<<<grid_for((j.n[0] + j.n[1]) / 4, 256, 4096), 256, 0, stream>>>(j);
    }
  }
  return launch_status();
}
