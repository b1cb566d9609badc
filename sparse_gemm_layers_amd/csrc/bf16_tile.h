// Tile product of two bf16 matrices: D[n, m] = sum_k L[n, k] R[m, k] with fp32
// sums, BN x BM per workgroup of 8 waves, each operand stored either with k along
// its rows ("KC": a row of the operand is contiguous in k) or across them ("KS":
// a row holds one k), so that a forward product, the gradient of its input and
// that of its weight all read the matrices as the caller has them.
//
// A step is 32 k: one 16x16x32 matrix instruction per pair of sub-tiles.  Steps go
// through a ring of S stages in LDS that buffer loads fill directly.  A KC stage
// holds 64-byte rows (16-byte piece c of row r at c ^ swz4(r)), read 16 bytes a
// lane; a KS stage holds 32 rows of one k each (64-byte piece c of row k at
// c ^ f(k)), read with ds_read_b64_tr_b16, which hands each lane four k of one
// column.  What a wave reads of stage k + 1 replaces what the matrix core has
// taken of stage k in registers, so a step's single barrier both opens stage
// k + 1 and frees stage k for the loads of k + S.
//
// Left rows are dealt to sub-tiles so that a lane's results of two neighbouring
// sub-tiles are 8 consecutive n: row i of sub-tile 2 p + b is
// n = 32 p + 8 (i / 4) + 4 b + i % 4.  Stores are 16 bytes a lane.
#pragma once

#include <type_traits>

#include "tile_epilogue.h"
#include "w4.h"

namespace sg {

#if SG_DEVICE_PASS
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

// Four k of one column a lane: lane 16 g + 4 j + a gives the address of row j's
// a-th group of 4 columns, lane 16 g + c gets column c of the 4 rows.
__device__ __forceinline__ uint2 lds_tr4(const uint8_t* p) {
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)p));
}
// 16 bytes a lane from the records of p (base, bytes; soff and off in bytes, off past
// the records: zero) to LDS, lane l's at address dst + 16 l.  In assembly because the compiler, which
// follows such loads into LDS, would wait for all of them before each of the reads
// above; run() counts them itself.  It has no result register to be overwritten.
__device__ __forceinline__ void lds_dma16(const void* p, uint32_t bytes, uint32_t off, int soff, uint32_t dst) {
  const uint64_t at = (uint64_t)p;
  const v4i r = {(int)at, (int)(at >> 32), (int)bytes, 0x00020000};
  uint32_t was;   // m0 is given back: the compiler does not let it be named as overwritten
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, %4 offen lds\n\t"
               "s_mov_b32 m0, %0"
               : "=&s"(was) : "s"(dst), "v"(off), "s"(r), "s"(soff) : "memory");
}
// n of row r of sub-tile s, relative to the wave's first.
__device__ __forceinline__ int tile_n(int s, int r) { return 32 * (s >> 1) + 8 * (r >> 2) + 4 * (s & 1) + (r & 3); }

// One wave's loads of a KC operand: U instructions of 16 rows a stage.  p[seg]: the
// first column of row 0 that off counts from; the two are the two segments of a sum
// over k (seg), or which of two matrices an instruction's rows are of (sel).
template <int U>
struct KcOp {
  const uint16_t* p[2];
  uint32_t bytes[2];
  uint32_t off[U];      // of this lane's piece, W4_OUT: row not there
  uint32_t last[U];     // the same in the last step of a segment, W4_OUT where k is past the end too
  int sel[U];
  // lane l's piece of 16-byte pieces of row l / 4
  __device__ static __forceinline__ int piece(int l) { return (l & 3) ^ swz4(l >> 2); }
  __device__ __forceinline__ void set(int u, bool there, int64_t row_off, int K, int l) {
    const int c = 8 * piece(l);
    off[u] = there ? (uint32_t)((row_off + c) * 2) : W4_OUT;
    last[u] = there && (cdiv_(K) - 1) * 32 + c < K ? off[u] : W4_OUT;
  }
  __device__ static __forceinline__ int cdiv_(int K) { return (K + 31) >> 5; }
  __device__ __forceinline__ void load(int u, uint32_t dst, int seg, int kb, int KB, bool live) const {
    const int s = sel[u] ^ seg;
    // an empty descriptor takes no scalar offset: the range check subtracts that from its size
    lds_dma16(s ? p[1] : p[0], live ? (s ? bytes[1] : bytes[0]) : 0u, kb == KB - 1 ? last[u] : off[u],
              live ? kb * 64 : 0, dst);
  }
};

// One wave's loads of a KS operand of B columns.  p[seg], ld[seg]: row k = 0, the
// tile's first column.  Rows past K are outside of the descriptor and read as zero.
template <int U, int B>
struct KsOp {
  const uint16_t* p[2];
  int64_t ld[2];
  uint32_t width;       // bytes of a row from the tile's first column on
  int K;
  uint32_t off[2][U];
  static constexpr int RPI = 512 / B;   // rows an instruction brings
  __device__ static __forceinline__ int swz(int k) { return B == 256 ? (k & 3) | ((k >> 1) & 4) : k & 3; }
  __device__ __forceinline__ void set(int wave, int l) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = RPI * (8 * u + wave) + l / (B / 8), c = l % (B / 8);   // 16-byte piece c of row k
#pragma unroll
      for (int s = 0; s < 2; ++s) off[s][u] = (uint32_t)(k * ld[s] * 2) + 16 * (c ^ (swz(k) << 2));
    }
  }
  __device__ __forceinline__ void load(int u, uint32_t dst, int seg, int kb, int, bool live) const {
    const int rows = live ? min(K - 32 * kb, 32) : 0;
    const int64_t d = seg ? ld[1] : ld[0];
    lds_dma16((seg ? p[1] : p[0]) + (int64_t)kb * 32 * d, rows > 0 ? (uint32_t)((rows - 1) * d * 2) + width : 0u,
              seg ? off[1][u] : off[0][u], 0, dst);
  }
};
#endif  // SG_DEVICE_PASS

// WN x WM waves of NI x MJ sub-tiles each.
template <bool LKS_, bool RKS_, int WN_, int WM_, int NI_, int MJ_, int S_ = 4>
struct Bf16Tile {
  static constexpr bool LKS = LKS_, RKS = RKS_;
  static constexpr int WN = WN_, WM = WM_, NI = NI_, MJ = MJ_, S = S_;
  static_assert(WN * WM == 8 && NI % 2 == 0 && MJ % 2 == 0, "waves");
  static constexpr int BN = WN * NI * 16, BM = WM * MJ * 16;
  static constexpr int L_BYTES = BN * 64, STAGE = (BN + BM) * 64, LDS = S * STAGE;
  static constexpr int LU = BN / 128, RU = BM / 128, LOADS = LU + RU;
  static_assert(LDS <= 160 * 1024, "LDS");
#if SG_DEVICE_PASS
  template <bool C, typename A, typename B> struct pick { using type = A; };
  template <typename A, typename B> struct pick<false, A, B> { using type = B; };
  using L = typename pick<LKS, KsOp<LU, BN>, KcOp<LU>>::type;
  using R = typename pick<RKS, KsOp<RU, BM>, KcOp<RU>>::type;

  // acc[i][j]: sub-tile row i, column j of this wave over steps kb0 .. kb1 - 1; step
  // kb is step kb % KB of segment kb / KB (at most two).
  __device__ static __forceinline__ void run(uint8_t* lds, const L& lo, const R& ro, int kb0, int kb1, int KB,
                                             int wave, int l, v4f (&acc)[NI][MJ]) {
    const int g = l >> 4, lr = l & 15, wn = wave / WM, wm = wave % WM;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < MJ; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
    const uint32_t lds0 = (uint32_t)(uintptr_t)(w4_lds_t*)lds;
    const auto load_one = [&](int n, int kb, int slot) {
      const int seg = kb >= KB, at = seg ? kb - KB : kb;
      const uint32_t dst = lds0 + slot * STAGE;
      if (n < LU) lo.load(n, dst + (8 * n + wave) * 1024, seg, at, KB, kb < kb1);
      else ro.load(n - LU, dst + L_BYTES + (8 * (n - LU) + wave) * 1024, seg, at, KB, kb < kb1);
    };
    // addresses within a stage
    constexpr int LP = LKS ? NI / 2 : 1, RP = RKS ? MJ / 2 : 1;
    int la[LP], ra[RP];
    const int kr = 8 * g + (lr >> 2), a = lr & 3;   // KS: row of the first four k, group of 4 columns
    if constexpr (LKS) {
#pragma unroll
      for (int p = 0; p < LP; ++p) la[p] = kr * (BN * 2) + (((wn * (NI / 2) + p) ^ KsOp<LU, BN>::swz(kr)) << 6) + 16 * a;
    } else {
      la[0] = (wn * NI * 16 + lr) * 64 + ((g ^ swz4(lr)) << 4);
    }
    if constexpr (RKS) {
#pragma unroll
      for (int p = 0; p < RP; ++p)
        ra[p] = L_BYTES + kr * (BM * 2) + (((wm * (MJ / 2) + p) ^ KsOp<RU, BM>::swz(kr)) << 6) + 8 * a;
    } else {
      ra[0] = L_BYTES + (wm * MJ * 16 + lr) * 64 + ((g ^ swz4(lr)) << 4);
    }
    const auto read_l = [&](const uint8_t* st, int i) {
      if constexpr (LKS) {
        const uint2 x = lds_tr4(st + la[i >> 1] + 8 * (i & 1)), y = lds_tr4(st + la[i >> 1] + 8 * (i & 1) + 4 * BN * 2);
        return (v4i){(int)x.x, (int)x.y, (int)y.x, (int)y.y};
      } else {
        return *reinterpret_cast<const v4i*>(st + la[0] + i * 1024);
      }
    };
    const auto read_r = [&](const uint8_t* st, int j) {
      if constexpr (RKS) {
        const uint2 x = lds_tr4(st + ra[j >> 1] + 32 * (j & 1)), y = lds_tr4(st + ra[j >> 1] + 32 * (j & 1) + 4 * BM * 2);
        return (v4i){(int)x.x, (int)x.y, (int)y.x, (int)y.y};
      } else {
        return *reinterpret_cast<const v4i*>(st + ra[0] + j * 1024);
      }
    };
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int n = 0; n < LOADS; ++n) load_one(n, kb0 + s, s);
    w4_wait<(S - 1) * LOADS>();
    lds_barrier();
    v4i fl[NI], fr[2][MJ];
#pragma unroll
    for (int i = 0; i < NI; ++i) fl[i] = read_l(lds, i);
#pragma unroll
    for (int j = 0; j < MJ; ++j) fr[0][j] = read_r(lds, j);
    int slot = 0;
    const auto step = [&](int kb, auto pr) {
      constexpr int PR = decltype(pr)::value;
      const int nslot = slot + 1 == S ? 0 : slot + 1;
      const uint8_t* const st = lds + nslot * STAGE;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
#pragma unroll
        for (int j = 0; j < MJ; ++j) acc[i][j] = w4_mfma(fl[i], fr[PR][j], acc[i][j]);
        if (i == 0) {
          // own loads of kb + 1 have landed; every wave has read all of kb
          w4_wait<(S - 2) * LOADS>();
          lds_barrier();
        }
        fl[i] = read_l(st, i);
#pragma unroll
        for (int j = i * MJ / NI; j < (i + 1) * MJ / NI; ++j) fr[PR ^ 1][j] = read_r(st, j);
#pragma unroll
        for (int n = i * LOADS / NI; n < (i + 1) * LOADS / NI; ++n) load_one(n, kb + S, slot);
        __builtin_amdgcn_sched_barrier(0);
      }
      slot = nslot;
    };
    using Z = std::integral_constant<int, 0>;
    using O = std::integral_constant<int, 1>;
    int kb = kb0;
    for (; kb + 1 < kb1; kb += 2) {
      step(kb, Z{});
      step(kb + 1, O{});
    }
    if (kb < kb1) step(kb, Z{});
    w4_wait<0>();   // loads past the end have landed before LDS is given up
  }
#endif  // SG_DEVICE_PASS
};

}  // namespace sg
