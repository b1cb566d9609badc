// Tile product of two bf16 matrices: D[n, m] = sum_k L[n, k] R[m, k] with fp32
// sums, BN x BM per workgroup of 8 waves, each operand stored either with k along
// its rows ("KC": a row of the operand is contiguous in k) or across them ("KS":
// a row holds one k), so that a forward product, the gradient of its input and
// that of its weight all read the matrices as the caller has them.
//
// k goes by blocks of 64, two in LDS at a time, which buffer loads fill directly;
// a block is two steps of 32, one 16x16x32 matrix instruction per pair of sub-tiles.
// A KC block holds 128-byte rows (16-byte piece c of row r at c ^ swz8q(r)), read 16
// bytes a lane: with 64-byte rows every line came from L2 twice.  A KS block holds
// 64 rows of one k each (64-byte piece c of row k at c ^ swz(k)), read with
// ds_read_b64_tr_b16, which hands each lane four k of one column.  What a wave reads of
// the next step replaces what the matrix core has taken of this one in registers; so
// the block's single barrier, in its second step, both opens the next block and frees
// this one for the loads of the one after.
//
// Left rows are dealt to sub-tiles so that a lane's results of two neighbouring
// sub-tiles are 8 consecutive n: row i of sub-tile 2 p + b is
// n = 32 p + 8 (i / 4) + 4 b + i % 4.  Stores are 16 bytes a lane.
#pragma once

#include <type_traits>

#include "tile_epilogue.h"
#include "w4.h"

namespace sg {

// Rows in order, one matrix a segment.
struct PlainRow {
#if SG_DEVICE_PASS
  __device__ static __forceinline__ int row(int u, int wave, int l) { return 8 * (8 * u + wave) + (l >> 3); }
  __device__ static __forceinline__ int sel(int, int) { return 0; }
#endif
};

#if SG_DEVICE_PASS
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

// Four k of one column a lane: lane 16 g + 4 j + a gives the address of row j's
// a-th group of 4 columns, lane 16 g + c gets column c of the 4 rows.
__device__ __forceinline__ uint2 lds_tr4(const uint8_t* p) {
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)p));
}
// 16 bytes a lane from the records of r to LDS, lane l's at address base + AT + 16 l.  In
// assembly because the compiler, which follows such loads into LDS, would wait for
// all of them before each of the reads above; run() counts them itself.  It has no
// result register to be overwritten.  m0 is written and not named: the compiler has
// no use of its own for it in these kernels (tests/test_tile_assembly.py).
template <int AT>
__device__ __forceinline__ void lds_dma16(const v4i& r, uint32_t off, int soff, uint32_t base) {
  asm volatile("s_add_u32 m0, %0, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(base), "v"(off),
               "s"(r), "s"(soff), "n"(AT)
               : "memory", "scc");
}
__device__ __forceinline__ v4i tile_rsrc(const void* p, uint32_t bytes) {
  const uint64_t at = (uint64_t)p;
  return (v4i){__builtin_amdgcn_readfirstlane((int)at), __builtin_amdgcn_readfirstlane((int)(at >> 32)),
               __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}
// n of row r of sub-tile s, relative to the wave's first.
__device__ __forceinline__ int tile_n(int s, int r) { return 32 * (s >> 1) + 8 * (r >> 2) + 4 * (s & 1) + (r & 3); }

// One wave's loads of a KC operand: U instructions of 8 rows a block.  The sum over k
// has one segment or two of KB blocks, each with a matrix of its own; p[seg] is the
// first column of row 0.  Row::row(u, wave, l) is the row that lane l of instruction u
// loads; Row::sel(u, wave) which of the two matrices it is of, where it is not the
// segment that says so.  Rows past the last lie outside of the descriptor (it ends
// with the last row) and read as zero.
template <int U, typename Row>
struct KcOp {
  const uint16_t* p[2];
  int64_t ld[2];
  uint32_t bytes[2];
  int K, wave, l;
  v4i r[U];             // where the next block's loads are
  uint32_t cur[U];
  int soff;
  // Block k of segment seg is next; none: nothing but zeros is.
  __device__ __forceinline__ void place(int k, int seg, int KB, bool none) {
    soff = none ? 0 : k * 128;   // an empty descriptor takes no scalar offset: the range check subtracts that from its size
    const int c = 8 * ((l & 7) ^ swz8q(l >> 3));   // k of this lane's piece of 16 bytes
    const bool out = k * 64 + c >= K;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = Row::sel(u, wave) ^ seg;
      r[u] = tile_rsrc(s ? p[1] : p[0], none ? 0u : s ? bytes[1] : bytes[0]);
      cur[u] = out ? W4_OUT : (uint32_t)((Row::row(u, wave, l) * (s ? ld[1] : ld[0]) + c) * 2);
    }
  }
  template <int AT>
  __device__ __forceinline__ void load(int u, uint32_t base) const { lds_dma16<AT>(r[u], cur[u], soff, base); }
  __device__ __forceinline__ void next() { soff += 128; }
};

// One wave's loads of a KS operand of B columns.  p[seg], ld[seg]: row k = 0, the
// tile's first column.  Rows past K are outside of the descriptor and read as zero.
template <int U, int B>
struct KsOp {
  const uint16_t* p[2];
  int64_t ld[2];
  uint32_t width;       // bytes of a row from the tile's first column on
  int K, wave, l;
  v4i r;
  uint32_t cur[U];
  uint32_t step;        // bytes of 64 rows
  static constexpr int RPI = 512 / B;   // rows an instruction brings
  __device__ static __forceinline__ int swz(int k) { return B == 256 ? (k & 3) | ((k >> 1) & 4) : k & 3; }
  __device__ __forceinline__ void place(int k, int seg, int, bool none) {
    const int64_t d = seg ? ld[1] : ld[0];
    step = (uint32_t)(128 * d);
    r = tile_rsrc((seg ? p[1] : p[0]) + (int64_t)k * 64 * d,
                  none ? 0u : (uint32_t)((min(K - 64 * k, 64) - 1) * d * 2) + width);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = RPI * (8 * u + wave) + l / (B / 8);   // 16-byte piece l % (B / 8) of this row
      cur[u] = (uint32_t)(row * d * 2) + 16 * ((l % (B / 8)) ^ (swz(row) << 2));
    }
  }
  template <int AT>
  __device__ __forceinline__ void load(int u, uint32_t base) const { lds_dma16<AT>(r, cur[u], 0, base); }
  __device__ __forceinline__ void next() {
    const uint64_t at = (((uint64_t)(uint32_t)r[1] << 32) | (uint32_t)r[0]) + step;
    r[0] = (int)at;
    r[1] = (int)(at >> 32);
  }
};
#endif  // SG_DEVICE_PASS

// WN x WM waves of NI x MJ sub-tiles each.  LRow: the left operand's rows, where it is KC.
template <bool LKS_, bool RKS_, int WN_, int WM_, int NI_, int MJ_, typename LRow = void>
struct Bf16Tile {
  static constexpr bool LKS = LKS_, RKS = RKS_;
  static constexpr int WN = WN_, WM = WM_, NI = NI_, MJ = MJ_;
  static_assert(WN * WM == 8 && NI % 2 == 0 && MJ % 2 == 0, "waves");
  static constexpr int BN = WN * NI * 16, BM = WM * MJ * 16;
  static constexpr int L_BYTES = BN * 128, BLOCK = (BN + BM) * 128, LDS = 2 * BLOCK;
  static constexpr int LU = BN / 64, RU = BM / 64, LOADS = LU + RU;
  static_assert(LDS <= 160 * 1024, "LDS");
#if SG_DEVICE_PASS
  template <bool C, typename A, typename B> struct pick { using type = A; };
  template <typename A, typename B> struct pick<false, A, B> { using type = B; };
  using L = typename pick<LKS, KsOp<LU, BN>, KcOp<LU, LRow>>::type;
  using R = typename pick<RKS, KsOp<RU, BM>, KcOp<RU, PlainRow>>::type;

  // acc[i][j]: sub-tile row i, column j of this wave over blocks kb0 .. kb1 - 1 (one at
  // least); block kb is block kb % KB of segment kb / KB (at most two).
  __device__ static __forceinline__ void run(uint8_t* lds, L& lo, R& ro, int kb0, int kb1, int KB, int wave, int l,
                                             v4f (&acc)[NI][MJ]) {
    const int g = l >> 4, lr = l & 15, wn = wave / WM, wm = wave % WM;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < MJ; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
    lo.wave = ro.wave = wave;
    lo.l = ro.l = l;
    // The block that is loaded next, and the one at which more than its place changes: a
    // segment's last (k may end within it), its end, the end of all (from there on zeros).
    int at = kb0, event;
    const auto place = [&] {
      const bool none = at >= kb1;
      const int seg = at >= KB, k = seg ? at - KB : at;
      lo.place(k, seg, KB, none);
      ro.place(k, seg, KB, none);
      asm volatile("");   // a branch, not a row of selects in every block
      const int e = seg * KB + (k == KB - 1 ? KB : KB - 1);
      event = none ? 0x7fffffff : min(e, kb1);
    };
    const auto next = [&] {
      ++at;
      lo.next();
      ro.next();
      if (at == event) place();
    };
    place();
    uint32_t base = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(w4_lds_t*)lds + wave * 1024);
    const auto load_one = [&](auto nn, auto half) {
      constexpr int n = decltype(nn)::value, s = decltype(half)::value * BLOCK;
      if constexpr (n < LU) lo.template load<s + 8192 * n>(n, base);
      else ro.template load<s + L_BYTES + 8192 * (n - LU)>(n - LU, base);
    };
    // addresses within the block that is read from, of its first step (KC: of both)
    constexpr int LP = LKS ? NI / 2 : 2, RP = RKS ? MJ / 2 : 2;
    int la[LP], ra[RP];
    const int kr = 8 * g + (lr >> 2), a = lr & 3;   // KS: row of the first four k, group of 4 columns
    const int lds0 = (int)(uintptr_t)(w4_lds_t*)lds;
#pragma unroll
    for (int p = 0; p < LP; ++p)
      la[p] = lds0 + (LKS ? kr * (BN * 2) + (((wn * (NI / 2) + p) ^ KsOp<LU, BN>::swz(kr)) << 6) + 16 * a
                          : (wn * NI * 16 + lr) * 128 + (((4 * p + g) ^ swz8q(lr)) << 4));
#pragma unroll
    for (int p = 0; p < RP; ++p)
      ra[p] = lds0 + L_BYTES + (RKS ? kr * (BM * 2) + (((wm * (MJ / 2) + p) ^ KsOp<RU, BM>::swz(kr)) << 6) + 8 * a
                                    : (wm * MJ * 16 + lr) * 128 + (((4 * p + g) ^ swz8q(lr)) << 4));
    int flip = BLOCK;   // to the other block
    const auto turn = [&] {
#pragma unroll
      for (int p = 0; p < LP; ++p) la[p] += flip;
#pragma unroll
      for (int p = 0; p < RP; ++p) ra[p] += flip;
    };
    typedef __attribute__((address_space(3))) const uint8_t lds_u8;
    typedef __attribute__((address_space(3))) const v4i lds_v4i;
    const auto tr8 = [&](lds_u8* p, int row4) {   // four k and the four after them, row4 bytes on
      const uint2 x = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)p));
      const uint2 y = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + row4)));
      return (v4i){(int)x.x, (int)x.y, (int)y.x, (int)y.y};
    };
    // operands of step q of the block
    const auto read_l = [&](int q, int i) {
      if constexpr (LKS) return tr8((lds_u8*)(la[i >> 1] + q * (32 * BN * 2) + 8 * (i & 1)), 4 * BN * 2);
      else return *(lds_v4i*)(la[q] + i * 2048);
    };
    const auto read_r = [&](int q, int j) {
      if constexpr (RKS) return tr8((lds_u8*)(ra[j >> 1] + q * (32 * BM * 2) + 32 * (j & 1)), 4 * BM * 2);
      else return *(lds_v4i*)(ra[q] + j * 2048);
    };
    using T = std::true_type;
    using F = std::false_type;
    using Zero = std::integral_constant<int, 0>;
    using One = std::integral_constant<int, 1>;
    unroll<LOADS>([&](auto nn) { load_one(nn, Zero{}); });
    next();
    unroll<LOADS>([&](auto nn) { load_one(nn, One{}); });
    next();
    w4_wait<LOADS>();
    lds_barrier();
    v4i fl[NI], fr[2][MJ];
#pragma unroll
    for (int i = 0; i < NI; ++i) fl[i] = read_l(0, i);
#pragma unroll
    for (int j = 0; j < MJ; ++j) fr[0][j] = read_r(0, j);
    // Step q of a block; NEXT: another step follows, whose operands are read; LOAD: the
    // block after the next is loaded into this one's place.
    const auto step = [&](auto qq, auto load, auto nextp) {
      constexpr int q = decltype(qq)::value;
      constexpr bool LOAD = decltype(load)::value && q == 1, NEXT = decltype(nextp)::value;
      unroll<NI>([&](auto ii) {
        constexpr int i = decltype(ii)::value;
#pragma unroll
        for (int j = 0; j < MJ; ++j) acc[i][j] = w4_mfma(fl[i], fr[q][j], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);   // the read below takes the registers of fl[i]
        if constexpr (i == 0 && q == 1 && NEXT) {
          // own loads of the next block have landed; every wave has read all of this one
          w4_wait<0>();
          lds_barrier();
          turn();
        }
        if constexpr (NEXT) {
          fl[i] = read_l(q ^ 1, i);
#pragma unroll
          for (int j = i * MJ / NI; j < (i + 1) * MJ / NI; ++j) fr[q ^ 1][j] = read_r(q ^ 1, j);
        }
        if constexpr (LOAD) {
          unroll<LOADS>([&](auto nn) {
            constexpr int n = decltype(nn)::value;
            if constexpr (n >= i * LOADS / NI && n < (i + 1) * LOADS / NI) load_one(nn, Zero{});
          });
        }
        __builtin_amdgcn_sched_barrier(0);
      });
      if constexpr (LOAD) next();
      if constexpr (q == 1) {
        base += flip;
        flip = -flip;
      }
    };
    // two blocks at least, zeros behind the last
    for (int left = max(kb1 - kb0, 2); left > 2; --left) {
      step(Zero{}, T{}, T{});
      step(One{}, T{}, T{});
    }
    step(Zero{}, F{}, T{});
    step(One{}, F{}, T{});
    step(Zero{}, F{}, T{});
    step(One{}, F{}, F{});
  }
  template <int N, int I = 0, typename Fn>
  __device__ static __forceinline__ void unroll(Fn fn) {
    if constexpr (I < N) {
      fn(std::integral_constant<int, I>{});
      unroll<N, I + 1>(fn);
    }
  }
#endif  // SG_DEVICE_PASS
};

}  // namespace sg
