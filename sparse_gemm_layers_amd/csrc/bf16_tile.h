// Tile product of two bf16 matrices: D[n, m] = sum_k L[n, k] R[m, k] with fp32
// sums, BN x BM per workgroup of 8 waves, each operand stored either with k along
// its rows ("KC": a row of the operand is contiguous in k) or across them ("KS":
// a row holds one k), so that a forward product, the gradient of its input and
// that of its weight all read the matrices as the caller has them.
//
// k goes by blocks of 64 (two steps of 32: one 16x16x32 matrix instruction per pair of
// sub-tiles), which buffer loads bring to LDS directly, SL of the left operand and
// SR of the right at a time.  A KC block holds 128-byte rows (16-byte piece c of row r
// at c ^ swz8q(r)), read 16 bytes a lane: with 64-byte rows every line came from L2
// twice.  A KS block holds 64 rows of one k each (64-byte piece c of row k at c ^ swz(k)),
// read with ds_read_b64_tr_b16, which hands each lane four k of one column.  (Three and
// two in the largest tile, which leave no LDS; more in those that few workgroups share out,
// where a block's way from memory is longer than its product.)
//
// LAG: a wave first takes a step's operands from LDS and asks for what comes blocks later,
// then multiplies; the second half of the 8 waves, one to a SIMD as those of the first, goes
// one phase behind: while one wave of a SIMD multiplies the other reads.  In the largest
// tiles both kept going at once, with operands read ahead, is no faster (2048 x 14336 x
// 4096 forward 400 us for 383), and one wave a SIMD with 128 x 128 results of its own, which
// reads a third less from LDS, has its sums moved about by the compiler (690).
// Without LAG a wave takes a whole block's operands at once and there is one barrier a block: better where
// products are short (40 x 1000 x 8000 in tiles of 64 28 us for 38, 128 x 11008 x 4096 in tiles of 128 with the
// weights in the cache 34 for 38), no better with 256 (256 x 11008 x 4096 65 for 63: here and below one launch
// after another from a graph, other weights each time where not said).
// What bounds a block is LDS: a KB written by a load or read costs it 8 cycles (measured), so 128 x
// 128 takes 1024 cycles (0.45 us a block), 128 x 256 1408 (0.60), 256 x 256 2048, as its products do.
// What is left in the largest: the card's power.  It holds 1.75 to 1.9 GHz under this load, with the
// matrix cores busy in 70% of the cycles of a full round; without the loads it is 80% at
// 2.05 GHz, and a product of the library's with nothing fused runs at 1.78 GHz.
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
template <int NW>
struct PlainRow {
  static constexpr int MATS = 1;
#if SG_DEVICE_PASS
  __device__ static __forceinline__ int row(int u, int wave, int l) { return 8 * (NW * u + wave) + (l >> 3); }
  __device__ static constexpr int sel(int) { return 0; }
  __device__ static constexpr int sel_wave(int) { return 0; }
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

// One wave's loads of a KC operand: U instructions of 8 rows a block, NW waves.  The sum over k
// has one segment or two of KB blocks, each with a matrix of its own; p[seg] is the
// first column of row 0.  Row::row(u, wave, l) is the row that lane l of instruction u
// loads; Row::sel(u) ^ Row::sel_wave(wave) which of the two matrices it is of, where it
// is not the segment that says so.  Rows past the last lie outside of the descriptor (it ends
// with the last row) and read as zero.
template <int U, int NW, typename Row>
struct KcOp {
  const uint16_t* p[2];
  int64_t ld[2];
  uint32_t bytes[2];
  int K, wave, l;
  v4i r[Row::MATS];     // where the next block's loads are
  uint32_t cur[U];
  int soff, step;
  // Block k of segment seg is next; none: nothing but zeros is.
  __device__ __forceinline__ void place(int k, int seg, int KB, bool none) {
    // an empty descriptor takes no scalar offset, nor do those after it: the range check
    // subtracts that from its size
    soff = none ? 0 : k * 128;
    step = none ? 0 : 128;
    const int c = 8 * ((l & 7) ^ swz8q(l >> 3));   // k of this lane's piece of 16 bytes
    const bool out = k * 64 + c >= K;
#pragma unroll
    for (int m = 0; m < Row::MATS; ++m) {
      const int s = m ^ seg ^ Row::sel_wave(wave);
      r[m] = tile_rsrc(s ? p[1] : p[0], none ? 0u : s ? bytes[1] : bytes[0]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = Row::sel(u) ^ seg ^ Row::sel_wave(wave);
      cur[u] = out ? W4_OUT : (uint32_t)((Row::row(u, wave, l) * (s ? ld[1] : ld[0]) + c) * 2);
    }
  }
  template <int N, int AT>
  __device__ __forceinline__ void load(uint32_t base) const { lds_dma16<AT>(r[Row::sel(N)], cur[N], soff, base); }
  __device__ __forceinline__ void next() { soff += step; }
};

// One wave's loads of a KS operand of B columns.  p[seg], ld[seg]: row k = 0, the
// tile's first column.  Rows past K are outside of the descriptor and read as zero.
template <int U, int NW, int B>
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
      const int row = RPI * (NW * u + wave) + l / (B / 8);   // 16-byte piece l % (B / 8) of this row
      cur[u] = (uint32_t)(row * d * 2) + 16 * ((l % (B / 8)) ^ (swz(row) << 2));
    }
  }
  template <int N, int AT>
  __device__ __forceinline__ void load(uint32_t base) const { lds_dma16<AT>(r, cur[N], 0, base); }
  __device__ __forceinline__ void next() {
    const uint64_t at = (((uint64_t)(uint32_t)r[1] << 32) | (uint32_t)r[0]) + step;
    r[0] = (int)at;
    r[1] = (int)(at >> 32);
  }
};
#endif  // SG_DEVICE_PASS

// WN x WM waves of NI x MJ sub-tiles each; SL and SR places for blocks of the operands (a wait
// counts loads in their order: one operand further ahead than the other by two would gain nothing.
// With each operand loaded by half of the waves, the weights four to seven blocks ahead: 128 x 11008 x
// 4096 53 us for 52, 256 tokens 67 for 62).
// LRow: the left operand's rows, where it is KC.
template <bool LKS_, bool RKS_, bool LAG_, int WN_, int WM_, int NI_, int MJ_, int SL_, int SR_, typename LRow = void>
struct Bf16Tile {
  static constexpr bool LKS = LKS_, RKS = RKS_;
  static constexpr int WN = WN_, WM = WM_, NI = NI_, MJ = MJ_, NW = WN * WM;
  static constexpr bool LAG = LAG_;
  static constexpr int SL = SL_, SR = SR_;
  static_assert(NI % 2 == 0 && (!RKS || MJ % 2 == 0) && SR >= 2 && (SL == SR || SL == SR + 1), "pairs of sub-tiles, places");
  static constexpr int BN = WN * NI * 16, BM = WM * MJ * 16;
  static constexpr int L_BLOCK = BN * 128, R_BLOCK = BM * 128, R_OFF = SL * L_BLOCK, LDS = R_OFF + SR * R_BLOCK;
  static constexpr int LU = BN / 8 / NW, RU = BM / 8 / NW;   // loads of one wave and block
  static_assert(LDS <= 160 * 1024, "LDS");
#if SG_DEVICE_PASS
  template <bool C, typename A, typename B> struct pick { using type = A; };
  template <typename A, typename B> struct pick<false, A, B> { using type = B; };
  using L = typename pick<LKS, KsOp<LU, NW, BN>, KcOp<LU, NW, LRow>>::type;
  using R = typename pick<RKS, KsOp<RU, NW, BM>, KcOp<RU, NW, PlainRow<NW>>>::type;

  // The block of one operand that is loaded next, and the one at which more than its place
  // changes: a segment's last (k may end within it), its end, the end of all (from there on zeros).
  template <typename Op>
  struct Feed {
    Op& op;
    int at, event, kb1, KB;
    __device__ __forceinline__ void place() {
      const bool none = at >= kb1;
      const int seg = at >= KB, k = seg ? at - KB : at;
      op.place(k, seg, KB, none);
      asm volatile("");   // a branch, not a row of selects in every block
      const int e = seg * KB + (k == KB - 1 ? KB : KB - 1);
      event = none ? 0x7fffffff : min(e, kb1);
    }
    __device__ __forceinline__ void next() {
      ++at;
      op.next();
      if (at == event) place();
    }
  };

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
    Feed<L> fl_ = {lo, kb0, 0, kb1, KB};
    Feed<R> fr_ = {ro, kb0, 0, kb1, KB};
    fl_.place();
    fr_.place();
    const int lds0 = (int)(uintptr_t)(w4_lds_t*)lds;
    const uint32_t lbase = __builtin_amdgcn_readfirstlane(lds0 + wave * 1024), rbase = lbase + R_OFF;
    // addresses within a block, of its first step (KC: of both)
    constexpr int LP = LKS ? NI / 2 : 2, RP = RKS ? MJ / 2 : 2;
    int la[LP], ra[RP], lat[LP], rat[RP];   // lat, rat: within the block that is read from
    const int kr = 8 * g + (lr >> 2), a = lr & 3;   // KS: row of the first four k, group of 4 columns
#pragma unroll
    for (int p = 0; p < LP; ++p)
      la[p] = lat[p] = lds0 + (LKS ? kr * (BN * 2) + (((wn * (NI / 2) + p) ^ KsOp<LU, NW, BN>::swz(kr)) << 6) + 16 * a
                                   : (wn * NI * 16 + lr) * 128 + (((4 * p + g) ^ swz8q(lr)) << 4));
#pragma unroll
    for (int p = 0; p < RP; ++p)
      ra[p] = rat[p] = lds0 + R_OFF + (RKS ? kr * (BM * 2) + (((wm * (MJ / 2) + p) ^ KsOp<RU, NW, BM>::swz(kr)) << 6) + 8 * a
                                  : (wm * MJ * 16 + lr) * 128 + (((4 * p + g) ^ swz8q(lr)) << 4));
    typedef __attribute__((address_space(3))) const uint8_t lds_u8;
    typedef __attribute__((address_space(3))) const v4i lds_v4i;
    const auto tr8 = [&](lds_u8* p, int row4) {   // four k and the four after them, row4 bytes on
      const uint2 x = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)p));
      const uint2 y = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + row4)));
      return (v4i){(int)x.x, (int)x.y, (int)y.x, (int)y.y};
    };
    // operands of step q of the block
    const auto read_l = [&](int q, int i) {
      if constexpr (LKS) return tr8((lds_u8*)(lat[i >> 1] + q * (32 * BN * 2) + 8 * (i & 1)), 4 * BN * 2);
      else return *(lds_v4i*)(lat[q] + i * 2048);
    };
    const auto read_r = [&](int q, int j) {
      if constexpr (RKS) return tr8((lds_u8*)(rat[j >> 1] + q * (32 * BM * 2) + 32 * (j & 1)), 4 * BM * 2);
      else return *(lds_v4i*)(rat[q] + j * 2048);
    };
    // Loads that may be in flight when a block's have landed: of the blocks after it.
    constexpr int FLY = (SL - 2) * LU + (SR - 2) * RU;
    unroll<(SL > SR ? SL : SR) - 1>([&](auto c) {
      if constexpr (c < SL - 1) {
        unroll<LU>([&](auto n) { lo.template load<n, c * L_BLOCK + 1024 * NW * n>(lbase); });
        fl_.next();
      }
      if constexpr (c < SR - 1) {
        unroll<RU>([&](auto n) { ro.template load<n, c * R_BLOCK + 1024 * NW * n>(rbase); });
        fr_.next();
      }
    });
    w4_wait<FLY>();
    lds_barrier();
    if (LAG && wave >= NW / 2) lds_barrier();   // from here on a phase behind
    v4i fl[NI], fr[MJ];
    int lread = 0, rread = 0, lfill = (SL - 1) * L_BLOCK, rfill = (SR - 1) * R_BLOCK;   // places in the rings
    // Block c + SR - 1 of the right operand, c + SL - 1 of the left one, zeros past the end,
    // into the places of block c - 1; then on to block c + 1.
    const auto fill_r = [&]() {
      const uint32_t to = rbase + rfill;
      unroll<RU>([&](auto n) { ro.template load<n, 1024 * NW * n>(to); });
      fr_.next();
      rfill = rfill == (SR - 1) * R_BLOCK ? 0 : rfill + R_BLOCK;
    };
    const auto fill_l = [&]() {
      const uint32_t to = lbase + lfill;
      unroll<LU>([&](auto n) { lo.template load<n, 1024 * NW * n>(to); });
      fl_.next();
      lfill = lfill == (SL - 1) * L_BLOCK ? 0 : lfill + L_BLOCK;
      lread = lread == (SL - 1) * L_BLOCK ? 0 : lread + L_BLOCK;
      rread = rread == (SR - 1) * R_BLOCK ? 0 : rread + R_BLOCK;
#pragma unroll
      for (int p = 0; p < LP; ++p) lat[p] = la[p] + lread;
#pragma unroll
      for (int p = 0; p < RP; ++p) rat[p] = ra[p] + rread;
    };
    // Step q of block c: its operands from LDS; then the right operand of block c + SR - 1
    // (q = 0) or the left one of block c + SL - 1 (q = 1), zeros past the end, is asked for.
    const auto step = [&](auto qq) {
      constexpr int q = decltype(qq)::value;
#pragma unroll
      for (int j = 0; j < MJ; ++j) fr[j] = read_r(q, j);
#pragma unroll
      for (int i = 0; i < NI; ++i) fl[i] = read_l(q, i);
      if constexpr (q == 0) {
        fill_r();
      } else {
        fill_l();
        w4_wait<FLY>();   // own loads of the next block have landed
      }
      lds_barrier();
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < MJ; ++j) acc[i][j] = w4_mfma(fl[i], fr[j], acc[i][j]);
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_sched_barrier(0);
      lds_barrier();
      __builtin_amdgcn_sched_barrier(0);
    };
    if constexpr (LAG) {
      for (int left = kb1 - kb0; left > 0; --left) {
        step(std::integral_constant<int, 0>{});
        step(std::integral_constant<int, 1>{});
      }
    } else {
      for (int left = kb1 - kb0; left > 0; --left) {
        v4i l2[2][NI], r2[2][MJ];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
#pragma unroll
          for (int j = 0; j < MJ; ++j) r2[q][j] = read_r(q, j);
#pragma unroll
          for (int i = 0; i < NI; ++i) l2[q][i] = read_l(q, i);
        }
        fill_r();
        fill_l();
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < MJ; ++j) acc[i][j] = w4_mfma(l2[q][i], r2[q][j], acc[i][j]);
        w4_wait<FLY>();   // own loads of the next block have landed
        lds_barrier();
      }
    }
    if (LAG && wave < NW / 2) lds_barrier();   // of the others' last phase
    w4_wait<0>();   // the zeros past the end too, before LDS is given up
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
