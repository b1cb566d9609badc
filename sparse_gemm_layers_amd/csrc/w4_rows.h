// Product of the 4-bit-weight kernels at few rows: one wave takes RB blocks of
// 16 W rows and up to 4 XI X rows over every step-th K block, without a barrier.
//
// What bounds it is how many loads a compute unit takes, about 16 cycles for one
// of 16 bytes a lane whether it brings 1 KB or nothing.  An X operand loaded as
// the matrix core wants it (lane 16 g + r: row r) takes 64, since neighbouring
// lanes then read different rows; so X rows come whole, four per load, into
// this wave's part of LDS and are read from there: 37 x 4096 x 14336 took 46 us
// with operands loaded directly and takes 16.  Scales take one load of 4 bytes a
// lane per row block (7 cycles), codes one of 16 (a packed chunk's 1 KB).
// Codes, which come from HBM, are loaded DW K blocks ahead, X rows, which L2
// holds, DX.
#pragma once

#include "w4.h"

namespace sg {

template <int GC, int RB, int XI, int DX_ = XI <= 2 ? 4 : XI <= 4 ? 2 : 1, int DW_ = DX_ == 1 ? 2 : 4>
struct W4Rows {
  using P = W4<GC>;
  static constexpr int MT = (XI + 3) / 4;                        // sub-tiles of 16 X rows
  static constexpr int DX = DX_, DW = DW_;                       // K blocks ahead: X; codes and scales
  static_assert(DW % DX == 0 && DX <= DW, "a block's slot in either ring follows from its place in DW");
  static constexpr int S_OFF = DX * XI * 1024;
  static constexpr int WAVE_LDS = S_OFF + DW * RB * 256;
  static constexpr int RED = W4_WAVES * RB * MT * 1024;          // the waves' partial tiles, in the same place later
  static constexpr int LDS = W4_WAVES * WAVE_LDS > RED ? W4_WAVES * WAVE_LDS : RED;
  static_assert(LDS <= 160 * 1024, "LDS");
#if SG_DEVICE_PASS
  struct Src {
    const void *x, *w[RB];             // w: each row block from its first chunk, KB chunks
    uint32_t x_bytes;                  // at most 2^31
    uint32_t xoff[XI];                 // byte offset in x of row 4 i + l / 16, W4_OUT: not there
    int K, KB;
  };

  // Loads into LDS are not ordered against this wave's LDS reads: a slot is refilled
  // once its reads are done (reads_done).  EARLY: right after the X operands have come,
  // the first row block's codes being widened meanwhile, and the multiplication follows;
  // otherwise after it.  Early / late, us: 24 x 4096 x 4096, groups of 32, 5.9 / 6.3; 33 x
  // 4096 x 4096 6.6 / 7.1; 41 x 4143 x 4096, groups of 32, 9.0 / 11.9 (late spills); but 4 x
  // 4096 x 14336 8.7 / 8.5, one token of the routed MLP 22.4 / 18.6, and with RB 4, XI 16,
  // which spills early, 256 x 4096 x 4096 18.2 / 15.6.
  static constexpr bool EARLY = XI >= 4 && !(RB == 4 && XI == 16);
  __device__ static __forceinline__ void reads_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

  // acc[rb][j] += rows of block rb times X rows 16 j + l % 16 (in units of
  // W4_UNIT) over K blocks first, first + step, ...  Columns of X rows that are
  // not there hold anything.  lds: this wave's WAVE_LDS bytes.
  __device__ static __forceinline__ void multiply(uint8_t* lds, const Src& s, int first, int step, int l,
                                                  v4f (&acc)[RB][MT]) {
    const int g = l >> 4, lr = l & 15;
    v4i cw[DW][RB];
    uint32_t xv[XI], xlast[XI];
    // row r's 16-byte piece c lies at c ^ (r & 15)
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const int c = lr ^ ((4 * i + g) & 15);
      xv[i] = s.xoff[i] == W4_OUT ? W4_OUT : s.xoff[i] + 16 * c;
      xlast[i] = (s.KB - 1) * 128 + 8 * c < s.K ? xv[i] : W4_OUT;
    }
    const uint32_t sv = l < 16 * P::NG ? (uint32_t)(W4_CODES + 4 * l) : W4_OUT;
    const auto load_x = [&](int slot, int kb) {
      const bool last = kb == s.KB - 1;
#pragma unroll
      for (int i = 0; i < XI; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(w4_rsrc(s.x, s.x_bytes), (w4_lds_t*)(lds + (slot * XI + i) * 1024),
                                                 16, last ? xlast[i] : xv[i], kb * 256, 0, 0);
      w4_pin();
    };
    const auto load_w = [&](int slot, int kb) {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        const __amdgpu_buffer_rsrc_t rw = w4_rsrc(s.w[rb], (uint32_t)(s.KB * P::CHUNK));
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (w4_lds_t*)(lds + S_OFF + (slot * RB + rb) * 256), 4, sv,
                                                 kb * P::CHUNK, 0, 0);
        cw[slot][rb] = w4_ld16(rw, (uint32_t)(16 * l), kb * P::CHUNK);
      }
      w4_pin();
    };
    // X operands are read once, a row block's codes widened and its scales read once.
    // refill: the loads into this X slot, once it has been read.
    const auto compute = [&](int n, auto refill) {
      v4i bx[MT][4];
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          // lanes past the last row that is kept read rows that are
          const int r = XI < 4 ? lr & (4 * XI - 1) : min(16 * j + lr, 4 * XI - 1);
          bx[j][q] = *reinterpret_cast<const v4i*>(lds + (n % DX) * XI * 1024 + r * 256 +
                                                   (((4 * q + g) ^ (r & 15)) << 4));
        }
      v4i aw[4];
      if (EARLY) {
#pragma unroll
        for (int q = 0; q < 4; ++q) aw[q] = w4_widen(cw[n][0][q]);
        __builtin_amdgcn_sched_barrier(0);
        reads_done();
        refill();
      }
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        v4f sw[P::NG];
        if (rb > 0 || !EARLY) {
#pragma unroll
          for (int q = 0; q < 4; ++q) aw[q] = w4_widen(cw[n][rb][q]);
        }
#pragma unroll
        for (int t = 0; t < P::NG; ++t)
          sw[t] = *reinterpret_cast<const v4f*>(lds + S_OFF + (n * RB + rb) * 256 + t * 64 + 16 * g);
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int t = 0; t < P::NG; ++t) {
            v4f p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = t * P::QPG; q < (t + 1) * P::QPG; ++q) p = w4_mfma(aw[q], bx[j][q], p);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[rb][j][e] = fmaf(p[e], sw[t][e], acc[rb][j][e]);
          }
      }
    };
    // Loads that may be in flight when X of block n, and all that was asked for
    // before it, has landed, given that the DW - 1 blocks after n have been asked for.
    constexpr int FLY = DX == DW ? (DX - 1) * (XI + 2 * RB) : (DX - 1) * XI + DX * 2 * RB;
#pragma unroll
    for (int n = -DW; n < 0; ++n) {
      if (n + DX >= 0 && first + (n + DX) * step < s.KB) load_x(n + DX, first + (n + DX) * step);
      if (first + (n + DW) * step < s.KB) load_w(n + DW, first + (n + DW) * step);
    }
    int kb = first;
    for (; kb + (2 * DW - 1) * step < s.KB; kb += DW * step) {
#pragma unroll
      for (int n = 0; n < DW; ++n) {
        w4_wait<FLY>();
        const auto refill = [&] { load_x(n % DX, kb + (n + DX) * step); };   // DX divides DW
        compute(n, refill);
        reads_done();
        if (!EARLY) refill();
        load_w(n, kb + (n + DW) * step);
      }
    }
    // The last 2 DW - 1 blocks at most, apart: a load past the end would cost as much as any other.
#pragma unroll
    for (int n = 0; n < 2 * DW - 1; ++n, kb += step) {
      if (kb >= s.KB) break;
      if (kb + (DW - 1) * step < s.KB) w4_wait<FLY>();
      else w4_wait<0>();
      const auto refill = [&] {
        if (kb + DX * step < s.KB) load_x(n % DX, kb + DX * step);
      };
      compute(n % DW, refill);
      // finished here: the compiler would carry unscaled sums into the branches that follow, and spill them
#pragma unroll
      for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int j = 0; j < MT; ++j) asm volatile("" : "+v"(acc[rb][j]));
      reads_done();
      if (!EARLY) refill();
      if (n < DW - 1 && kb + DW * step < s.KB) load_w(n, kb + DW * step);
    }
    w4_wait<0>();
  }
#endif  // SG_DEVICE_PASS
};

// Many row blocks against the same few X rows: these lie in LDS for the whole of
// K, and each wave streams whole row blocks past them, one after the other,
// without a barrier, a join or a gap between blocks.
template <int GC>
struct W4Stream {
  using P = W4<GC>;
  static constexpr int DW = 4;   // K blocks ahead
#if SG_DEVICE_PASS
  // X rows in LDS: K block kb's R rows (4, 8 or 16) of 256 B at kb * R * 256,
  // row r's 16-byte piece c at c ^ r.  Loads them, 4 rows a load: K blocks wave,
  // wave + 8, ...; off(r): byte offset of row r in x, W4_OUT: not there (zeros).
  template <typename Off>
  __device__ static __forceinline__ void load_x(uint8_t* lds, const void* x, uint32_t x_bytes, int K, int R, int n,
                                                int wave, int l, Off off) {
    const int KB = (K + 127) >> 7;
    const __amdgpu_buffer_rsrc_t rx = w4_rsrc(x, x_bytes);
    for (int i = 0; i < R / 4; ++i) {
      const int r = 4 * i + (l >> 4), c = (l & 15) ^ r;
      const uint32_t o = r < n ? off(r) : W4_OUT;
      for (int kb = wave; kb < KB; kb += W4_WAVES)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (w4_lds_t*)(lds + (kb * R + 4 * i) * 256), 16,
                                                 o != W4_OUT && kb * 128 + 8 * c < K ? o + kb * 256 + 16 * c : W4_OUT,
                                                 0, 0, 0);
    }
  }

  // Row blocks 0 .. units - 1 of this wave: base(u) is block u's first chunk; done(u, acc) takes its
  // sums (in units of W4_UNIT): rows 4 g .. 4 g + 3 against X row l % 16 (repeating after R).
  template <typename Base, typename Done>
  __device__ static __forceinline__ void run(const uint8_t* lds, int KB, int R, int units, int l, Base base,
                                             Done done) {
    const int g = l >> 4, r0 = l & (R - 1);
    v4i cw[DW];
    v4f sw[DW][P::NG];
    int pu = 0, pkb = 0;   // what is asked for next
    const uint8_t* pw = base(0);
    const auto load = [&](int n) {
      const __amdgpu_buffer_rsrc_t rw = w4_rsrc(pw, pu < units ? (uint32_t)(KB * P::CHUNK) : 0u);
      const int at = pu < units ? pkb * P::CHUNK : 0;
      cw[n] = w4_ld16(rw, (uint32_t)(16 * l), at);
#pragma unroll
      for (int t = 0; t < P::NG; ++t)
        sw[n][t] = __builtin_bit_cast(v4f, w4_ld16(rw, (uint32_t)(W4_CODES + 64 * t + 16 * g), at));
      if (++pkb == KB) {
        pkb = 0;
        ++pu;
        pw = base(pu < units ? pu : 0);
      }
    };
#pragma unroll
    for (int n = 0; n < DW; ++n) load(n);
    v4f acc = {0.f, 0.f, 0.f, 0.f};
    int u = 0, kb = 0;
    while (u < units) {
#pragma unroll
      for (int n = 0; n < DW; ++n) {
        v4i aw[4], bx[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          aw[q] = w4_widen(cw[n][q]);
          bx[q] = *reinterpret_cast<const v4i*>(lds + (kb * R + r0) * 256 + (((4 * q + g) ^ r0) << 4));
        }
#pragma unroll
        for (int t = 0; t < P::NG; ++t) {
          v4f p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = t * P::QPG; q < (t + 1) * P::QPG; ++q) p = w4_mfma(aw[q], bx[q], p);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] = fmaf(p[e], sw[n][t][e], acc[e]);
        }
        load(n);
        if (++kb == KB) {
          kb = 0;
          if (u < units) done(u, acc);
          ++u;
          acc = (v4f){0.f, 0.f, 0.f, 0.f};
        }
      }
    }
  }
#endif  // SG_DEVICE_PASS
};

}  // namespace sg
