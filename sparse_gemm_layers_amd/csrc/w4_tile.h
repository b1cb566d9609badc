// Tile product of the 4-bit-weight kernels at many rows: 128 IW W rows x up to
// 128 X rows per workgroup of 8 waves.  A wave owns IW row blocks of 16 W rows
// ("slots" IW w ..) and every X row, so each code is widened by one wave alone:
// widening (13 instructions per 8 codes) is much of what a wave issues, one
// instruction in 8 cycles with two waves a SIMD.  2048 x 4096 x 4096: 59 to 61 us
// with groups of 128, 1.13 PFLOP/s at the 1.8 to 2.1 GHz that the card holds under this
// load, 66 with groups of 64, 76 of 32 (four sums to scale a block for one).  A 2 x 4
// grid of waves, which widens each code four times, took 83 us where this took 70.
// The price is that every wave reads every X row from LDS.
// IW = 1 is for products that leave compute units empty otherwise.
//
// A K block is one stage of a ring of three.  A wave's own codes and scales are
// loaded one K block ahead of X, so that they are widened while the block
// before is multiplied; X operands are read one pair of sub-tile columns ahead.
// The block's single barrier stands before its last pair, whose operands are in
// registers by then: it frees the block's stage for the loads of block kb + 3
// and opens that of kb + 1.
//
// Stage (bytes): X in two halves of 64 columns, 128 rows of 128 B each, the
// 16-byte piece c of row r at c ^ swz8q(r); the 8 IW slots' codes as packed, 1 KB
// each.  The slots' scales, 256 B each, have a ring of four of their own.
#pragma once

#include <type_traits>

#include "tile_epilogue.h"
#include "w4.h"

namespace sg {

template <int GC, int IW = 2>
struct W4Tile {
  using P = W4<GC>;
  static constexpr int BN = 128 * IW, BM = 128;
  static constexpr int W_OFF = BM * 256, STAGE = W_OFF + 8 * IW * W4_CODES;
  static constexpr int S_OFF = 3 * STAGE, S_STAGE = 8 * IW * 256;   // scales: a ring of four
  static constexpr int LDS = S_OFF + 4 * S_STAGE;
  static_assert(LDS <= 160 * 1024, "LDS");
  static constexpr int LOADS = 4 + 2 * IW;   // of one wave and stage

#if SG_DEVICE_PASS
  struct Src {
    const void *x, *w[IW];            // w: this wave's row blocks, each from its first chunk, KB chunks
    uint32_t x_bytes;                 // at most 2^31
    uint32_t xoff[2];                 // byte offset in x of this lane's rows, W4_OUT: not there
    int K, KB;
  };
  // The X rows that lane l loads, u = 0, 1.
  __device__ static __forceinline__ int x_row(int u, int wave, int l) { return 8 * (8 * u + wave) + (l >> 3); }


  // acc[i][j] (rows of slot IW wave + i, X rows 16 j + l % 16, in units of
  // W4_UNIT) over all K blocks, for the first 32 JP X rows.
  template <int JP>
  __device__ static __forceinline__ void multiply(uint8_t* lds, const Src& s, int wave, int l, v4f (&acc)[IW][8]) {
    const int g = l >> 4, lr = l & 15;
#pragma unroll
    for (int i = 0; i < IW; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
    int cur = 0, nxt = STAGE, far = 2 * STAGE;   // the stages of kb, kb + 1, kb + 2

    // Loads past the last K block read that block again, columns past K of it are
    // W4_OUT: the same few scalar instructions for every block (a wave issues one
    // instruction in 8 cycles, of whatever kind).
    const int c = 8 * ((l & 7) ^ swz8q(l >> 3));   // first column of this lane's piece; its rows mod 8 are l >> 3
    uint32_t xv[2][2], xlast[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        xv[u][h] = s.xoff[u] == W4_OUT ? W4_OUT : s.xoff[u] + 2 * (64 * h + c);
        xlast[u][h] = (s.KB - 1) * 128 + 64 * h + c < s.K ? xv[u][h] : W4_OUT;
      }
    const uint32_t cv = 16 * l, sv = l < 16 * P::NG ? (uint32_t)(W4_CODES + 4 * l) : W4_OUT;
    const uint32_t w_bytes = (uint32_t)(s.KB * P::CHUNK);
    const __amdgpu_buffer_rsrc_t rx = w4_rsrc(s.x, s.x_bytes), rw0 = w4_rsrc(s.w[0], w_bytes),
                                 rw1 = w4_rsrc(s.w[IW - 1], w_bytes);
    const auto load_codes = [&](int i, int stage, int kb) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(i ? rw1 : rw0,
                                               (w4_lds_t*)(lds + stage + W_OFF + (IW * wave + i) * W4_CODES), 16, cv,
                                               min(kb, s.KB - 1) * P::CHUNK, 0, 0);
    };
    // load group b: codes of b + 1, scales and X of b, one at a time
    const auto load_one = [&](int n, int codes, int x, int b) {
      if (n < IW) {
        load_codes(n, codes, b + 1);
      } else if (n < 2 * IW) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            n == 3 ? rw1 : rw0, (w4_lds_t*)(lds + S_OFF + (b & 3) * S_STAGE + (IW * wave + n - IW) * 256), 4, sv,
            min(b, s.KB - 1) * P::CHUNK, 0, 0);
      } else {
        const int u = (n - 2 * IW) >> 1, h = n & 1;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (w4_lds_t*)(lds + x + h * (BM * 128) + (8 * u + wave) * 1024), 16,
                                                 b >= s.KB - 1 ? xlast[u][h] : xv[u][h], min(b, s.KB - 1) * 256, 0, 0);
      }
    };
    const auto load = [&](int codes, int x, int b) {
#pragma unroll
      for (int n = 0; n < LOADS; ++n) load_one(n, codes, x, b);
    };
#pragma unroll
    for (int i = 0; i < IW; ++i) load_codes(i, cur, 0);
    load(nxt, cur, 0);
    load(far, nxt, 1);
    const int q0 = lr * 128 + ((g ^ swz8q(lr)) << 4), q1 = lr * 128 + (((4 + g) ^ swz8q(lr)) << 4);
    const int wo = W_OFF + IW * wave * W4_CODES + 16 * l, so = S_OFF + IW * wave * 256 + 16 * g;   // of this wave's slots
    // X operands of pair jj, columns 32 q .. 32 q + 31
    const auto read_x = [&](v4i (&bx)[2][4], int stage, int jj, int q) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
        bx[b][q] = *reinterpret_cast<const v4i*>(lds + stage + (q & 1 ? q1 : q0) + (q >> 1) * (BM * 128) +
                                                 (2 * jj + b) * 2048);
    };

    v4i aw[2][IW][4], bx[2][4], cw[IW];
    // Sums of the group in work and of the one before; the scales of the block's
    // groups, each read anew for the next block once its last sums are scaled.
    v4f p[2][IW][2], sw[P::NG][IW];
    const v4f zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < IW; ++i) {
      p[0][i][0] = p[0][i][1] = p[1][i][0] = p[1][i][1] = zero;
      sw[P::NG - 1][i] = zero;   // of the group before the first
    }
    const auto read_scales = [&](int u, int kb) {
#pragma unroll
      for (int i = 0; i < IW; ++i)
        sw[u][i] = *reinterpret_cast<const v4f*>(lds + so + (kb & 3) * S_STAGE + i * 256 + u * 64);
    };
    w4_wait<2 * LOADS>();
#pragma unroll
    for (int i = 0; i < IW; ++i) cw[i] = *reinterpret_cast<const v4i*>(lds + cur + wo + i * W4_CODES);
    lds_barrier();           // block 0's codes are in registers: block 3's may take their place
    load(cur, far, 2);
#pragma unroll
    for (int i = 0; i < IW; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) aw[0][i][q] = w4_widen(cw[i][q]);
    w4_wait<2 * LOADS>();
    lds_barrier();
#pragma unroll
    for (int q = 0; q < 4; ++q) read_x(bx, cur, 0, q);
#pragma unroll
    for (int u = 0; u < P::NG - 1; ++u) read_scales(u, 0);
#pragma unroll
    for (int i = 0; i < IW; ++i) cw[i] = *reinterpret_cast<const v4i*>(lds + nxt + wo + i * W4_CODES);

    // One K block: JP pairs of sub-tile columns, 8 IW matrix instructions each.
    // What else there is to do is spread between those by hand, and the order is
    // kept: the compiler's own left the matrix cores idle half of the time, both
    // waves of a SIMD widening or both multiplying.  After each matrix
    // instruction come, where due, the scaling of one 16 x 16 sum of the group
    // before, a part of the next block's widening, the operands of the next
    // pair in place of those just used, and a load of block kb + 3.
    // PA: which half of aw holds this block; PU: which of p its first group.
    const auto block = [&](int kb, auto pa, auto pu) {
      constexpr int PA = decltype(pa)::value, PU = decltype(pu)::value;
      constexpr int TS = 8 * IW, L = 2 * IW * P::QPG;   // matrix instructions per pair, per group
      constexpr int B = IW;                             // the one of the last pair that the barrier follows
      v4i ahead[IW];   // codes of kb + 2
      float half0 = 0.f, half1 = 0.f;
#pragma unroll
      for (int jj = 0; jj < JP; ++jj) {
#pragma unroll
        for (int t = 0; t < TS; ++t) {
          const int q = t / (2 * IW), i = (t >> 1) & (IW - 1), c = t & 1;
          const int u = jj * P::NG + t / L, in = t % L;   // group of the block, instruction of the group
          const int now = (PU + u) & 1, old = now ^ 1;
          const int oj = u == 0 ? JP - 1 : (u - 1) / P::NG;        // pair of the group before,
          const int og = (u + P::NG - 1) % P::NG;                  // its place among the block's groups
          // both X operands of these 32 columns: six reads at least were asked for after them
          if (t % (2 * IW) == 0) __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4) | (6 << 8));
          p[now][i][c] = w4_mfma(aw[PA][i][q], bx[c][q], in < 2 * IW ? zero : p[now][i][c]);
          if (in % P::QPG == P::QPG / 2) {
            const int k = in / P::QPG, ki = k >> 1, kc = k & 1;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[ki][2 * oj + kc][e] = fmaf(p[old][ki][kc][e], sw[og][ki][e], acc[ki][2 * oj + kc][e]);
          }
          if (in == L - 1 && oj == JP - 1) read_scales(og, u == 0 ? kb : kb + 1);
#pragma unroll
          for (int d = (jj * TS + t) * 2 / JP; d < (jj * TS + t + 1) * 2 / JP; ++d) {   // 4 of each row block and 32 columns
            // a pair's halves are joined a step later: right after the conversions a wait would come between
            if (d > 0) aw[PA ^ 1][((d - 1) >> 2) & (IW - 1)][(d - 1) / (4 * IW)][(d - 1) & 3] = w4_join(half0, half1);
            const int w = cw[(d >> 2) & (IW - 1)][d / (4 * IW)];
            half0 = (d & 3) == 0 ? w4_code<0>(w) : (d & 3) == 1 ? w4_code<1>(w) : (d & 3) == 2 ? w4_code<2>(w) : w4_code<3>(w);
            const uint32_t h = (uint32_t)w >> 4;
            half1 = (d & 3) == 0 ? w4_code<0>(h) : (d & 3) == 1 ? w4_code<1>(h) : (d & 3) == 2 ? w4_code<2>(h) : w4_code<3>(h);
          }
          if (jj == JP - 1) {
            if (t == B) {
              // own loads of kb + 1 have landed (kb + 2's may fly); every wave holds its last operands of kb
              w4_wait<LOADS>();
              lds_barrier();
            }
            if (t == (B + LOADS + 1 < TS ? B + LOADS + 1 : TS - 1)) {
#pragma unroll
              for (int k = 0; k < IW; ++k) ahead[k] = *reinterpret_cast<const v4i*>(lds + far + wo + k * W4_CODES);
            }
            if (t > B && t <= B + LOADS) load_one(t - B - 1, nxt, cur, kb + 3);   // block kb + 1's codes are in registers
          }
          if ((t + 1) % (2 * IW) == 0) {
            if (jj < JP - 1) read_x(bx, cur, jj + 1, q);
            else read_x(bx, nxt, 0, q);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      aw[PA ^ 1][IW - 1][3][3] = w4_join(half0, half1);
#pragma unroll
      for (int i = 0; i < IW; ++i) cw[i] = ahead[i];
      const int was = cur;
      cur = nxt;
      nxt = far;
      far = was;
    };
    using Z = std::integral_constant<int, 0>;
    using O = std::integral_constant<int, 1>;
    using S1 = std::integral_constant<int, (JP * P::NG) & 1>;   // an odd number of groups leaves p the other way round
    int kb = 0;
    for (; kb + 1 < s.KB; kb += 2) {
      block(kb, Z{}, Z{});
      block(kb + 1, O{}, S1{});
    }
    if (kb < s.KB) block(kb, Z{}, Z{});
    // the last group's sums; which of p holds them depends on the parity of all groups
    const bool odd = ((s.KB * JP * P::NG) & 1) != 0;
#pragma unroll
    for (int i = 0; i < IW; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[i][2 * JP - 2 + c][e] = fmaf(odd ? p[0][i][c][e] : p[1][i][c][e], sw[P::NG - 1][i][e],
                                           acc[i][2 * JP - 2 + c][e]);
    w4_wait<0>();   // loads past the end, of the last block again, have landed before LDS is given up
  }
#endif  // SG_DEVICE_PASS
};

}  // namespace sg
