// Tile product of the 4-bit-weight kernels at many rows: BN W rows x BM X rows
// per workgroup of 8 waves in an NW (W) x MW (X) grid, each wave IW x JW
// sub-tiles of 16 x 16.  One 128-wide K block per LDS stage, two stages: the
// waves multiply stage kb while kb + 1 streams in by buffer loads that write
// LDS.  Stage layout (bytes): X, BM rows of 256 B whose 16-byte piece c lies at
// c ^ (row & 15), so that the 16 rows of an operand read hit different banks;
// the 8 row blocks' codes as packed, 1 KB each; their scales, 256 B each.  Slot
// s of the row blocks is sub-tile row s % IW of wave column s / IW.
#pragma once

#include "tile_epilogue.h"
#include "w4.h"

namespace sg {

template <int GC, int NW_, int MW_, int IW_, int JW_>
struct W4Tile {
  using P = W4<GC>;
  static constexpr int NW = NW_, MW = MW_, IW = IW_, JW = JW_;
  static_assert(NW * MW == 8, "8 waves");
  static constexpr int BN = NW * IW * 16, BM = MW * JW * 16;
  static_assert(BN == 128, "one W row block per wave and stage");
  static constexpr int W_OFF = BM * 256, S_OFF = W_OFF + 8 * W4_CODES, STAGE = S_OFF + 8 * 256;
  static_assert(2 * STAGE <= 160 * 1024, "LDS");
  static constexpr int XL = BM / 32;      // X loads per wave and stage: 4 rows each

#if SG_DEVICE_PASS
  // The X row that lane l's load i fills.
  __device__ static __forceinline__ int x_row(int i, int wave, int l) { return 4 * (8 * i + wave) + (l >> 4); }

  // rw: the row block that this wave loads (slot `wave` of the stage).  Its
  // scales take 64 NG of the 256 bytes that one load of 4 bytes a lane fills.
  __device__ static __forceinline__ void issue(uint8_t* st, __amdgpu_buffer_rsrc_t rx, __amdgpu_buffer_rsrc_t rw,
                                               const uint32_t (&xoff)[XL], int kb, int K, int wave, int l) {
    // rows 4 (8 i + wave) + (l >> 4): the same row mod 16 for every i
    const int c = (l & 15) ^ ((4 * wave + (l >> 4)) & 15);
    const bool in = kb * 128 + c * 8 < K;
#pragma unroll
    for (int i = 0; i < XL; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (w4_lds_t*)(st + (8 * i + wave) * 1024), 16,
                                               in && xoff[i] != W4_OUT ? xoff[i] + c * 16 : W4_OUT, kb * 256, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (w4_lds_t*)(st + W_OFF + wave * W4_CODES), 16, (uint32_t)(16 * l),
                                             kb * P::CHUNK, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (w4_lds_t*)(st + S_OFF + wave * 256), 4,
                                             l < 16 * P::NG ? (uint32_t)(W4_CODES + 4 * l) : W4_OUT, kb * P::CHUNK, 0,
                                             0);
  }

  __device__ static __forceinline__ void compute(const uint8_t* st, int wn, int wm, int l, v4f (&acc)[IW][JW]) {
    const int g = l >> 4, lr = l & 15;
    v4i aw[IW][4];
    v4f sw[IW][P::NG];
#pragma unroll
    for (int i = 0; i < IW; ++i) {
      const int rb = wn * IW + i;
      const v4i cw = *reinterpret_cast<const v4i*>(st + W_OFF + rb * W4_CODES + 16 * l);
#pragma unroll
      for (int q = 0; q < 4; ++q) aw[i][q] = w4_widen(cw[q]);
#pragma unroll
      for (int u = 0; u < P::NG; ++u)
        sw[i][u] = *reinterpret_cast<const v4f*>(st + S_OFF + rb * 256 + u * 64 + 16 * g);
    }
#pragma unroll
    for (int j = 0; j < JW; ++j) {
      v4i bx[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        bx[q] = *reinterpret_cast<const v4i*>(st + ((wm * JW + j) * 16 + lr) * 256 + (((4 * q + g) ^ lr) << 4));
#pragma unroll
      for (int i = 0; i < IW; ++i)
#pragma unroll
        for (int u = 0; u < P::NG; ++u) {
          v4f p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = u * P::QPG; q < (u + 1) * P::QPG; ++q) p = w4_mfma(aw[i][q], bx[q], p);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(p[e], sw[i][u][e], acc[i][j][e]);
        }
    }
  }

  // acc = the wave's sums (in units of W4_UNIT) over all K blocks.  xoff: byte
  // offset of each of the lane's X rows in rx, W4_OUT for a row that is not there.
  __device__ static __forceinline__ void multiply(uint8_t* lds, __amdgpu_buffer_rsrc_t rx, __amdgpu_buffer_rsrc_t rw,
                                                  const uint32_t (&xoff)[XL], int KB, int K, int wave, int l,
                                                  v4f (&acc)[IW][JW]) {
#pragma unroll
    for (int i = 0; i < IW; ++i)
#pragma unroll
      for (int j = 0; j < JW; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
    const int wn = wave % NW, wm = wave / NW;
    uint8_t* const s0 = lds;
    uint8_t* const s1 = lds + STAGE;
    issue(s0, rx, rw, xoff, 0, K, wave, l);
    wait_vmcnt<0>();
    __syncthreads();
    for (int kb = 0; kb < KB; kb += 2) {
      if (kb + 1 < KB) issue(s1, rx, rw, xoff, kb + 1, K, wave, l);
      compute(s0, wn, wm, l, acc);
      wait_vmcnt<0>();
      __syncthreads();
      if (kb + 1 < KB) {
        if (kb + 2 < KB) issue(s0, rx, rw, xoff, kb + 2, K, wave, l);
        compute(s1, wn, wm, l, acc);
        wait_vmcnt<0>();
        __syncthreads();
      }
    }
  }
#endif  // SG_DEVICE_PASS
};

}  // namespace sg
