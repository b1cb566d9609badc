// Dense 4-bit weights with group scales: packed layout, widening to bf16 and
// the operand loads shared by the linear and the routed kernels.
//
// Packed layout of an N x K weight with one fp32 scale per row and group of GC
// (32, 64 or 128) columns: one chunk per block of 16 rows and 128 columns, a
// row block's chunks one after the other along K.  A chunk holds the codes as
// the matrix core reads them, 16 bytes per lane: lane 16 g + r's dword q holds
// row r's columns 32 q + 8 g .. + 7 (element 2 j in the low half of byte j), so
// four v_mfma_f32_16x16x32_bf16 take a lane's 16 bytes as they were loaded.
// The scales follow, [group][row].  Rows past N and columns past K are zero.
#pragma once

#include "gemm_common.h"

namespace sg {

typedef __bf16 w4_bf8 __attribute__((ext_vector_type(8)));

constexpr int W4_CODES = 1024, W4_WAVES = 8;
template <int GC>
struct W4 {
  static constexpr int NG = 128 / GC;              // groups per chunk
  static constexpr int CHUNK = W4_CODES + 64 * NG;
  static constexpr int QPG = 4 / NG;               // matrix instructions per group
};
__host__ __device__ inline int w4_chunk(int gc) { return W4_CODES + 64 * (128 / gc); }

// Widened codes are c / 16 (v_cvt_off_f32_i4 gives sixteenths); finished sums
// are multiplied by this, which is exact.
constexpr float W4_UNIT = 16.0f;

#if SG_DEVICE_PASS
typedef __attribute__((address_space(3))) void w4_lds_t;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t w4_rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ v4i w4_ld16(__amdgpu_buffer_rsrc_t r, uint32_t off, int soff) {
  return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, off, soff, 0));
}

// The signed code in the low half of byte B of w, in sixteenths.
template <int B>
__device__ __forceinline__ float w4_code(uint32_t w) {
  float f;
  if constexpr (B == 0)
    asm("v_cvt_off_f32_i4_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_0" : "=v"(f) : "v"(w));
  else if constexpr (B == 1)
    asm("v_cvt_off_f32_i4_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_1" : "=v"(f) : "v"(w));
  else if constexpr (B == 2)
    asm("v_cvt_off_f32_i4_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_2" : "=v"(f) : "v"(w));
  else
    asm("v_cvt_off_f32_i4_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_3" : "=v"(f) : "v"(w));
  return f;
}

// Eight codes -> eight bf16 (exact: a sixteenth of a 4-bit integer has at most
// three significant bits), 13 instructions: 8 conversions that pick their byte,
// one shift for the odd codes, 4 joins of two high halves.  w4_pair<B> is the
// B-th pair.
__device__ __forceinline__ int w4_join(float even, float odd) {
  return (int)__builtin_amdgcn_perm(__float_as_uint(odd), __float_as_uint(even), 0x07060302u);
}
template <int B>
__device__ __forceinline__ int w4_pair(int code) {
  return w4_join(w4_code<B>((uint32_t)code), w4_code<B>((uint32_t)code >> 4));
}
__device__ __forceinline__ v4i w4_widen(int code) {
  return (v4i){w4_pair<0>(code), w4_pair<1>(code), w4_pair<2>(code), w4_pair<3>(code)};
}

__device__ __forceinline__ v4f w4_mfma(const v4i& a, const v4i& b, const v4f& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(w4_bf8, a), __builtin_bit_cast(w4_bf8, b), c, 0,
                                                 0, 0);
}

// Waits until at most N of this wave's loads are in flight.  Nothing that touches
// memory moves across it, nor across w4_pin: waits that count loads need them in
// the order they are written in.
template <int N>
__device__ __forceinline__ void w4_wait() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void w4_pin() { asm volatile("" ::: "memory"); }

// Past every descriptor's records (all hold under 2^31 bytes): such a lane reads zero.
constexpr uint32_t W4_OUT = 0x80000000u;
#endif  // SG_DEVICE_PASS

}  // namespace sg
