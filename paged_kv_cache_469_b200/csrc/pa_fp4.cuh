// pa_fp4.cuh -- the 4-bit cache's tile layout and its number formats.
//
// A pool block holds, for one kv-head, the K and V of 16 tokens as one tile of
// 18 D bytes (2304 at D = 128, 1152 at D = 64), 4.5 bits a value:
//
//   K codes   [16 tokens][D / 2 bytes]        dim 2j in the low half of byte j
//   V codes   [2 h][8 c][4 t][2 i][D / 16]    token 4 t + 2 h + i, dims c D/8 ..
//   K scales  [16 tokens][D / 16]             one e4m3 byte per 16 dims
//   V scales  [D / 16][16 tokens]
//
// A code is e2m1 (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives); a value is
// code * scale * (the tensor's own fp32 scale).  code * scale has at most six
// significant bits and lies between 2^-10 and 2688, so it is exact in f16.
//
// Why this order: an MMA lane takes its K operand as 16 bytes of one token's
// row (the order of the dims within the product is free, the query is held in
// the same order).  Its V operand pairs two tokens of one dim in a register,
// four neighbouring tokens in all: with the two tokens of a pair 4 or 8 bytes
// apart, a warp reads both with one 16-byte access per lane and no bank
// conflict, and pairs them by half-byte selects before they are converted.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "pa_internal.cuh"

namespace pa {

template <int D>
struct Fp4Tile {
  static constexpr int kVecs = D / 8;             // 8-dim vectors of a row: one word of codes
  static constexpr int kGroups = D / 16;          // scales of a row
  static constexpr int k_off = 0;
  static constexpr int v_off = 8 * D;
  static constexpr int ks_off = 16 * D;
  static constexpr int vs_off = 17 * D;
  static constexpr int bytes = 18 * D;
  static constexpr int kChunkBytes = D / 16;      // of one token in a chunk of V codes
  // the word of codes of 8-dim vector `vec` of token `off`
  __host__ __device__ static constexpr int k_word(int off, int vec) {
    return k_off + off * (D / 2) + vec * 4;
  }
  __host__ __device__ static constexpr int v_word(int off, int vec) {
    return v_off +
           ((((off >> 1 & 1) * 8 + vec / (D / 64)) * 4 + (off >> 2)) * 2 + (off & 1)) *
               kChunkBytes +
           vec % (D / 64) * 4;
  }
  __host__ __device__ static constexpr int k_scale(int off, int g) {
    return ks_off + off * kGroups + g;
  }
  __host__ __device__ static constexpr int v_scale(int off, int g) {
    return vs_off + g * 16 + off;
  }
};

// the four bytes of a word, two codes each.  The word is taken apart into .b8
// registers: the conversion then selects its byte itself, where shifting and
// masking costs an instruction per byte on the pipe that converts (a loop of
// conversions and products: 168 against 81 cycles for 64 codes a lane).
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t w, __half2 (&d)[4]) {
  uint32_t r[4];
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] = *reinterpret_cast<__half2*>(&r[i]);
}
// two scales (the low byte first) as f16
__device__ __forceinline__ __half2 e4m3x2_to_half2(uint32_t two) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3));
}
__device__ __forceinline__ float e4m3_to_float(uint32_t byte) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
}

}  // namespace pa
