// The paged 4-bit KV cache's numbers and byte order, shared by the kernels
// that write and read it.
//
// A record holds 16 positions of one kv head: K codes, K scales, V codes, V
// scales (8, 1, 8 and 1 bytes per element of head_dim).  Codes are in the order
// of the m16n8k16 tensor-core operand A: a warp that loads 16 bytes per lane
// has, for four 16-element scale blocks, the fragments of
//   K:   rows = the 16 positions, contraction = 16 elements of the head, lane
//        (g, t) holding elements 4t .. 4t+3 of positions g and g + 8;
//   V^T: rows = 16 elements of the head (2g and 2g + 1 in lane g), contraction
//        = the 16 positions, lane (g, t) holding positions 2t, 2t+1, 2t+8, 2t+9.
#pragma once

#include <cuda_fp16.h>

#include "g4_device.cuh"

namespace g4 {

constexpr int kKv4Group = 16;  // positions per record

template <int HD>
struct Kv4Rec {
  static constexpr int KC = 0;            // K codes
  static constexpr int KS = 8 * HD;       // K scales
  static constexpr int VC = 9 * HD;       // V codes
  static constexpr int VS = 17 * HD;      // V scales
  static constexpr int BYTES = 18 * HD;
  static constexpr int NP = HD / 64;      // 64-element pieces of a row
};

// Byte offsets in a record of element d (even) of position m, and of the scale of its 16.
template <int HD>
__device__ __forceinline__ int kv4_k_code_at(int m, int d) {
  return Kv4Rec<HD>::KC + (d >> 6) * 512 + ((m & 7) * 4 + ((d >> 2) & 3)) * 16 + (m >> 3) * 8 + ((d >> 4) & 3) * 2 +
         ((d >> 1) & 1);
}
template <int HD>
__device__ __forceinline__ int kv4_k_scale_at(int m, int d) {
  return Kv4Rec<HD>::KS + (d >> 6) * 64 + (m & 7) * 8 + ((d >> 4) & 3) * 2 + (m >> 3);
}
template <int HD>
__device__ __forceinline__ int kv4_v_code_at(int m, int d) {
  const int t = (m >> 1) & 3, i = (m >> 3) * 2 + (m & 1);
  return Kv4Rec<HD>::VC + (d >> 6) * 512 + (((d >> 1) & 7) * 4 + t) * 16 + i * 4 + ((d >> 4) & 3);
}
template <int HD>
__device__ __forceinline__ int kv4_v_scale_at(int m, int d) {
  const int t = (m >> 1) & 3, i = (m >> 3) * 2 + (m & 1);
  return Kv4Rec<HD>::VS + (d >> 6) * 64 + t * 16 + ((d >> 4) & 3) * 4 + i;
}

// The two e2m1 codes of byte N of w as fp16 (low half: the low code).
template <int N>
__device__ __forceinline__ uint32_t e2m1x2_f16x2(uint32_t w) {
  uint32_t r;
  if constexpr (N == 0)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
  else if constexpr (N == 1)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
  else if constexpr (N == 2)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(w));
  else
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

// Two e4m3 scales (the low 16 bits of w) as fp16.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_hi_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<__half2*>(&w); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// The nearest e4m3 of x >= 0 (ties to even, saturating at 448), and its value.
__device__ __forceinline__ uint32_t e4m3_byte(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(x));
  return r;
}
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  return __low2float(as_half2(e4m3x2_f16x2(byte)));
}

// The nearest e2m1 codes of lo and hi (ties to even, saturating at 6), lo in the low half.
__device__ __forceinline__ uint32_t e2m1x2_byte(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 a;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.u32.u8 %0, a;\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

// The record of the 16 positions that slot's position belongs to (one block's
// records of a head follow each other).
template <int HD>
__device__ __forceinline__ size_t kv4_record(int block, int kvh, int group, int Hkv, int block_shift) {
  return (((static_cast<size_t>(block) * Hkv + kvh) << (block_shift - 4)) + group) * Kv4Rec<HD>::BYTES;
}

}  // namespace g4
