// nq_kv_layout.cuh — the byte order of a cache atom (16 tokens x D dimensions of
// one kv head, keys and values) and the conversions from its formats.
//
// The order is that of the fragments of a 16 x 8 x 16 matrix product: lane 4 r
// + j of a warp holds, as its share of the 16 x D key matrix, rows r and r + 8
// and the dimensions [j D/4, (j+1) D/4) (the contraction runs over dimensions
// in any order, so a lane's share is contiguous), and of the value matrix
// transposed the dimensions [r D/8, (r+1) D/8) of tokens 2j, 2j+1, 2j+8, 2j+9.
// Every lane then reads its codes as whole 16-byte words, lane after lane, and
// a token's bytes belong to that token alone, so appending one never reads its
// neighbours.
#pragma once

#include <cuda_fp16.h>

#include "nq_device.cuh"
#include "nq_kv.h"

namespace nq {

template <int D>
struct KvAtom {
  static_assert(D == 64 || D == 128 || D == 256, "head dimension");
  static constexpr int kBytes = 18 * D;
  static constexpr int kVCodes = 8 * D, kKScales = 16 * D, kVScales = 17 * D;
  static constexpr int kN = D / 64;                         // 16-element key blocks of a lane per row
  static constexpr int kW = D / 128 > 0 ? D / 128 : 1;      // value blocks of a lane per token

  // Byte offsets of token t's block b (16 dimensions): 8 bytes of codes, 1 of scale.
  __device__ static __forceinline__ int k_codes(int t, int b) {
    const int s = (t >> 3) * kN + b % kN, lane = (t & 7) * 4 + b / kN;
    return (s >> 1) * 512 + lane * 16 + (s & 1) * 8;
  }
  __device__ static __forceinline__ int k_scale(int t, int b) {
    return kKScales + ((t & 7) * 4 + b / kN) * (2 * kN) + (t >> 3) * kN + b % kN;
  }
  __device__ static __forceinline__ int v_codes(int t, int b) {
    const int i = (t >> 3) * 2 + (t & 1), j = (t >> 1) & 3;
    const int r = 16 * b / (D / 8);
    const int w = i * (D / 16) + 8 * b - r * (D / 16);  // byte in the lane's sequence
    return kVCodes + (w >> 4) * 512 + (4 * r + j) * 16 + (w & 15);
  }
  __device__ static __forceinline__ int v_scale(int t, int b) {
    const int i = (t >> 3) * 2 + (t & 1), j = (t >> 1) & 3;
    return kVScales + ((b / kW) * 4 + j) * (4 * kW) + i * kW + b % kW;
  }
};

// Eight e2m1 codes -> four f16 pairs, code 2i in the low half of pair i (exact).
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// Two e4m3 codes (low 16 bits of c) -> an f16 pair (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t c) {
  uint32_t h;
  asm("{\n\t.reg .b16 c2;\n\tcvt.u16.u32 c2, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c2;\n\t}" : "=r"(h) : "r"(c));
  return h;
}
// Softmax weights 2^(s - m) are rounded to f16.  m lies kHeadroom below a score that was the running maximum and is
// raised once a score exceeds that one by more than kRaise (both log2): weights reach 2^15, in f16's range, and the
// largest of a row is 2^7 at least, so f16's smallest half step, 2^-25, is 2^-32 of it.  Without the headroom a long,
// flat tail 2^25 below one early peak was lost whole.
constexpr float kHeadroom = 7.0f, kRaise = 8.0f;
// log sum exp of the scores: from m and the sum of 2^(s - m); exact in m's part whatever m was rounded to.
__device__ __forceinline__ float lse_of(float m, float sum) {
  return sum == 0.0f ? -INFINITY : ((m + kHeadroom) + log2f(sum * 0.0078125f)) * 0.6931471805599453f;
}
// The largest power of two by which a query row is scaled: its inverse, too, is a normal number.
constexpr int kMostPower = 126;
// 0, or NaN for a score factor that is none: added to the sum of a row that has keys, as its c hides a NaN.
__device__ __forceinline__ float nan_of(float factor) { return factor - factor; }
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

}  // namespace nq
