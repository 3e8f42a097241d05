// Layout of a page of the 4-bit cache: 16 tokens of one lane, K and V.
//
// G = d / 32 groups a row.  A page holds, one after the other,
//   K codes   16 rows of d/2 bytes; word c * G + w of a row (c = 0..3) holds
//             the eight codes of elements 32 w + 8 c .. + 7, element j in
//             bits 4 j: thread c of a quad gets its share of every group with
//             one wide load;
//   V codes   words in the order of the 16x16 tiles the tensor core takes as
//             its left operand, V transposed: tile dt (elements 16 dt .. + 15),
//             thread 4 gq + cq of the warp.  The word's nibbles 0, 4, 2, 6 are
//             element 16 dt + gq of tokens 2 cq, 2 cq + 1, 2 cq + 8, 2 cq + 9,
//             nibbles 1, 5, 3, 7 element 16 dt + gq + 8 of the same tokens, so
//             each half-word pair (nibble i, nibble i + 4) is one operand
//             register.  Four tiles of a thread are adjacent (16 bytes);
//   K scales  bf16 [16 tokens][G];
//   V ratios  fp16 [4 cq][G][4 tokens 2 cq, 2 cq + 1, 2 cq + 8, 2 cq + 9];
//   V exponents int8 [16 tokens]: the scale of (token, group) is
//             ratio * 2^exponent.
// A stored code is code + 8 (1..15).  Every word of codes is kept rotated left
// by two bits: nibbles 0 and 4 then lie in bits 2-5 of the two halves, nibbles 1
// and 5 in bits 6-9 (all within an fp16 mantissa), and one rotation by 8 brings
// nibbles 2, 6 and 3, 7 there.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace kve {

template <int D>
struct Kv4Page {
  static constexpr int kG = D / 32;
  static constexpr int kRow = D / 2;                       // bytes of a K row's codes
  static constexpr int kV = 16 * kRow;                     // offset of the V codes
  static constexpr int kKScale = 32 * kRow;
  static constexpr int kVRatio = kKScale + 16 * kG * 2;
  static constexpr int kVExp = kVRatio + 16 * kG * 2;
  static constexpr int kUsed = kVExp + 16;                 // bytes a reader copies (a multiple of 16)
  static constexpr int kBytes = (kUsed + 31) / 32 * 32;    // page stride: whole 32-byte sectors
  static constexpr int kExpMin = -64, kExpMax = 62;

  __host__ __device__ static constexpr int v_word(int dt, int lane) {
    return ((dt / 4) * 32 + lane) * 4 + dt % 4;
  }
  __device__ static __forceinline__ uint32_t pack(uint32_t nibbles) { return __funnelshift_l(nibbles, nibbles, 2); }
  __device__ static __forceinline__ uint32_t unpack(uint32_t word) { return __funnelshift_r(word, word, 2); }
  __host__ __device__ static constexpr int v_ratio(int t, int w) {
    return (((t & 7) >> 1) * kG + w) * 4 + (t & 1) + (t >= 8 ? 2 : 0);
  }
};

}  // namespace kve
