// The 4-bit weight form (moe_w4_t): constants and the device-side steps that its kernels share.
//
// A matrix [N, K] (nn.Linear layout, K contracted, both multiples of 64) stands for
//     W[n, k] = row_scale[n] * (scale[k / g, n] * (code[n, k] - zero[k / g, n]))
// with 4-bit codes, e4m3 scales per group of g = 32, 64 or 128 consecutive k, 4-bit zero points
// (8 everywhere when absent) and one fp32 factor per row.  code - zero has at most 4 significant
// bits and so has an e4m3 number: the product in the inner brackets has at most 8 and is a bf16
// exactly.  The tensor cores therefore take scale * (code - zero) as their bf16 operand (or, for
// few rows, code - zero as their fp16 operand and scale on the group's fp32 sum) without any
// rounding, and row_scale is one fp32 factor on the finished sum.  Scales and zero points
// are stored [K / g, N] (rows of a tile are neighbours in memory).
//
// Codes: 64 consecutive k of a row are 32 bytes, eight little-endian words; word 2 c + j holds
// the eight k from 32 j + 8 c on, k + 2 i in nibble i and k + 2 i + 1 in nibble 4 + i (i < 4).
// So (word >> 4 i) & 0x000f000f is the pair (k + 2 i, k + 2 i + 1) in two 16-bit halves, and a
// thread's 8 bytes (words 2 c, 2 c + 1) hold 8 k of either 32-element half.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace moe {

constexpr int W4_BLOCK = 64;                    // k per block of the code layout (32 bytes)

__device__ __forceinline__ float w4_scale(uint8_t s) {
  __nv_fp8_e4m3 v;
  v.__x = s;
  return static_cast<float>(v);
}

struct W4Ptrs {                                 // device views of a moe_w4_t
  const uint32_t* codes;                        // [G, N, K / 8] words
  const uint8_t* scales;                        // [G, groups, N]
  const uint8_t* zeros;                         // [G, groups, N] or null
  const float* row_scale;                       // [G, N]
};

}  // namespace moe
