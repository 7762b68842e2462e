// Device helpers shared by the microscaled (MXFP4) kernels.
//
// Format: e2m1 codes, 4 bits each, in gptq_pack's 4-bit layout (the code of
// column k at bits [4k, 4k + 4) of its row's stream of 32-bit words), and one
// e8m0 byte for every 32 columns of a row: the scale 2^(byte - 127), 255 = NaN.
// A block's 32 codes are four words: one 16-byte load, and exactly the share
// of one lane in the scaled matrix instructions.
#pragma once

#include "common.h"

namespace gptq {

constexpr int kMxBlock = 32;                 // columns that share a scale
constexpr int64_t kMxMaxCols = 1 << 20;      // keeps in-row offsets far below 32 bits
constexpr int kMxScaleOne = 127;             // byte of the scale 1
constexpr int kMxScaleNan = 255;

// Sixteen bytes at any element-aligned address (gfx950 global loads and
// stores take unaligned addresses; the type tells the compiler so).
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef _Float16 halfx2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float floatx2 __attribute__((ext_vector_type(2)));

// The float32 whose exponent field is the byte, as the conversion and matrix
// instructions take scales: they use the field alone, so byte 0 is 2^-127 and
// 255 is NaN there.
__device__ inline float mx_scale_operand(uint32_t byte) { return __uint_as_float(byte << 23); }

}  // namespace gptq
