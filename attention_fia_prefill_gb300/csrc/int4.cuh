// The 4-bit key/value cache (fia_cache_write_int4 and its readers).
//
// A row (one token, one kv head) of D values is cut into groups of G = D / NG.
// A group holds (step, low) in the type of the keys and values and a code in
// 0..15 for each value:
//   low = min x,  step = max((max x - min x) / 15 rounded up, tiny),
//   code = ceil((x - low) / step - 1/2),  value = low + step * code.
// low is a value of the type, so it is exact, and a step that is rounded up
// leaves no value past code 15.  In f16 it is rounded down where low + 15 step would
// be more than the type holds: code 15 then stands for a little less than the group's
// largest value (2^-10 of 15 steps at most, so it is the nearest still), and a finite
// value reads back finite.  tiny, 2^-60 (bf16) or 2^-24 (f16, its smallest),
// and the largest value, 2^60, keep 1 / step and, in the attention, a step's or a
// low value's products with the weights within fp32.
//
// The 16-bit unit (D/32) g + j of a row (g in 0..7, j < D/32) holds columns
// 32 j + 4 g .. + 3, lowest nibble first.  A lane of a matrix product's fragment
// then finds whole words of columns, and the columns that one product of depth
// 16 (or 16 output columns) covers are of one j, so of one group for every G.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "ptx.cuh"

namespace fia {

constexpr float kInt4Most = 0x1p60f;                                // groups with larger values read back as NaN
constexpr float kInt4MostHalf = 65504.f;                            // the largest f16
template <bool BF16>
constexpr float kInt4Tiny = BF16 ? 0x1p-60f : 0x1p-24f;

// (step, low) of a group's 32-bit word.
template <bool BF16>
__device__ __forceinline__ float2 int4_pair(uint32_t w) {
  if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Two outputs of a decode.  They are averages of values within the type, of weights
// rounded to 11 bits: one of 65504 may come out above, and is not to be an infinity.
template <bool BF16>
__device__ __forceinline__ uint32_t int4_out(float lo, float hi) {
  uint32_t u = pack2(lo, hi, BF16);
  if constexpr (!BF16) {   // (a NaN stays)
    asm("min.NaN.f16x2 %0, %0, %1;" : "+r"(u) : "r"(0x7bff7bffu));
    asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(u) : "r"(0xfbfffbffu));
  }
  return u;
}

}  // namespace fia
