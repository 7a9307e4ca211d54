// The 4-bit cache record (include/gqa.h): its sizes and the conversions that
// writing, reading back and attending share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "gqa.h"

namespace gqa {
namespace q4 {

constexpr int kGroup = GQA_Q4_GROUP;
constexpr int kHeadBytes = 16;  // scale and minimum of up to four groups

__host__ __device__ constexpr int groups_of(int D) { return (D + kGroup - 1) / kGroup; }
__host__ __device__ constexpr int record_bytes(int D) { return kHeadBytes + 16 * groups_of(D); }

template <bool V>
struct BoolConst {
  static constexpr bool value = V;
};

// 16-bit pattern <-> fp32 of the cache's type.
template <bool F16>
__device__ __forceinline__ float to_f32(uint32_t bits16) {
  if (F16) return __half2float(__ushort_as_half(static_cast<unsigned short>(bits16)));
  return __uint_as_float(bits16 << 16);
}
template <bool F16>
__device__ __forceinline__ uint32_t to_16(float x) {
  if (F16) return __half_as_ushort(__float2half_rn(x));
  return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// Scale and minimum of a group from its 4 bytes in the record's head.
template <bool F16>
__device__ __forceinline__ float scale_of(uint32_t word) {
  if (F16) return __low2float(*reinterpret_cast<const __half2*>(&word));
  return __uint_as_float(word << 16);
}
template <bool F16>
__device__ __forceinline__ float min_of(uint32_t word) {
  if (F16) return __high2float(*reinterpret_cast<const __half2*>(&word));
  return __uint_as_float(word & 0xFFFF0000u);
}

}  // namespace q4
}  // namespace gqa
