// The row format of the 4-bit paged cache, shared by the kernels that write it,
// read it back and attend to it.
//
// A row is one token of one key head, K and V together, in 160 bytes:
//   bytes   0 ..  63  K codes, 4 bits each, as 16 little-endian words
//   bytes  64 .. 127  V codes, 4 bits each, as 16 little-endian words
//   bytes 128 .. 159  16 bfloat16: K scales, K minima, V scales, V minima
// with one scale and one minimum per group of 32 channels; a value is
// minimum + scale * code.  K and V sit in one row because every reader wants
// both: a row is then exactly five 32-byte sectors wherever it lies, which is
// what a gather of single rows pays for.
//
// Order of the codes.  The attention kernel feeds codes to mma.sync fragments,
// whose lanes are (gid, tig) = (lane / 4, lane % 4), without any shuffle:
//   K channel 32g + 8t + j   word 4t + g, nibble j: the 16 bytes of lane t hold
//                            8 channels of each of the 4 scale groups
//   V channel 32g + 4r + i   word 2r + g/2, half g%2, nibble i: the 8 bytes of
//                            lane group r hold 4 channels of each scale group
#pragma once

#include <cstdint>

#include "common.cuh"

namespace kascade {

constexpr int kQ4Row = 160;      // bytes of a row
constexpr int kQ4V = 64;         // byte offset of the V codes
constexpr int kQ4Tail = 128;     // byte offset of the scales and minima

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <bool F16>
__device__ __forceinline__ void unpack2(uint32_t w, float& lo, float& hi) {
  if constexpr (F16) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    lo = f.x;
    hi = f.y;
  } else {
    lo = bf16_lo(w);
    hi = bf16_hi(w);
  }
}

}  // namespace kascade
