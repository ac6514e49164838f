// Device helpers of the W4A8 products on the stored operands: nibbles and codes
// to fp16 (w4a8_rows.cu), and an expert's row range (also w4a8_grouped.cu).
#pragma once

#include <cstdint>

#include "common.cuh"
#include "internal.h"

namespace sixbit {

// One FMA or subtraction per fp16 pair, exact (integers below 2048).
__device__ __forceinline__ uint32_t sub2(uint32_t x, uint32_t c) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t fma2(uint32_t x, uint32_t m, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(x), "r"(m), "r"(c));
  return d;
}

// Eight nibbles -> pairs o[j] = (k = j, k = j + 4).  Flipping a nibble's sign
// bit makes it v + 8; under the exponent of 1024 the low nibbles read
// 1032 + v, the high ones 1024 + 16 (v + 8).
__device__ __forceinline__ void nibbles_f16(uint32_t w, uint32_t (&o)[4]) {
  const uint32_t h = w >> 8;
  o[0] = sub2((w & 0x000F000Fu) ^ 0x64086408u, 0x64086408u);
  o[1] = fma2((w & 0x00F000F0u) ^ 0x64806480u, 0x2C002C00u, 0xD480D480u);  // / 16 - 72
  o[2] = sub2((h & 0x000F000Fu) ^ 0x64086408u, 0x64086408u);
  o[3] = fma2((h & 0x00F000F0u) ^ 0x64806480u, 0x2C002C00u, 0xD480D480u);
}

// Eight s8 codes (k = 0..3 in a, 4..7 in b) -> the same pairs.
__device__ __forceinline__ void codes_f16(uint32_t a, uint32_t b, uint32_t (&o)[4]) {
  a ^= 0x80808080u;
  b ^= 0x80808080u;
  const uint32_t lo = __byte_perm(a, b, 0x5140), hi = __byte_perm(a, b, 0x7362);
  o[0] = sub2(__byte_perm(lo, 0x64646464u, 0x4140), 0x64806480u);
  o[1] = sub2(__byte_perm(lo, 0x64646464u, 0x4342), 0x64806480u);
  o[2] = sub2(__byte_perm(hi, 0x64646464u, 0x4140), 0x64806480u);
  o[3] = sub2(__byte_perm(hi, 0x64646464u, 0x4342), 0x64806480u);
}

// Rows [*first, *first + *count) of expert e; an offset pair that is not
// ascending within [0, M] is reported and read as an expert without rows.
__device__ __forceinline__ void expert_rows(const RowsParams& p, int e, bool report, int* first, int* count) {
  *first = 0;
  *count = p.M;
  if (p.offsets == nullptr) return;
  const int a = __ldg(p.offsets + e), b = __ldg(p.offsets + e + 1);
  const bool ok = a >= 0 && a <= b && b <= p.M;
  if (!ok && report) set_error(p.err, SIXBIT_EDEVICE);
  *first = ok ? a : 0;
  *count = ok ? b - a : 0;
}

}  // namespace sixbit
