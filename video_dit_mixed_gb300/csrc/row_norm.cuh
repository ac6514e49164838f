// What the kernels that norm rows and quantize them share: 16-element chunks of
// bf16, the block-Hadamard butterfly across a warp's chunks, and a row's INT8
// codes from its largest magnitude.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace sixbit {

constexpr int kChunk = 16;  // elements of a chunk: 32 bytes of bf16, 16 of codes

__device__ __forceinline__ void load32(const uint16_t* p, bool wide, uint32_t (&r)[8]) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p)
                 : "memory");
  } else {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    r[0] = a.x, r[1] = a.y, r[2] = a.z, r[3] = a.w, r[4] = b.x, r[5] = b.y, r[6] = b.z, r[7] = b.w;
  }
}
__device__ __forceinline__ void store32(uint16_t* p, bool wide, const uint32_t (&r)[8]) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(r[0], r[1], r[2], r[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(r[4], r[5], r[6], r[7]);
  }
}

// Unscaled fixed-order butterfly (ascending strides) over blocks of B; u holds
// elements 16 t .. 16 t + 15 of lane t's chunk as pairs.  Every lane of the
// warp takes part.
template <int B>
__device__ __forceinline__ void fwht(uint64_t (&u)[8]) {
  if constexpr (B >= 16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = f2_lo(u[i]), b = f2_hi(u[i]);
      u[i] = f2_pack(__fadd_rn(a, b), __fsub_rn(a, b));
    }
#pragma unroll
    for (int h = 1; h < 8; h <<= 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if ((i & h) == 0) {
          const uint64_t a = u[i], b = u[i | h];
          u[i] = f2_add(a, b);
          u[i | h] = f2_sub(a, b);
        }
      }
    }
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 1; h < B / kChunk; h <<= 1) {
      const float sg = (lane & h) ? -1.f : 1.f;  // upper lane: other - mine
      const uint64_t s2 = f2_pack(sg, sg);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t o = __shfl_xor_sync(0xFFFFFFFFu, static_cast<unsigned long long>(u[i]), h);
        u[i] = f2_fma(u[i], s2, o);
      }
    }
  }
}

// 16 weights from channel k on, as pairs (1 without weights, or beyond the row).
__device__ __forceinline__ void load_weights(const float* weight, int k, bool live, uint64_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = f2_pack(1.f, 1.f);
  if (weight != nullptr && live) {
    const float4* w4 = reinterpret_cast<const float4*>(weight + k);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = __ldg(w4 + i);
      w[2 * i] = f2_pack(v.x, v.y);
      w[2 * i + 1] = f2_pack(v.z, v.w);
    }
  }
}

// max over |u| as bit patterns: a NaN compares above infinity, so it is kept
__device__ __forceinline__ uint32_t max_bits(const uint64_t (&u)[8], uint32_t m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t a = f2_abs(u[i]);
    m = max(m, max(static_cast<uint32_t>(a), static_cast<uint32_t>(a >> 32)));
  }
  return m;
}

// 1 / sqrt(ss / K + eps)
__device__ __forceinline__ float rms_inv(float ss, int K, float eps) {
  return __fdiv_rn(1.f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, static_cast<float>(K)), eps)));
}
__device__ __forceinline__ bool finite_sum(float ss) { return ss < __uint_as_float(0x7F800000u); }

// A row's scale, and the multiplier of u that gives codes (pre: applied to u
// first, so that the multiplier is finite for the smallest maxima): z is u times
// `factor`, mbits the bits of max|u|, and `fine` says that the row's sums are
// finite.  A row whose sums or maximum are not gets a NaN scale and zero codes.
struct RowOut {
  float scale, mul, pre;
};
__device__ __forceinline__ RowOut row_out(float factor, bool fine, uint32_t mbits) {
  const float a = __uint_as_float(mbits);
  RowOut o;
  o.pre = a < 1e-30f ? 0x1p100f : 1.f;
  const bool bad = mbits >= 0x7F800000u || !fine;
  o.mul = (bad || mbits == 0) ? 0.f : __fdiv_rn(127.f, a * o.pre);
  o.scale = bad ? __uint_as_float(0x7FC00000u) : __fdiv_rn(a * factor, 127.f);
  return o;
}

__device__ __forceinline__ void store_codes(int8_t* codes, const RowOut& o, uint64_t (&u)[8]) {
  if (o.pre != 1.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = f2_mul(u[i], f2_pack(o.pre, o.pre));
  }
  const uint64_t mul = f2_pack(o.mul, o.mul), magic = f2_pack(12582912.f, 12582912.f);
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t a = f2_fma(u[2 * i], mul, magic), b = f2_fma(u[2 * i + 1], mul, magic);
    const uint32_t lo = __byte_perm(static_cast<uint32_t>(a), static_cast<uint32_t>(a >> 32), 0x0040);
    const uint32_t hi = __byte_perm(static_cast<uint32_t>(b), static_cast<uint32_t>(b >> 32), 0x0040);
    q[i] = o.mul == 0.f ? 0u : __byte_perm(lo, hi, 0x5410);  // (a NaN times 0 is not a code)
  }
  *reinterpret_cast<uint4*>(codes) = make_uint4(q[0], q[1], q[2], q[3]);
}

}  // namespace sixbit
