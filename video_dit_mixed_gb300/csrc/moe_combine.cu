// The sum that ends a routed feed-forward layer:
//
//   y[t] = sum_j w[t][j] . d[rows[t][j]],   j = 0 .. k - 1
//
// in FP32, rounded once to bf16 (or kept).  Term j joins partial sum j % 4 and the
// partial sums are added in their order, whatever the launch.
#include <cstdint>

#include "common.cuh"
#include "internal.h"

namespace sixbit {
namespace combine {

constexpr int kThreads = 256;

// Eight (VEC) or one element of row r from column c on.
template <bool VEC, bool F32>
__device__ __forceinline__ void load(const void* d, size_t at, float (&v)[8]) {
  if constexpr (VEC && F32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(d) + at);
    const float4 a = __ldg(q), b = __ldg(q + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else if constexpr (VEC) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(d) + at));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else if constexpr (F32) {
    v[0] = __ldg(static_cast<const float*>(d) + at);
  } else {
    v[0] = __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(d) + at)) << 16);
  }
}

template <bool VEC, bool F32>
__global__ void __launch_bounds__(kThreads) kernel(const CombineParams p) {
  constexpr int E = VEC ? 8 : 1;
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * E;
  if (c >= p.H) return;
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    float acc[4][E] = {};
    const size_t tk = static_cast<size_t>(t) * p.k;
    for (int j0 = 0; j0 < p.k; j0 += 4) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (j0 + q >= p.k) break;
        const int r = __ldg(p.rows + tk + j0 + q);
        if (r >= 0 && r < p.R) {
          const float w = __ldg(p.weights + tk + j0 + q);
          float v[8];
          load<VEC, F32>(p.d, static_cast<size_t>(r) * p.H + c, v);
#pragma unroll
          for (int i = 0; i < E; ++i) acc[q][i] = __fadd_rn(acc[q][i], __fmul_rn(w, v[i]));
        } else if (r != -1) {
          set_error(p.err, SIXBIT_EDEVICE);
        }
      }
    }
    float y[E];
#pragma unroll
    for (int i = 0; i < E; ++i) y[i] = ((acc[0][i] + acc[1][i]) + acc[2][i]) + acc[3][i];
    const size_t at = static_cast<size_t>(t) * p.H + c;
    if constexpr (VEC) {
      if (p.Yf != nullptr) {
        reinterpret_cast<float4*>(p.Yf + at)[0] = make_float4(y[0], y[1], y[2], y[3]);
        reinterpret_cast<float4*>(p.Yf + at)[1] = make_float4(y[4], y[5], y[6], y[7]);
      } else {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = f2_to_bf16x2(f2_pack(y[2 * i], y[2 * i + 1]));
        *reinterpret_cast<uint4*>(p.Y + at) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    } else if (p.Yf != nullptr) {
      p.Yf[at] = y[0];
    } else {
      p.Y[at] = __bfloat16_as_ushort(__float2bfloat16_rn(y[0]));
    }
  }
}

}  // namespace combine

cudaError_t launch_moe_combine(const CombineParams& p, cudaStream_t st) {
  const auto a16 = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; };
  const bool vec = p.H % 8 == 0 && a16(p.d) && a16(p.Y) && a16(p.Yf);
  const int64_t units = vec ? p.H / 8 : p.H;
  const int threads = static_cast<int>(units < combine::kThreads ? (units + 31) / 32 * 32 : combine::kThreads);
  const dim3 grid(static_cast<unsigned>(p.T), static_cast<unsigned>((units + threads - 1) / threads));
  note_launch();
  if (vec && p.f32)
    combine::kernel<true, true><<<grid, threads, 0, st>>>(p);
  else if (vec)
    combine::kernel<true, false><<<grid, threads, 0, st>>>(p);
  else if (p.f32)
    combine::kernel<false, true><<<grid, threads, 0, st>>>(p);
  else
    combine::kernel<false, false><<<grid, threads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace sixbit
