// The sum that ends a routed feed-forward layer:
//
//   y[t] = sum_j w[t][j] . d[rows[t][j]],   j = 0 .. k - 1
//
// in FP32, rounded once to bf16 (or kept).  Term j joins partial sum j % 4 and the
// partial sums are added in their order, whatever the launch.
//
// Bytes bound it: 17,776 tokens of two rows of 1920 floats 54 us (6.3 TB/s, 93% of a
// copy), of bf16 35 (85%); 8 tokens 1.7 us, 226 of eight rows of bf16 4.5.  (A token
// a CTA, its rows' numbers loaded when they are needed: 78 and 60 us.)
#include <cstdint>

#include "common.cuh"
#include "ctx_cache.h"
#include "internal.h"

namespace sixbit {
namespace combine {

constexpr int kThreads = 256;

// Eight (VEC) or one element of d from element `at` on, as they lie in memory.
template <bool VEC, bool F32>
struct Piece {
  uint32_t w[VEC ? (F32 ? 8 : 4) : 1];
  __device__ __forceinline__ void load(const void* d, size_t at, bool wide) {
    if constexpr (VEC && F32) {
      const float* q = static_cast<const float*>(d) + at;
      if (wide) {
        asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(q));
      } else {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(q)), b = __ldg(reinterpret_cast<const uint4*>(q) + 1);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
      }
    } else if constexpr (VEC) {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(d) + at));
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    } else if constexpr (F32) {
      w[0] = __ldg(static_cast<const uint32_t*>(d) + at);
    } else {
      w[0] = static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(d) + at)) << 16;
    }
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (VEC && !F32)
      return __uint_as_float((i & 1) ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    else
      return __uint_as_float(w[i]);
  }
};

template <bool VEC>
__device__ __forceinline__ void store(const CombineParams& p, size_t at, const float (&y)[VEC ? 8 : 1]) {
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

// A thread takes eight columns (VEC) or one of every gridDim.x-th token, U tokens
// at once and C choices of each.  The rows and weights of the next choices are
// loaded while these are summed: they are a trip to memory in front of the rows
// themselves.  C = 2 is for k <= 2.
template <bool VEC, bool F32, int C, int U>
__global__ void __launch_bounds__(kThreads) kernel(const CombineParams p) {
  constexpr int E = VEC ? 8 : 1;
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * E;
  if (c >= p.H) return;
  int r[U][C];
  float w[U][C];
  auto choices = [&](int64_t t, int j0) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int q = 0; q < C; ++q) {
        r[u][q] = -1;
        w[u][q] = 0.f;
        const int64_t tu = t + static_cast<int64_t>(u) * gridDim.x;
        if (tu < p.T && j0 + q < p.k) {
          r[u][q] = __ldg(p.rows + tu * p.k + j0 + q);
          w[u][q] = __ldg(p.weights + tu * p.k + j0 + q);
        }
      }
  };
  choices(blockIdx.x, 0);
  const int64_t step = static_cast<int64_t>(gridDim.x) * U;
  for (int64_t t = blockIdx.x; t < p.T; t += step) {
    float acc[U][C][E] = {};
    for (int j0 = 0;; j0 += C) {
      Piece<VEC, F32> v[U][C];
      float wt[U][C];
      bool in[U][C];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int q = 0; q < C; ++q) {
          const int row = r[u][q];
          in[u][q] = static_cast<unsigned>(row) < static_cast<unsigned>(p.R);
          if (!in[u][q] && row != -1) set_error(p.err, SIXBIT_EDEVICE);
          wt[u][q] = w[u][q];
          if (in[u][q]) v[u][q].load(p.d, static_cast<size_t>(row) * p.H + c, p.wide);
        }
      const bool last = C == 2 || j0 + C >= p.k;
      if (!last)
        choices(t, j0 + C);
      else if (t + step < p.T)
        choices(t + step, 0);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int q = 0; q < C; ++q)
          if (in[u][q]) {
#pragma unroll
            for (int i = 0; i < E; ++i) acc[u][q][i] = __fadd_rn(acc[u][q][i], __fmul_rn(wt[u][q], v[u][q].value(i)));
          }
      if (last) break;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t tu = t + static_cast<int64_t>(u) * gridDim.x;
      if (tu >= p.T) break;
      float y[E];
#pragma unroll
      for (int i = 0; i < E; ++i) {
        y[i] = acc[u][0][i] + acc[u][1][i];
#pragma unroll
        for (int q = 2; q < C; ++q) y[i] += acc[u][q][i];
      }
      store<VEC>(p, static_cast<size_t>(tu) * p.H + c, y);
    }
  }
}

template <bool VEC, bool F32, int C, int U>
cudaError_t launch_form(const CombineParams& p, cudaStream_t st) {
  // the CTAs that are resident at once, each with an equal share of the tokens
  const int64_t units = VEC ? p.H / 8 : p.H;
  const int threads = static_cast<int>(units < kThreads ? (units + 31) / 32 * 32 : kThreads);
  const int groups = static_cast<int>((units + threads - 1) / threads);
  static ContextCache<int> cache[kThreads / 32 + 1];
  int per_sm = 0;
  const cudaError_t e = cache[threads / 32].get(&per_sm, [&](int* o) {
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(o, kernel<VEC, F32, C, U>, threads, 0);
  });
  if (e != cudaSuccess) return e;
  const int64_t most = static_cast<int64_t>(sm_count()) * (per_sm > 0 ? per_sm : 1) / groups;
  int64_t x = p.T;
  if (x > most && most > 0) {
    const int64_t turns = (p.T + most * U - 1) / (most * U);
    x = (p.T + turns * U - 1) / (turns * U);
  }
  note_launch();
  kernel<VEC, F32, C, U><<<dim3(static_cast<unsigned>(x), static_cast<unsigned>(groups)), threads, 0, st>>>(p);
  return cudaGetLastError();
}

template <bool VEC, bool F32>
cudaError_t launch(const CombineParams& p, cudaStream_t st) {
  return p.k <= 2 ? launch_form<VEC, F32, 2, 2>(p, st) : launch_form<VEC, F32, 4, 1>(p, st);
}

}  // namespace combine

cudaError_t launch_moe_combine(CombineParams p, cudaStream_t st) {
  const auto to = [](const void* q, uintptr_t n) { return (reinterpret_cast<uintptr_t>(q) & (n - 1)) == 0; };
  p.wide = p.f32 && to(p.d, 32) && p.H % 8 == 0;
  if (p.H % 8 == 0 && to(p.d, 16) && to(p.Y, 16) && to(p.Yf, 16))
    return p.f32 ? combine::launch<true, true>(p, st) : combine::launch<true, false>(p, st);
  return p.f32 ? combine::launch<false, true>(p, st) : combine::launch<false, false>(p, st);
}

}  // namespace sixbit
