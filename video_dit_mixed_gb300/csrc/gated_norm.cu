// The norms before and after a transformer block's branch with its gate, the
// scaled residual and the next branch's modulation, rotated and quantized to
// INT8 per token (or left in bf16), one pass over the rows:
//
//   u = x, or x / sqrt(mean x^2 + eps) . post_w          (the branch's norm)
//   h = rs . residual + gate_s . u                       (sum_out = bf16(h))
//   y = h / sqrt(mean h^2 + eps) . w . (1 + scale_s) + shift_s
//   z = y . blockdiag(H_b / sqrt b),  s = max|z| / 127,  q = rint(z / s)
//
// s is the row's segment (text or frames, or a sample of the batch).
#include <cstdint>

#include "common.cuh"
#include "ctx_cache.h"
#include "internal.h"
#include "row_norm.cuh"

namespace sixbit {
namespace gnorm {

struct Params {
  GatedNormParams g;
  float inv_sqrt_b;
  int wide;  // x, res, sum_out, y are 32-byte aligned
};

// Sum (and maximum) over the CTA; two buffers, so that a later call's writes
// need no barrier of their own.
struct Joint {
  float ss[2][16];
  uint32_t mx[2][16];
};
__device__ __forceinline__ float cta_sum(float v, Joint& j, int buf, int nwarps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (nwarps == 1) return v;
  if ((threadIdx.x & 31) == 0) j.ss[buf][threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int i = 0; i < nwarps; ++i) v += j.ss[buf][i];
  return v;
}
__device__ __forceinline__ uint32_t cta_max(uint32_t v, Joint& j, int buf, int nwarps) {
  v = __reduce_max_sync(0xFFFFFFFFu, v);
  if (nwarps == 1) return v;
  if ((threadIdx.x & 31) == 0) j.mx[buf][threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
  for (int i = 0; i < nwarps; ++i) v = max(v, j.mx[buf][i]);
  return v;
}

__device__ __forceinline__ void load16f(const float* v, float fill, uint64_t (&o)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = f2_pack(fill, fill);
  if (v != nullptr) {
    const float4* v4 = reinterpret_cast<const float4*>(v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 a = __ldg(v4 + i);
      o[2 * i] = f2_pack(a.x, a.y);
      o[2 * i + 1] = f2_pack(a.z, a.w);
    }
  }
}

// A CTA takes whole rows, every gridDim-th one, V chunks of 16 elements a thread.
template <int B, int V>
__global__ void __launch_bounds__(512) row_kernel(const Params p) {
  const GatedNormParams& g = p.g;
  if (g.mode_dev != nullptr && SIXBIT_MODE_OF(*g.mode_dev) != SIXBIT_MODE_INT8) return;
  __shared__ Joint post, pre, top;
  const int chunks = g.K / kChunk, nwarps = blockDim.x >> 5;
  const float nan = __uint_as_float(0x7FC00000u);
  int buf = 0;
  for (int row = blockIdx.x; row < g.M; row += gridDim.x, buf ^= 1) {
    const size_t base = static_cast<size_t>(row) * g.K;
    int seg = 0;
    bool bad = false;
    if (g.segment != nullptr) {
      seg = __ldg(g.segment + row);
      bad = seg < 0 || seg >= g.S;
      if (bad) {
        seg = 0;
        if (threadIdx.x == 0) set_error(g.err, SIXBIT_EDEVICE);
      }
    } else if (g.S > 1) {
      seg = row / g.rows_per_seg;
    }
    const size_t mod = static_cast<size_t>(seg) * g.K;
    uint64_t u[V][8];
    uint64_t ss = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = threadIdx.x + v * blockDim.x;
      uint32_t xr[8] = {};
      if (c < chunks) load32(g.x + base + static_cast<size_t>(c) * kChunk, p.wide, xr);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        u[v][i] = bad ? f2_pack(nan, nan) : f2_from_bf16x2(xr[i]);
        ss = f2_fma(u[v][i], u[v][i], ss);
      }
    }
    float rpost = 1.f;
    if (g.post_w != nullptr) {
      const float sum = cta_sum(f2_lo(ss) + f2_hi(ss), post, buf, nwarps);
      rpost = finite_sum(sum) ? rms_inv(sum, g.K, g.eps) : nan;
    }
    ss = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = threadIdx.x + v * blockDim.x;
      if (c < chunks) {
        const int k = c * kChunk;
        if (g.post_w != nullptr) {
          uint64_t w[8];
          load16f(g.post_w + k, 1.f, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) u[v][i] = f2_mul(u[v][i], f2_mul(w[i], f2_pack(rpost, rpost)));
        }
        if (g.gate != nullptr) {
          uint64_t w[8];
          load16f(g.gate + mod + k, 1.f, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) u[v][i] = f2_mul(u[v][i], w[i]);
        }
        if (g.res != nullptr) {
          uint32_t rr[8];
          load32(g.res + base + k, p.wide, rr);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            u[v][i] = f2_fma(f2_from_bf16x2(rr[i]), f2_pack(g.res_scale, g.res_scale), u[v][i]);
        }
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = f2_to_bf16x2(u[v][i]);
        if (g.sum_out != nullptr) store32(g.sum_out + base + k, p.wide, o);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = f2_fma(u[v][i], u[v][i], ss);
      }
    }
    const float sum = cta_sum(f2_lo(ss) + f2_hi(ss), pre, buf, nwarps);
    const float rpre = finite_sum(sum) ? rms_inv(sum, g.K, g.eps) : nan;
    uint32_t mb = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = threadIdx.x + v * blockDim.x, k = c * kChunk;
      if (c < chunks) {
        uint64_t w[8];
        load16f(g.w != nullptr ? g.w + k : nullptr, 1.f, w);
        if (g.scale != nullptr) {
          uint64_t t[8];
          load16f(g.scale + mod + k, 0.f, t);
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = f2_fma(w[i], t[i], w[i]);
        }
        uint64_t t[8];
        load16f(g.shift != nullptr ? g.shift + mod + k : nullptr, 0.f, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[v][i] = f2_fma(f2_mul(u[v][i], f2_pack(rpre, rpre)), w[i], t[i]);
        if (g.y != nullptr) {
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = f2_to_bf16x2(u[v][i]);
          store32(g.y + base + k, p.wide, o);
        }
      }
      if (g.y == nullptr) {  // (every lane of the warp takes part)
        if (c >= chunks) {
#pragma unroll
          for (int i = 0; i < 8; ++i) u[v][i] = 0;
        }
        fwht<B>(u[v]);
        mb = max_bits(u[v], mb);
      }
    }
    if (g.y != nullptr) continue;
    mb = cta_max(mb, top, buf, nwarps);
    const RowOut o = row_out(p.inv_sqrt_b, true, mb);
    if (threadIdx.x == 0) g.row_scale[row] = o.scale;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = threadIdx.x + v * blockDim.x;
      if (c < chunks) store_codes(g.codes + base + static_cast<size_t>(c) * kChunk, o, u[v]);
    }
  }
}

template <int B, int V>
cudaError_t launch_rows(const Params& p, int threads, cudaStream_t st) {
  static ContextCache<int> cache[17];  // resident CTAs an SM, by warps
  int per_sm = 0;
  const cudaError_t e = cache[threads / 32].get(&per_sm, [&](int* o) {
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(o, row_kernel<B, V>, threads, 0);
  });
  if (e != cudaSuccess) return e;
  const int most = sm_count() * (per_sm > 0 ? per_sm : 1);
  note_launch();
  row_kernel<B, V><<<p.g.M < most ? p.g.M : most, threads, 0, st>>>(p);
  return cudaGetLastError();
}

template <int B>
cudaError_t launch(const Params& p, cudaStream_t st) {
  const int chunks = p.g.K / kChunk;
  const int v = chunks <= 256 ? 1 : 2;
  const int threads = ((chunks + v - 1) / v + 31) / 32 * 32;
  return v == 1 ? launch_rows<B, 1>(p, threads, st) : launch_rows<B, 2>(p, threads, st);
}

}  // namespace gnorm

cudaError_t launch_gated_norm(const GatedNormParams& g, int b, cudaStream_t st) {
  gnorm::Params p{};
  p.g = g;
  p.inv_sqrt_b = b == 16 ? 0.25f : b == 64 ? 0.125f : b == 256 ? 0.0625f : 1.f;
  const auto a32 = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 31u) == 0; };
  p.wide = a32(g.x) && a32(g.res) && a32(g.sum_out) && a32(g.y);
  switch (b) {
    case 16: return gnorm::launch<16>(p, st);
    case 64: return gnorm::launch<64>(p, st);
    case 256: return gnorm::launch<256>(p, st);
    default: return gnorm::launch<0>(p, st);
  }
}

}  // namespace sixbit
