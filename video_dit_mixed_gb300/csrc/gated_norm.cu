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

// Up to three factors a channel remain when those of the same place are joined:
// post_w . gate, w . (1 + scale) and shift.  Each thread keeps those of its own
// channels in shared memory (four 16-byte pieces a chunk, side by side across the
// threads) and joins them anew when a row's segment differs from the last one's.
struct Vectors {
  float4* at;  // [3][V][4][threads]
  int threads;
  template <int V>
  __device__ __forceinline__ float4* place(int which, int v) const {
    return at + (static_cast<size_t>(which) * V + v) * 4 * threads + threadIdx.x;
  }
  template <int V>
  __device__ __forceinline__ void put(int which, int v, const uint64_t (&w)[8]) const {
    float4* o = place<V>(which, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i * threads] = make_float4(f2_lo(w[2 * i]), f2_hi(w[2 * i]), f2_lo(w[2 * i + 1]), f2_hi(w[2 * i + 1]));
  }
  template <int V>
  __device__ __forceinline__ void get(int which, int v, uint64_t (&w)[8]) const {
    const float4* o = place<V>(which, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = o[i * threads];
      w[2 * i] = f2_pack(f.x, f.y);
      w[2 * i + 1] = f2_pack(f.z, f.w);
    }
  }
};

// A CTA takes whole rows, every gridDim-th one, V chunks of 16 elements a thread,
// with the next row's loads in flight while this one is reduced and stored.  The
// row's second factor multiplies every y but the shift: without one it drops out
// of the codes, and the sum and the maximum are one reduction.
template <int B, int V>
__global__ void __launch_bounds__(512) row_kernel(const Params p) {
  const GatedNormParams& g = p.g;
  if (g.mode_dev != nullptr && SIXBIT_MODE_OF(*g.mode_dev) != SIXBIT_MODE_INT8) return;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ Joint post, pre, top;
  const Vectors vec{reinterpret_cast<float4*>(smem), static_cast<int>(blockDim.x)};
  const int chunks = g.K / kChunk, nwarps = blockDim.x >> 5;
  const bool has_p = g.post_w != nullptr || g.gate != nullptr, has_w = g.w != nullptr || g.scale != nullptr;
  const bool has_t = g.shift != nullptr, late = !has_t && g.y == nullptr;  // late: the factor goes to the scale
  const float nan = __uint_as_float(0x7FC00000u);
  uint32_t xr[V][8], rr[V][8];
  int seg_next = 0;
  auto load = [&](int row) {
    seg_next = g.segment != nullptr ? __ldg(g.segment + row) : g.S > 1 ? row / g.rows_per_seg : 0;
    const size_t base = static_cast<size_t>(row) * g.K;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = threadIdx.x + v * blockDim.x;
#pragma unroll
      for (int i = 0; i < 8; ++i) xr[v][i] = rr[v][i] = 0;
      if (c < chunks) {
        load32(g.x + base + static_cast<size_t>(c) * kChunk, p.wide, xr[v]);
        if (g.res != nullptr) load32(g.res + base + static_cast<size_t>(c) * kChunk, p.wide, rr[v]);
      }
    }
  };
  auto join = [&](int seg) {
    const size_t mod = static_cast<size_t>(seg) * g.K;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = threadIdx.x + v * blockDim.x, k = c * kChunk;
      if (c >= chunks) continue;
      uint64_t a[8], b[8];
      if (has_p) {
        load16f(g.post_w != nullptr ? g.post_w + k : nullptr, 1.f, a);
        load16f(g.gate != nullptr ? g.gate + mod + k : nullptr, 1.f, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = f2_mul(a[i], b[i]);
        vec.put<V>(0, v, a);
      }
      if (has_w) {
        load16f(g.w != nullptr ? g.w + k : nullptr, 1.f, a);
        load16f(g.scale != nullptr ? g.scale + mod + k : nullptr, 0.f, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = f2_fma(a[i], b[i], a[i]);
        vec.put<V>(1, v, a);
      }
      if (has_t) {
        load16f(g.shift + mod + k, 0.f, a);
        vec.put<V>(2, v, a);
      }
    }
  };
  if (blockIdx.x < static_cast<unsigned>(g.M)) load(blockIdx.x);
  int buf = 0, held = -1;
  for (int row = blockIdx.x; row < g.M; row += gridDim.x, buf ^= 1) {
    const size_t base = static_cast<size_t>(row) * g.K;
    int seg = seg_next;
    const bool bad = seg < 0 || seg >= g.S;
    if (bad) {
      seg = 0;
      if (threadIdx.x == 0) set_error(g.err, SIXBIT_EDEVICE);
    }
    if (seg != held) join(seg);  // (a thread reads back what it wrote itself)
    held = seg;
    uint64_t u[V][8];
    float rpost = 1.f;
    uint64_t ss = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) u[v][i] = bad ? f2_pack(nan, nan) : f2_from_bf16x2(xr[v][i]);
    if (g.post_w != nullptr) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = f2_fma(u[v][i], u[v][i], ss);
      const float sum = cta_sum(f2_lo(ss) + f2_hi(ss), post, buf, nwarps);
      rpost = finite_sum(sum) ? rms_inv(sum, g.K, g.eps) : nan;
      ss = 0;
    }
    const uint64_t rp = f2_pack(rpost, rpost), rs = f2_pack(g.res_scale, g.res_scale);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = threadIdx.x + v * blockDim.x;
      if (c >= chunks) {
#pragma unroll
        for (int i = 0; i < 8; ++i) u[v][i] = 0;
        continue;
      }
      if (has_p) {
        uint64_t w[8];
        vec.get<V>(0, v, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[v][i] = f2_mul(f2_mul(u[v][i], rp), w[i]);
      }
      if (g.res != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) u[v][i] = f2_fma(f2_from_bf16x2(rr[v][i]), rs, u[v][i]);
      }
      if (g.sum_out != nullptr) {
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = f2_to_bf16x2(u[v][i]);
        store32(g.sum_out + base + static_cast<size_t>(c) * kChunk, p.wide, o);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = f2_fma(u[v][i], u[v][i], ss);
    }
    if (row + static_cast<int64_t>(gridDim.x) < g.M) load(row + gridDim.x);
    float sum = f2_lo(ss) + f2_hi(ss), rpre = 1.f;
    if (!late) {
      sum = cta_sum(sum, pre, buf, nwarps);
      rpre = finite_sum(sum) ? rms_inv(sum, g.K, g.eps) : nan;
    }
    const uint64_t r2 = f2_pack(rpre, rpre);
    uint32_t mb = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = threadIdx.x + v * blockDim.x;
      if (c < chunks) {
        uint64_t w[8];
        if (!late) {
#pragma unroll
          for (int i = 0; i < 8; ++i) u[v][i] = f2_mul(u[v][i], r2);
        }
        if (has_w) {
          vec.get<V>(1, v, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) u[v][i] = f2_mul(u[v][i], w[i]);
        }
        if (has_t) {
          vec.get<V>(2, v, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) u[v][i] = f2_add(u[v][i], w[i]);
        }
        if (g.y != nullptr) {
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = f2_to_bf16x2(u[v][i]);
          store32(g.y + base + static_cast<size_t>(c) * kChunk, p.wide, o);
        }
      }
      if (g.y == nullptr) {  // (every lane of the warp takes part)
        fwht<B>(u[v]);
        mb = max_bits(u[v], mb);
      }
    }
    if (g.y != nullptr) continue;
    mb = __reduce_max_sync(0xFFFFFFFFu, mb);
    if (late) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    }
    if (nwarps > 1) {
      if ((threadIdx.x & 31) == 0) {
        top.ss[buf][threadIdx.x >> 5] = sum;
        top.mx[buf][threadIdx.x >> 5] = mb;
      }
      __syncthreads();
      mb = 0;
      for (int i = 0; i < nwarps; ++i) mb = max(mb, top.mx[buf][i]);
      if (late) {
        sum = 0.f;
        for (int i = 0; i < nwarps; ++i) sum += top.ss[buf][i];
      }
    }
    const RowOut o = late ? row_out(rms_inv(sum, g.K, g.eps) * p.inv_sqrt_b, finite_sum(sum), mb)
                          : row_out(p.inv_sqrt_b, true, mb);
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
  const int smem = 3 * V * 64 * threads;
  int per_sm = 0;
  cudaError_t e = set_smem_once<row_kernel<B, V>>(3 * V * 64 * 512);
  if (e != cudaSuccess) return e;
  e = cache[threads / 32].get(&per_sm, [&](int* o) {
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(o, row_kernel<B, V>, threads, smem);
  });
  if (e != cudaSuccess) return e;
  const int most = sm_count() * (per_sm > 0 ? per_sm : 1);
  note_launch();
  row_kernel<B, V><<<p.g.M < most ? p.g.M : most, threads, smem, st>>>(p);
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
