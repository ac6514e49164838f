// Residual add + root-mean-square norm + block-Hadamard rotation + per-token
// INT8 quantization in one pass: what stands between two quantized layers of a
// transformer block and feeds the W4A8 products (technical summary sections
// 2.A and 4: the quantization is fused with the work around it).
//
//   h = x + r                                 (r optional; sum_out = bf16(h))
//   z = (h . rinv . w) . blockdiag(H_b / sqrt b),  rinv = 1 / sqrt(mean h^2 + eps)
//   s = max|z| / 127,  q = rint(z / s)
//
// The row's factor rinv / sqrt b multiplies every z of the row, so it drops
// out of q: with u = (h . w) . blockdiag(H_b unscaled) and a = max|u|,
//   q = rint(u . 127 / a),   s = a . rinv / sqrt b / 127.
// The sum of squares and the maximum are therefore one reduction with one
// barrier, and u stays in registers from the load to the code store: the row
// is read once and written once.  All of it is FP32 (sum_out is the only
// rounding to bf16; the norm uses the unrounded h); the quotient's rounding is
// one FMA onto 1.5 * 2^23, whose low byte is the code.
//
// Each thread holds chunks of 16 consecutive elements, 32 bytes of bf16: one
// 256-bit load per operand, one 256-bit store of the sum and one 16-byte store
// of the codes, all contiguous across the warp.  The butterfly strides 1..8
// stay in the thread (packed f32x2), 16 and up go across lanes (2 shuffle
// stages for b = 64, 4 for b = 256).
//
// The floor is bytes: 7 an element with a residual, 3 without.  17,776 rows of
// 1920 with a residual 40.5 us (5.9 TB/s, 88% of a copy), of 12288 69 us (4,444
// rows); one row 2.0 us, 226 rows 2.7 us (a launch and two round trips); 1,003
// rows of 7680 without a residual 7.4 us (floor 3.5: registers hold the one row
// in flight of each of two CTAs an SM); 2,000 of 16640, computed twice, 91 us
// (floor 35).
#include <cstdint>

#include "common.cuh"
#include "ctx_cache.h"
#include "internal.h"
#include "row_norm.cuh"

namespace sixbit {
namespace arq {

struct Params {
  const uint16_t* x;
  const uint16_t* res;   // or NULL
  const float* w;        // or NULL
  uint16_t* sum_out;     // or NULL
  int8_t* codes;
  float* row_scale;
  const int32_t* mode_dev;
  int M, K;
  float eps, inv_sqrt_b;
  int wide;              // x, res, sum_out are 32-byte aligned
  int team_log;          // warp form: lanes of one row = 1 << team_log
};

constexpr int kWarpThreads = 128;  // CTA of the warp form

// h = x + r of one chunk (into u) and its contribution to the sum of squares;
// the bf16 sum is stored when `put`.
__device__ __forceinline__ void add(const Params& p, size_t at, bool live, bool put, const uint32_t (&xr)[8],
                                    const uint32_t (&rr)[8], uint64_t& ss, uint64_t (&u)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = f2_from_bf16x2(xr[i]);
  if (p.res != nullptr) {
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      u[i] = f2_add(u[i], f2_from_bf16x2(rr[i]));
      o[i] = f2_to_bf16x2(u[i]);
    }
    if (live && put && p.sum_out != nullptr) store32(p.sum_out + at, p.wide, o);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = f2_fma(u[i], u[i], ss);
}

// A CTA takes whole rows, every gridDim-th one, V chunks a thread, kept in
// registers; the thread's weights stay there too, and the next row's loads are
// in flight while this one is rotated, reduced and stored.  (One CTA per row,
// which read the weights again for each row, was bound by L1: 17776 x 1920
// 47.2 us.)  V = 0: any K, each chunk computed twice (the second time the row
// comes from L2).
template <int B, int V>
__global__ void __launch_bounds__(512) row_kernel(const Params p) {
  if (p.mode_dev != nullptr && SIXBIT_MODE_OF(*p.mode_dev) != SIXBIT_MODE_INT8) return;
  __shared__ float s_ss[2][16];
  __shared__ uint32_t s_mx[2][16];
  constexpr int R = V > 0 ? V : 1;
  constexpr bool kKeep = V > 0;  // weights in registers
  const int chunks = p.K / kChunk;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
  const int loops = V > 0 ? 1 : (chunks + blockDim.x - 1) / blockDim.x;
  uint64_t w[kKeep ? R : 1][8];
  uint32_t xr[R][8], rr[R][8];
  auto at_of = [&](int row, int c) { return static_cast<size_t>(row) * p.K + static_cast<size_t>(c) * kChunk; };
  auto load = [&](int row, int it) {
#pragma unroll
    for (int v = 0; v < R; ++v) {
      const int c = threadIdx.x + (it + v) * blockDim.x;
#pragma unroll
      for (int i = 0; i < 8; ++i) xr[v][i] = rr[v][i] = 0;
      if (c < chunks) {
        load32(p.x + at_of(row, c), p.wide, xr[v]);
        if (p.res != nullptr) load32(p.res + at_of(row, c), p.wide, rr[v]);
      }
    }
  };
  if constexpr (kKeep) {
#pragma unroll
    for (int v = 0; v < R; ++v) {
      const int c = threadIdx.x + v * blockDim.x;
      load_weights(p.w, c * kChunk, c < chunks, w[v]);
    }
  }
  auto rotate = [&](int v, int c, uint64_t (&u)[8]) {
    if constexpr (!kKeep) load_weights(p.w, c * kChunk, c < chunks, w[0]);
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = f2_mul(u[i], w[kKeep ? v : 0][i]);
    fwht<B>(u);
  };
  if (V > 0) load(blockIdx.x, 0);
  int buf = 0;
  for (int row = blockIdx.x; row < p.M; row += gridDim.x, buf ^= 1) {
    uint64_t u[R][8], ss2 = 0;
    uint32_t mb = 0;
    for (int it = 0; it < loops; ++it) {
      if (V == 0) load(row, it);
#pragma unroll
      for (int v = 0; v < R; ++v) {
        const int c = threadIdx.x + (it + v) * blockDim.x;
        add(p, at_of(row, c), c < chunks, V > 0, xr[v], rr[v], ss2, u[v]);
      }
      if (V > 0 && row + gridDim.x < p.M) load(row + gridDim.x, 0);
#pragma unroll
      for (int v = 0; v < R; ++v) {
        rotate(v, threadIdx.x + (it + v) * blockDim.x, u[v]);
        mb = max_bits(u[v], mb);
      }
    }
    float ss = f2_lo(ss2) + f2_hi(ss2);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    mb = __reduce_max_sync(0xFFFFFFFFu, mb);
    if (nwarps > 1) {
      if (lane == 0) {
        s_ss[buf][warp] = ss;
        s_mx[buf][warp] = mb;
      }
      __syncthreads();  // (two buffers: the next row's writes need no barrier of their own)
      ss = 0.f;
      mb = 0;
      for (int i = 0; i < nwarps; ++i) {
        ss += s_ss[buf][i];
        mb = max(mb, s_mx[buf][i]);
      }
    }
    const RowOut o = row_out(rms_inv(ss, p.K, p.eps) * p.inv_sqrt_b, finite_sum(ss), mb);
    if (threadIdx.x == 0) p.row_scale[row] = o.scale;
    for (int it = 0; it < loops; ++it) {
#pragma unroll
      for (int v = 0; v < R; ++v) {
        const int c = threadIdx.x + (it + v) * blockDim.x;
        if constexpr (V == 0) {
          load(row, it);
          uint64_t unused = 0;
          add(p, at_of(row, c), c < chunks, true, xr[v], rr[v], unused, u[v]);
          rotate(v, c, u[v]);
        }
        if (c < chunks) store_codes(p.codes + at_of(row, c), o, u[v]);
      }
    }
  }
}

// K <= 512: 1 << team_log lanes of a warp per row, no barrier.
template <int B>
__global__ void __launch_bounds__(kWarpThreads) team_kernel(const Params p) {
  if (p.mode_dev != nullptr && SIXBIT_MODE_OF(*p.mode_dev) != SIXBIT_MODE_INT8) return;
  const int team = 1 << p.team_log;
  const int t = threadIdx.x & (team - 1);
  const int64_t row = blockIdx.x * static_cast<int64_t>(kWarpThreads >> p.team_log) + (threadIdx.x >> p.team_log);
  const bool live = row < p.M && t < p.K / kChunk;
  const size_t at = static_cast<size_t>(row) * p.K + t * kChunk;
  uint32_t xr[8], rr[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) xr[i] = rr[i] = 0;
  if (live) {
    load32(p.x + at, p.wide, xr);
    if (p.res != nullptr) load32(p.res + at, p.wide, rr);
  }
  uint64_t u[8], w[8], ss2 = 0;
  add(p, at, live, true, xr, rr, ss2, u);
  load_weights(p.w, t * kChunk, live, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = f2_mul(u[i], w[i]);
  fwht<B>(u);
  uint32_t mb = max_bits(u, 0);
  float ss = f2_lo(ss2) + f2_hi(ss2);
  for (int o = team >> 1; o > 0; o >>= 1) {
    ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    mb = max(mb, __shfl_xor_sync(0xFFFFFFFFu, mb, o));
  }
  const RowOut o = row_out(rms_inv(ss, p.K, p.eps) * p.inv_sqrt_b, finite_sum(ss), mb);
  if (live && t == 0) p.row_scale[row] = o.scale;
  if (live) store_codes(p.codes + at, o, u);
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
  row_kernel<B, V><<<p.M < most ? p.M : most, threads, 0, st>>>(p);
  return cudaGetLastError();
}

template <int B>
cudaError_t launch(Params& p, cudaStream_t st) {
  const int chunks = p.K / kChunk;
  note_launch();
  if (chunks <= 32) {
    p.team_log = chunks <= 8 ? 3 : chunks <= 16 ? 4 : 5;
    const int rows = kWarpThreads >> p.team_log;
    team_kernel<B><<<(p.M + rows - 1) / rows, kWarpThreads, 0, st>>>(p);
    return cudaGetLastError();
  }
  // one chunk a thread up to K = 4096, two up to 16384 (four spill: 4444 x
  // 12288 119.7 us)
  const int v = chunks <= 256 ? 1 : 2;
  const int threads = ((chunks + v - 1) / v + 31) / 32 * 32;
  if (threads > 512) return launch_rows<B, 0>(p, 512, st);
  return v == 1 ? launch_rows<B, 1>(p, threads, st) : launch_rows<B, 2>(p, threads, st);
}

}  // namespace arq

cudaError_t launch_add_rmsnorm_quant(const uint16_t* x, const uint16_t* res, const float* w, int M, int K, float eps,
                                     int b, const int32_t* mode_dev, uint16_t* sum_out, int8_t* codes,
                                     float* row_scale, cudaStream_t st) {
  arq::Params p{};
  p.x = x;
  p.res = res;
  p.w = w;
  p.sum_out = sum_out;
  p.codes = codes;
  p.row_scale = row_scale;
  p.mode_dev = mode_dev;
  p.M = M;
  p.K = K;
  p.eps = eps;
  p.inv_sqrt_b = b == 16 ? 0.25f : b == 64 ? 0.125f : b == 256 ? 0.0625f : 1.f;
  const auto a32 = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 31u) == 0; };
  p.wide = a32(x) && a32(res) && a32(sum_out);
  switch (b) {
    case 16: return arq::launch<16>(p, st);
    case 64: return arq::launch<64>(p, st);
    case 256: return arq::launch<256>(p, st);
    default: return arq::launch<0>(p, st);
  }
}

}  // namespace sixbit
