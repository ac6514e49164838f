// W4A8 products of few rows: INT8 activation codes against INT4 weights with
// one scale per 128 inputs, for single tokens and for experts that got a few
// (technical summary sections 2.A and 4; the GEMM form is qgemm_w4a8.cu).
//
//   Y[m, n] = s_m[m] * sum_g s_w[g][n] * acc_g[m, n]
//   acc_g[m, n] = sum_{k in group g} qa[m, k] * qw[n, k]    (exact integers)
//
// With so few rows the call reads each weight byte once and multiplies it a few
// times, so they go straight from global memory to registers as INT4 and are
// never expanded in memory.  Measured, weights cold (a copy of their bytes would
// take 1.2, 3.0 and 3.1 us): one token, 7680 x 1920 4.3 us and 3072 x 12288
// 6.2 us, bound by the latencies of a launch, its loads and the join; 32 tokens,
// 12288 x 3072 17 us, bound by the conversions of codes and nibbles (the grouped
// product with one expert, whose CTAs convert weights only, takes 11.3 us there,
// but 24.6 against 22.4 for 3072 x 12288).
#include <cstdint>

#include "common.cuh"
#include "ctx_cache.h"
#include "gemm_common.cuh"
#include "internal.h"
#include "w4a8_common.cuh"

namespace sixbit {
namespace rows {

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The row's scale, the epilogue and the store of one output.
__device__ __forceinline__ void finish(const RowsParams& p, int row, int col, float y) {
  y = __fmul_rn(y, __ldg(p.row_scale + row));
  const size_t at = static_cast<size_t>(row) * p.N + col;
  if (p.epilogue == SIXBIT_EPI_GELU)
    y = f2_lo(gelu_pair(f2_pack(y, y)));
  else if (p.epilogue == SIXBIT_EPI_RESIDUAL)
    y = __fadd_rn(y, __uint_as_float(static_cast<uint32_t>(p.residual[at]) << 16));
  if (p.Yf != nullptr)
    p.Yf[at] = y;
  else
    p.Y[at] = static_cast<uint16_t>(f2_to_bf16x2(f2_pack(y, 0.f)) & 0xFFFFu);
}

// -------------------------------------------------------- one or two tokens --
// Four-byte dot products: a warp takes four weight rows by 1024 k, 16 bytes of
// nibbles a lane and row in one load each (a nibble stands in the upper half
// of its byte: 16 v).  A group's sum is joined over its four lanes as
// integers, exact, before the scale.  `split` warps share a row's chunks.
constexpr int kR = 4;         // weight rows of a warp
constexpr int kChunk = 1024;  // k of a warp's load

// Rows [first, first + count) of the expert blockIdx.y, T tokens at a time.
template <int T>
__device__ __forceinline__ void dot_rows(const RowsParams& p, int split, int first, int count, float* part) {
  constexpr int kV = kR * T;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wr = (blockDim.x >> 5) / split;  // row blocks of the CTA
  const int kw = warp % split, rw = warp / split;
  const int groups = p.K / 128, chunks = (p.K + kChunk - 1) / kChunk;
  const int nc = blockIdx.x * wr * kR, n0 = nc + rw * kR;
  const size_t kb = static_cast<size_t>(p.K) / 2;
  const uint8_t* w4 = p.w4 + static_cast<size_t>(blockIdx.y) * p.N * kb + lane * 16;
  const float* w4s = p.w4_scale + static_cast<size_t>(blockIdx.y) * groups * p.N;
  int n[kR];
#pragma unroll
  for (int r = 0; r < kR; ++r) n[r] = min(n0 + r, p.N - 1);  // (the surplus rows are not stored)

  for (int t0 = 0; t0 < count; t0 += T) {
    const int8_t* xrow[T];
#pragma unroll
    for (int j = 0; j < T; ++j) xrow[j] = p.codes + static_cast<size_t>(first + min(t0 + j, count - 1)) * p.K + lane * 32;
    float v[T];  // of row n0 + lane % 4, this lane's groups (lane / 4 and every eighth after it)
#pragma unroll
    for (int j = 0; j < T; ++j) v[j] = 0.f;
    for (int c = kw; c < chunks; c += split) {
      const int gr = c * 8 + (lane >> 2);
      const bool live = gr < groups;
      uint4 w[kR], x[T][2];
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        w[r] = make_uint4(0, 0, 0, 0);
        if (live) w[r] = __ldg(reinterpret_cast<const uint4*>(w4 + n[r] * kb + static_cast<size_t>(c) * 512));
      }
#pragma unroll
      for (int j = 0; j < T; ++j) {
        x[j][0] = x[j][1] = make_uint4(0, 0, 0, 0);
        if (live) {
          const uint4* xp = reinterpret_cast<const uint4*>(xrow[j] + c * kChunk);
          x[j][0] = __ldg(xp);
          x[j][1] = __ldg(xp + 1);
        }
      }
      // (a nibble stands 4 bits up in its byte: 1 / 16)
      const float s = live ? __ldg(w4s + static_cast<size_t>(gr) * p.N + min(n0 + (lane & 3), p.N - 1)) * 0.0625f : 0.f;
      // codes: even k in one word, odd k in the other, as the two nibbles of a byte stand
      uint32_t e[T][4], o[T][4];
#pragma unroll
      for (int j = 0; j < T; ++j) {
        const uint32_t q[8] = {x[j][0].x, x[j][0].y, x[j][0].z, x[j][0].w, x[j][1].x, x[j][1].y, x[j][1].z, x[j][1].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[j][i] = __byte_perm(q[2 * i], q[2 * i + 1], 0x6420);
          o[j][i] = __byte_perm(q[2 * i], q[2 * i + 1], 0x7531);
        }
      }
      int acc[T][kR];
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        const uint32_t q[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
#pragma unroll
        for (int j = 0; j < T; ++j) acc[j][r] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int we = static_cast<int>((q[i] << 4) & 0xF0F0F0F0u), wo = static_cast<int>(q[i] & 0xF0F0F0F0u);
#pragma unroll
          for (int j = 0; j < T; ++j) {
            acc[j][r] = __dp4a(we, static_cast<int>(e[j][i]), acc[j][r]);
            acc[j][r] = __dp4a(wo, static_cast<int>(o[j][i]), acc[j][r]);
          }
        }
      }
      // The group's sum over its four lanes, exact, row lane % 4 to each lane.
      const bool up2 = (lane & 2) != 0, up1 = (lane & 1) != 0;
#pragma unroll
      for (int j = 0; j < T; ++j) {
        int a[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          a[i] = (up2 ? acc[j][i + 2] : acc[j][i]) + __shfl_xor_sync(0xFFFFFFFFu, up2 ? acc[j][i] : acc[j][i + 2], 2);
        const int sum = (up1 ? a[1] : a[0]) + __shfl_xor_sync(0xFFFFFFFFu, up1 ? a[0] : a[1], 1);
        v[j] = fmaf(s, static_cast<float>(sum), v[j]);
      }
    }
    // Sum over the eight groups: while more than one token is left, a lane
    // hands half of them to its partner and keeps the other half.
    int o = 16;
#pragma unroll
    for (int m = T; m > 1; m >>= 1, o >>= 1) {
      const bool up = (lane & o) != 0;
#pragma unroll
      for (int i = 0; i < m / 2; ++i) {
        const float send = up ? v[i] : v[i + m / 2], keep = up ? v[i + m / 2] : v[i];
        v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, o);
      }
    }
#pragma unroll
    for (; o > 2; o >>= 1) v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
    if (lane % (32 / T) < kR) part[warp * kV + lane / (32 / T) * kR + (lane & 3)] = v[0];
    __syncthreads();
    const int width = wr * kR;
    for (int i = threadIdx.x; i < width * T; i += blockDim.x) {
      const int j = i / width, c = i % width;
      if (t0 + j < count && nc + c < p.N) {
        float y = 0.f;
        for (int k = 0; k < split; ++k) y += part[((c / kR) * split + k) * kV + j * kR + c % kR];
        finish(p, first + t0 + j, nc + c, y);
      }
    }
    if (t0 + T < count) __syncthreads();
  }
}

// T tokens at a time; T = 0: one or two, by the expert's own count.
template <int T>
__global__ void __launch_bounds__(256) dot_kernel(const RowsParams p, int split) {
  if (p.mode_dev != nullptr && SIXBIT_MODE_OF(*p.mode_dev) != SIXBIT_MODE_INT8) return;
  __shared__ float part[8 * kR * (T > 0 ? T : 2)];
  int first, count;
  expert_rows(p, blockIdx.y, threadIdx.x == 0, &first, &count);
  if (count == 0) return;
  if constexpr (T > 0)
    dot_rows<T>(p, split, first, count, part);
  else if (count == 1)
    dot_rows<1>(p, split, first, count, part);
  else
    dot_rows<2>(p, split, first, count, part);
}

cudaError_t launch_dot(const RowsParams& p, cudaStream_t st) {
  const int chunks = (p.K + kChunk - 1) / kChunk;
  const int turns = (chunks + 7) / 8, split = (chunks + turns - 1) / turns, wr = 8 / split;
  const dim3 grid((p.N + wr * kR - 1) / (wr * kR), p.E);
  const int threads = split * wr * 32;
  if (p.offsets != nullptr)
    dot_kernel<0><<<grid, threads, 0, st>>>(p, split);
  else if (p.M == 1)
    dot_kernel<1><<<grid, threads, 0, st>>>(p, split);
  else
    dot_kernel<2><<<grid, threads, 0, st>>>(p, split);
  note_launch();
  return cudaGetLastError();
}

// ------------------------------------------------------ three to 32 tokens --
// The products run on mma.m16n8k16 with fp16 operands and FP32 accumulation:
// weight rows are the 16-row operand (MT of them), tokens the 8-column one (NT
// tiles).  Codes and nibbles are exact in fp16 and a group's sum stays below
// 2^17, so the accumulator holds the exact integer; the scale is applied after
// each group.  (The other integer forms lose: s8 MMAs take 64 cycles on this
// part for 8 of the fp16 one at half the k, and E4M3 ones, with both digits of
// a code, measured 38 us against 20 at 32 tokens, 12288 x 3072.)  The sum over
// k may be taken in any order as long as both operands agree, so a lane keeps
// 32 consecutive k of a group (16 bytes of nibbles, 32 code bytes) and hands
// four of them to each MMA; within a word of eight nibbles the pairs are
// (k, k + 4), the two halves of one masked word.
//
// A CTA owns 16 MT weight rows and its W warps split the groups of K (the next
// group's nibbles are loaded while this one's are multiplied); their FP32 sums
// meet in shared memory in a fixed order, where the epilogue runs.  The
// conversions bound it from 16 tokens on (integer instructions issue every
// second cycle): per 16 rows, 16 k and eight tokens the MMA takes 8 cycles, the
// codes 10, the nibbles 18 shared by all tokens.
template <int MT, int NT, int W>
__global__ void __launch_bounds__(W * 32, MT > 1 ? 3 : (NT == 1 ? 32 : NT == 2 ? 24 : 16) / W) tile_kernel(const RowsParams p) {
  if (p.mode_dev != nullptr && SIXBIT_MODE_OF(*p.mode_dev) != SIXBIT_MODE_INT8) return;
  constexpr int kT = 8 * NT, kN = 16 * MT;
  __shared__ float part[W][kT][kN + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int groups = p.K / 128, n0 = blockIdx.x * kN;
  const size_t kb = static_cast<size_t>(p.K) / 2;
  int n[2 * MT];
  const uint8_t* wrow[2 * MT];
#pragma unroll
  for (int h = 0; h < 2 * MT; ++h) {
    n[h] = min(n0 + 8 * h + g, p.N - 1);  // (the surplus rows are not stored)
    wrow[h] = p.w4 + n[h] * kb + t * 16;
  }
  const int8_t* xrow = p.codes + static_cast<size_t>(g) * p.K + t * 32;
  float sum[MT][NT][4] = {};

  uint4 w[2 * MT];
  float sc[2 * MT];
  auto fetch = [&](int gr) {
#pragma unroll
    for (int h = 0; h < 2 * MT; ++h) {
      w[h] = __ldg(reinterpret_cast<const uint4*>(wrow[h] + static_cast<size_t>(gr) * 64));
      sc[h] = __ldg(p.w4_scale + static_cast<size_t>(gr) * p.N + n[h]);
    }
  };
  if (warp < groups) fetch(warp);
  for (int gr = warp; gr < groups; gr += W) {
    uint4 wc[2 * MT];
    float s[2 * MT];
#pragma unroll
    for (int h = 0; h < 2 * MT; ++h) {
      wc[h] = w[h];
      s[h] = sc[h];
    }
    uint4 x[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      x[j][0] = x[j][1] = make_uint4(0, 0, 0, 0);
      if (8 * j + g < p.M) {  // (a surplus token's column is not stored)
        const uint4* xp = reinterpret_cast<const uint4*>(xrow + static_cast<size_t>(8 * j) * p.K + gr * 128);
        x[j][0] = __ldg(xp);
        x[j][1] = __ldg(xp + 1);
      }
    }
    if (gr + W < groups) fetch(gr + W);
    float acc[MT][NT][4] = {};
#pragma unroll
    for (int q = 0; q < 4; ++q) {  // eight k of the lane
      uint32_t a0[MT][4], a1[MT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint32_t lo[4], hi[4];
        nibbles_f16(word(wc[2 * m], q), lo);
        nibbles_f16(word(wc[2 * m + 1], q), hi);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          a0[m][2 * i] = lo[i];
          a0[m][2 * i + 1] = hi[i];
          a1[m][2 * i] = lo[2 + i];
          a1[m][2 * i + 1] = hi[2 + i];
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint32_t b[4];
        codes_f16(word(x[j][q >> 1], 2 * (q & 1)), word(x[j][q >> 1], 2 * (q & 1) + 1), b);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          mma16816(acc[m][j], a0[m], b[0], b[1]);
          mma16816(acc[m][j], a1[m], b[2], b[3]);
        }
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[m][j][i] = fmaf(s[2 * m + (i >> 1)], acc[m][j][i], sum[m][j][i]);
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[warp][8 * j + 2 * t + (i & 1)][16 * m + 8 * (i >> 1) + g] = sum[m][j][i];
  __syncthreads();
  for (int i = threadIdx.x; i < kT * kN; i += W * 32) {
    const int tok = i / kN, c = i % kN;
    if (tok >= p.M || n0 + c >= p.N) continue;
    float y = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) y += part[k][tok][c];
    finish(p, tok, n0 + c, y);
  }
}

template <int MT, int NT, int W>
cudaError_t launch_tile(const RowsParams& p, cudaStream_t st) {
  tile_kernel<MT, NT, W><<<(p.N + 16 * MT - 1) / (16 * MT), W * 32, 0, st>>>(p);
  note_launch();
  return cudaGetLastError();
}

// Sixteen warps a CTA where K has groups for them and every CTA is resident
// at once (two of them an SM with one token tile, one with two), else eight:
// 8 tokens, 1920 x 7680 weights 10.7 -> 6.9 us, 3072 x 12288 15.0 -> 10.9, but
// 5760 x 1920 4.7 -> 5.6 and 16 tokens, 3072 x 12288 17.1 -> 18.8.  Above 16
// tokens and with more 16-row tiles than four an SM, a warp takes two of them
// for each conversion of the codes, four warps a CTA: 32 tokens, 12288 x 3072
// 19.6 -> 16.5 us, though that form spills 76 bytes a thread, but 5760 x 1920
// 9.4 -> 10.6 and 3072 x 12288 22 -> 44.
cudaError_t launch_tiles(const RowsParams& p, cudaStream_t st) {
  const int tiles = (p.N + 15) / 16;
  const bool deep = p.K > 16 * 128;
  if (p.M <= 8) return deep && tiles <= 2 * sm_count() ? launch_tile<1, 1, 16>(p, st) : launch_tile<1, 1, 8>(p, st);
  if (p.M <= 16) return deep && tiles <= sm_count() ? launch_tile<1, 2, 16>(p, st) : launch_tile<1, 2, 8>(p, st);
  if (tiles > 4 * sm_count()) return p.M <= 24 ? launch_tile<2, 3, 4>(p, st) : launch_tile<2, 4, 4>(p, st);
  return p.M <= 24 ? launch_tile<1, 3, 8>(p, st) : launch_tile<1, 4, 8>(p, st);
}

}  // namespace rows

// One weight (up to 32 rows): dot products up to two rows, MMAs above (two
// tokens, 7680 x 1920: 4.7 us, where MMAs take 5.1 for three and 5.3 for eight;
// 3072 x 12288 6.9 against 10.6).  Experts: any rows, one or two at a time.
cudaError_t launch_w4a8_rows(const RowsParams& p, cudaStream_t st) {
  return p.offsets != nullptr || p.M <= 2 ? rows::launch_dot(p, st) : rows::launch_tiles(p, st);
}

}  // namespace sixbit
