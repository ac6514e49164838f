// Low-rank adapters of many requests beside one shared projection:
//
//   y[m] = epilogue(base[m] + alpha_l . B_l (A_l x_m)),   l = ids[m]  (-1: base alone)
//
// x: INT8 codes with a scale per row (rotated, as the W4A8 products read them;
// A_l is rotated when it is packed) or bf16.  A_l [R, K] and B_l [N, R] bf16.
//
// Two kernels: v = A_l x (sums over K, FP32, to the workspace), then the product
// with B_l on top of the base and its epilogue.  Both run on mma.m16n8k16 with
// bf16 operands and FP32 sums, rows as the 16-row operand; 32 rows are one tile,
// and a tile's rows are taken adapter by adapter: __match_any_sync finds the rows
// of one, and they fill the MMA's rows however they lie.  Codes are exact in
// bf16.  v enters the second product as two bf16 parts (v to 2^-16, three parts
// and 2^-24 where the result is FP32): one part alone would add an error as large
// as the output's own rounding.
#include <cstdint>

#include "common.cuh"
#include "ctx_cache.h"
#include "gemm_common.cuh"
#include "internal.h"

namespace sixbit {
namespace lowrank {

constexpr int kTile = 32;   // rows of a tile
constexpr int kWarps = 8;
constexpr int kUnit = 64;   // k of a warp's turn
constexpr unsigned kAll = 0xFFFFFFFFu;

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two s8 codes (bytes 0 and 2 of w) as bf16, exact: 128 + the low seven bits, less
// 128, or 256 where the sign bit is set.
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w) {
  const uint32_t a = (w & 0x007F007Fu) | 0x43004300u, b = (w & 0x00800080u) | 0x43004300u;
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) { return f2_to_bf16x2(f2_pack(lo, hi)); }

// What a part leaves of v: nothing of an infinity or a NaN, which the part holds.
__device__ __forceinline__ float rest(float v, uint32_t part) {
  const float r = v - __uint_as_float(part);
  return fabsf(r) < INFINITY ? r : 0.f;
}

// The rows of a tile by adapter.  Lane i holds row i's adapter (-1: none).
struct Groups {
  int id;            // this lane's row's
  uint32_t same;     // rows of the same adapter
  uint32_t leaders;  // the first row of each
};
__device__ __forceinline__ Groups groups_of(const LowRankParams& p, int64_t row0, bool none_too, bool report) {
  const int lane = threadIdx.x & 31;
  Groups g;
  int id = -2;  // (beyond the last row)
  if (row0 + lane < p.M) {
    id = __ldg(p.ids + row0 + lane);
    if (id < 0 || id >= p.L) {
      if (id != -1 && report) set_error(p.err, SIXBIT_EDEVICE);
      id = -1;
    }
  }
  g.id = id;
  g.same = __match_any_sync(kAll, id);
  g.leaders = __ballot_sync(kAll, id >= (none_too ? -1 : 0) && lane == __ffs(g.same) - 1);
  return g;
}
// Row numbers of the group that `leader` leads, in list[0 .. its count): the count.
__device__ __forceinline__ int rows_of(const Groups& g, int leader, uint8_t* list, int* id) {
  const int lane = threadIdx.x & 31;
  const uint32_t rows = __shfl_sync(kAll, g.same, leader);
  *id = __shfl_sync(kAll, g.id, leader);
  __syncwarp();
  if ((rows >> lane) & 1) list[__popc(rows & ((1u << lane) - 1))] = static_cast<uint8_t>(lane);
  __syncwarp();
  return __popc(rows);
}

// v [splits][M][R] = A_l x.  Grid: tiles x slots x splits; slot s takes a tile's
// groups s, s + slots, ...; the CTA's warps share the split's part of K, and their
// sums meet in shared memory in a fixed order.  RT: tiles of eight ranks at a time.
template <bool INT8, int RT>
__global__ void __launch_bounds__(kWarps * 32) shrink_kernel(const LowRankParams p) {
  if (p.mode_dev != nullptr && SIXBIT_MODE_OF(*p.mode_dev) != SIXBIT_MODE_INT8) return;
  extern __shared__ float part[];  // [kWarps][kTile][8 RT + 1]
  __shared__ uint8_t lists[kWarps][kTile];
  constexpr int kP = 8 * RT + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, q = lane & 3;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const Groups groups = groups_of(p, row0, false, blockIdx.y == 0 && blockIdx.z == 0 && warp == 0);
  uint32_t left = groups.leaders;
  for (int turn = 0; left != 0; ++turn, left &= left - 1) {
    if (turn % gridDim.y != blockIdx.y) continue;
    int id;
    const int count = rows_of(groups, __ffs(left) - 1, lists[warp], &id);
    size_t at[4];
    bool live[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      live[i] = g8 + 8 * i < count;
      at[i] = static_cast<size_t>(row0 + (live[i] ? lists[warp][g8 + 8 * i] : 0)) * p.K;
    }
    for (int r0 = 0; r0 < p.R; r0 += 8 * RT) {
      const int tiles = min(RT, (p.R - r0) / 8);
      const uint16_t* a = p.a + (static_cast<size_t>(id) * p.R + r0 + g8) * p.K;
      float acc[2][RT][4] = {};
      for (int u = blockIdx.z * kWarps + warp; u < p.K / kUnit; u += gridDim.z * kWarps) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // 32 k; a lane keeps eight of them, four for each MMA
          const int k = u * kUnit + 32 * h + 8 * q;
          uint4 b[RT];
#pragma unroll
          for (int j = 0; j < RT; ++j)
            if (j < tiles) b[j] = __ldg(reinterpret_cast<const uint4*>(a + static_cast<size_t>(8 * j) * p.K + k));
          uint32_t x[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0;
            if (live[i]) {
              if constexpr (INT8) {
                const uint2 w = __ldg(reinterpret_cast<const uint2*>(p.codes + at[i] + k));
                x[i][0] = codes_bf16(__byte_perm(w.x, 0, 0x4140));
                x[i][1] = codes_bf16(__byte_perm(w.x, 0, 0x4342));
                x[i][2] = codes_bf16(__byte_perm(w.y, 0, 0x4140));
                x[i][3] = codes_bf16(__byte_perm(w.y, 0, 0x4342));
              } else {
                const uint4 w = __ldg(reinterpret_cast<const uint4*>(p.x + at[i] + k));
                x[i][0] = w.x, x[i][1] = w.y, x[i][2] = w.z, x[i][3] = w.w;
              }
            }
          }
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            if (m == 1 && count <= 16) break;
            const uint32_t a0[4] = {x[2 * m][0], x[2 * m + 1][0], x[2 * m][1], x[2 * m + 1][1]};
            const uint32_t a1[4] = {x[2 * m][2], x[2 * m + 1][2], x[2 * m][3], x[2 * m + 1][3]};
#pragma unroll
            for (int j = 0; j < RT; ++j)
              if (j < tiles) {
                mma(acc[m][j], a0, b[j].x, b[j].y);
                mma(acc[m][j], a1, b[j].z, b[j].w);
              }
          }
        }
      }
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < RT; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            part[(warp * kTile + 16 * m + 8 * (i >> 1) + g8) * kP + 8 * j + 2 * q + (i & 1)] = acc[m][j][i];
      __syncthreads();
      const int width = 8 * tiles;
      for (int i = threadIdx.x; i < count * width; i += kWarps * 32) {
        const int row = i / width, r = i % width;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += part[(w * kTile + row) * kP + r];
        p.v[(static_cast<size_t>(blockIdx.z) * p.M + row0 + lists[warp][row]) * p.R + r0 + r] = v;
      }
      __syncthreads();
    }
  }
}

// Eight consecutive outputs of one row from column n on: base, epilogue, store.
template <bool VEC>
__device__ __forceinline__ void finish(const LowRankParams& p, int64_t row, int n, float (&v)[8]) {
  const size_t at = static_cast<size_t>(row) * p.N + n;
  if constexpr (VEC) {
    if (n >= p.N) return;
    if (p.base_f32 != nullptr) {
      const float4 a = reinterpret_cast<const float4*>(p.base_f32 + at)[0];
      const float4 b = reinterpret_cast<const float4*>(p.base_f32 + at)[1];
      v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w, v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
    } else if (p.base != nullptr) {
      const uint4 a = *reinterpret_cast<const uint4*>(p.base + at);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] += __uint_as_float(w[i] << 16);
        v[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
    if (p.epilogue == SIXBIT_EPI_GELU) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t g = gelu_pair(f2_pack(v[2 * i], v[2 * i + 1]));
        v[2 * i] = f2_lo(g);
        v[2 * i + 1] = f2_hi(g);
      }
    } else if (p.epilogue == SIXBIT_EPI_RESIDUAL) {
      const uint4 a = *reinterpret_cast<const uint4*>(p.residual + at);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] += __uint_as_float(w[i] << 16);
        v[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
    if (p.Yf != nullptr) {
      reinterpret_cast<float4*>(p.Yf + at)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(p.Yf + at)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *reinterpret_cast<uint4*>(p.Y + at) =
          make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (n + i >= p.N) return;
      float y = v[i];
      if (p.base_f32 != nullptr) y += p.base_f32[at + i];
      if (p.base != nullptr) y += __uint_as_float(static_cast<uint32_t>(p.base[at + i]) << 16);
      if (p.epilogue == SIXBIT_EPI_GELU) y = f2_lo(gelu_pair(f2_pack(y, y)));
      if (p.epilogue == SIXBIT_EPI_RESIDUAL) y += __uint_as_float(static_cast<uint32_t>(p.residual[at + i]) << 16);
      if (p.Yf != nullptr)
        p.Yf[at + i] = y;
      else
        p.Y[at + i] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
    }
  }
}

// One group's rows times B_l, 32 columns from n0 on.  Ranks and columns may stand
// in any order as long as the operands agree: a lane keeps four consecutive ranks
// of an MMA's 16, and column c of MMA j stands for n0 + 8 (c / 2) + 2 j + c % 2,
// so that a lane ends up with eight consecutive outputs of each of its rows.
template <bool VEC, int PARTS>
__device__ __forceinline__ void expand_group(const LowRankParams& p, int64_t row0, int n0, int id, int count,
                                             const uint8_t* list) {
  const int lane = threadIdx.x & 31, g8 = lane >> 2, q = lane & 3;
  int64_t row[4];
  bool live[4];
  float f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    live[i] = g8 + 8 * i < count;
    row[i] = row0 + (live[i] ? list[g8 + 8 * i] : 0);
    f[i] = 0.f;
    if (id >= 0 && live[i])
      f[i] = (p.row_scale != nullptr ? __ldg(p.row_scale + row[i]) : 1.f) * (p.alpha != nullptr ? __ldg(p.alpha + id) : 1.f);
  }
  float acc[2][4][4] = {};
  if (id >= 0) {
    const uint16_t* bl = p.b + static_cast<size_t>(id) * p.N * p.R;
    for (int r = 0; r < p.R; r += 16) {
      uint2 b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + 8 * (g8 >> 1) + 2 * j + (g8 & 1);
        b[j] = make_uint2(0, 0);
        if (n < p.N) b[j] = __ldg(reinterpret_cast<const uint2*>(bl + static_cast<size_t>(n) * p.R + r + 4 * q));
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        if (m == 1 && count <= 16) break;
        uint32_t a[PARTS][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float v[4] = {};
          if (live[2 * m + i])
            for (int s = 0; s < p.splits; ++s) {
              const float4 t = *reinterpret_cast<const float4*>(
                  p.v + (static_cast<size_t>(s) * p.M + row[2 * m + i]) * p.R + r + 4 * q);
              v[0] += t.x, v[1] += t.y, v[2] += t.z, v[3] += t.w;
            }
#pragma unroll
          for (int c = 0; c < 4; ++c) v[c] *= f[2 * m + i];
#pragma unroll
          for (int s = 0; s < PARTS; ++s) {
            a[s][i] = pack_bf16(v[0], v[1]);
            a[s][2 + i] = pack_bf16(v[2], v[3]);
            v[0] = rest(v[0], a[s][i] << 16), v[1] = rest(v[1], a[s][i] & 0xFFFF0000u);
            v[2] = rest(v[2], a[s][2 + i] << 16), v[3] = rest(v[3], a[s][2 + i] & 0xFFFF0000u);
          }
        }
#pragma unroll
        for (int s = PARTS - 1; s >= 0; --s)
#pragma unroll
          for (int j = 0; j < 4; ++j) mma(acc[m][j], a[s], b[j].x, b[j].y);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (!live[i]) continue;
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = acc[i >> 1][j][2 * (i & 1)];
      v[2 * j + 1] = acc[i >> 1][j][2 * (i & 1) + 1];
    }
    finish<VEC>(p, row[i], n0 + 8 * q, v);
  }
}

// FEW: a CTA has 32 columns and its warps take turns at a tile's groups.  Else a
// warp has 32 columns and all groups of the CTA's tiles.
template <bool FEW, bool VEC, int PARTS>
__global__ void __launch_bounds__(kWarps * 32) expand_kernel(const LowRankParams p) {
  if (p.mode_dev != nullptr && SIXBIT_MODE_OF(*p.mode_dev) != SIXBIT_MODE_INT8) return;
  __shared__ uint8_t lists[kWarps][kTile];
  const int warp = threadIdx.x >> 5;
  const int n0 = (FEW ? blockIdx.y : blockIdx.y * kWarps + warp) * 32;
  if (n0 >= p.N) return;
  for (int i = 0; i < p.tiles_per_cta; ++i) {
    const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * p.tiles_per_cta + i) * kTile;
    if (row0 >= p.M) return;
    const Groups groups = groups_of(p, row0, true, false);
    uint32_t left = groups.leaders;
    for (int turn = 0; left != 0; ++turn, left &= left - 1) {
      if (FEW && turn % kWarps != warp) continue;
      int id;
      const int count = rows_of(groups, __ffs(left) - 1, lists[warp], &id);
      expand_group<VEC, PARTS>(p, row0, n0, id, count, lists[warp]);
    }
  }
}

template <bool INT8, int RT>
cudaError_t launch_shrink(const LowRankParams& p, int tiles, int slots, cudaStream_t st) {
  const int smem = kWarps * kTile * (8 * RT + 1) * 4;
  if (smem > 48 * 1024) {
    const cudaError_t e = set_smem_once<shrink_kernel<INT8, RT>>(smem);
    if (e != cudaSuccess) return e;
  }
  note_launch();
  shrink_kernel<INT8, RT><<<dim3(tiles, slots, p.splits), kWarps * 32, smem, st>>>(p);
  return cudaGetLastError();
}

template <bool INT8>
cudaError_t launch_shrink(const LowRankParams& p, int tiles, int slots, cudaStream_t st) {
  if (p.R <= 16) return launch_shrink<INT8, 2>(p, tiles, slots, st);
  if (p.R <= 32) return launch_shrink<INT8, 4>(p, tiles, slots, st);
  return launch_shrink<INT8, 8>(p, tiles, slots, st);
}

template <bool VEC, int PARTS>
cudaError_t launch_expand(LowRankParams p, int tiles, cudaStream_t st) {
  const bool few = tiles <= 8;
  p.tiles_per_cta = few ? 1 : 4;
  const int strips = (p.N + 31) / 32;
  note_launch();
  if (few)
    expand_kernel<true, VEC, PARTS><<<dim3(tiles, strips), kWarps * 32, 0, st>>>(p);
  else
    expand_kernel<false, VEC, PARTS>
        <<<dim3((tiles + 3) / 4, (strips + kWarps - 1) / kWarps), kWarps * 32, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace lowrank

int lowrank_splits(int M, int K) {
  // K over several CTAs where few rows leave SMs idle
  const int units = K / lowrank::kUnit, fill = 152 / (M < 32 ? M : 32);
  if (M > 32) return 1;
  const int most = (units + lowrank::kWarps - 1) / lowrank::kWarps;
  return most < fill ? (most < 8 ? most : 8) : (fill < 8 ? fill : 8);
}

cudaError_t launch_lowrank(LowRankParams p, cudaStream_t st) {
  const int tiles = (p.M + lowrank::kTile - 1) / lowrank::kTile;
  p.splits = lowrank_splits(p.M, p.K);
  const int most = 608 / tiles > 0 ? 608 / tiles : 1, rows = p.M < 32 ? p.M : 32;
  const int slots = most < rows ? most : rows;
  const cudaError_t e = p.codes != nullptr ? lowrank::launch_shrink<true>(p, tiles, slots, st)
                                           : lowrank::launch_shrink<false>(p, tiles, slots, st);
  if (e != cudaSuccess) return e;
  const auto a16 = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; };
  const bool vec = p.N % 8 == 0 && a16(p.base) && a16(p.base_f32) && a16(p.residual) && a16(p.Y) && a16(p.Yf);
  if (p.Yf != nullptr) return vec ? lowrank::launch_expand<true, 3>(p, tiles, st) : lowrank::launch_expand<false, 3>(p, tiles, st);
  return vec ? lowrank::launch_expand<true, 2>(p, tiles, st) : lowrank::launch_expand<false, 2>(p, tiles, st);
}

}  // namespace sixbit
