// Low-rank adapters of many requests beside one shared projection:
//
//   y[m] = epilogue(base[m] + alpha_l . B_l (A_l x_m)),   l = ids[m]  (-1: base alone)
//
// x: INT8 codes with a scale per row (rotated, as the W4A8 products read them;
// A_l is rotated when it is packed) or bf16.  A_l [R, K] and B_l [N, R] bf16.
//
// v = A_l x is summed over K into the workspace, and a second kernel adds its
// product with B_l to the base and applies the epilogue.  Both run on
// mma.m16n8k16 with bf16 operands and FP32 sums, rows as the 16-row operand.
// Codes are exact in bf16.  v, with the row's scale and alpha on it, enters the
// second product as two bf16 parts (v to 2^-16; three and 2^-24 where the result
// is FP32): one part alone would add an error as large as the output's own
// rounding.
//
// Rows are taken in the order of their adapters, 32 positions a tile, so that an
// MMA's rows share one however requests are mixed.  Up to 32 rows every warp sorts
// them by itself; above, a counting sort by one CTA goes first.  The order of rows
// of one adapter is not fixed (atomics), and does not matter: a row's sums do not
// depend on its place.
#include <climits>
#include <cooperative_groups.h>
#include <cstdint>

#include "common.cuh"
#include "ctx_cache.h"
#include "gemm_common.cuh"
#include "internal.h"

namespace sixbit {
namespace lowrank {

constexpr int kTile = 32;        // positions of a tile
constexpr int kWarps = 8;
constexpr int kUnit = 64;        // k of a warp's turn
constexpr int kFew = kTile;      // rows that need no sorting kernel
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

// What a launch with a programmatic dependence on the one before needs of it.
__device__ __forceinline__ void before_done() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A row's adapter, -1 for none.
__device__ __forceinline__ int adapter_of(const LowRankParams& p, int row, bool report) {
  const int id = __ldg(p.ids + row);
  if (id >= 0 && id < p.L) return id;
  if (id != -1 && report) set_error(p.err, SIXBIT_EDEVICE);
  return -1;
}

// Counting sort of the rows by adapter: perm[pos] = row, sid[pos] = its adapter.
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const LowRankParams p) {
  next_may_start();
  if (p.mode_dev != nullptr && SIXBIT_MODE_OF(*p.mode_dev) != SIXBIT_MODE_INT8) return;
  extern __shared__ int at[];  // [L + 1]: rows of adapter i - 1, then where they go
  __shared__ int part[kPlanThreads / 32];
  const int bins = p.L + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < bins; i += kPlanThreads) at[i] = 0;
  __syncthreads();
  auto walk = [&](bool place) {
    for (int64_t r0 = threadIdx.x - lane; r0 < p.M; r0 += kPlanThreads) {
      const int64_t row = r0 + lane;
      const int id = row < p.M ? adapter_of(p, static_cast<int>(row), !place) : INT_MAX;
      const uint32_t same = __match_any_sync(kAll, id);
      const int leader = __ffs(same) - 1;
      int first = 0;
      if (id != INT_MAX && lane == leader) first = atomicAdd(&at[id + 1], __popc(same));
      if (place) {
        first = __shfl_sync(kAll, first, leader);
        if (id != INT_MAX) {
          const int pos = first + __popc(same & ((1u << lane) - 1));
          p.perm[pos] = static_cast<int>(row);
          p.sid[pos] = id;
        }
      }
    }
  };
  walk(false);
  __syncthreads();
  // exclusive sums of the bins, each thread a run of them
  const int run = (bins + kPlanThreads - 1) / kPlanThreads, i0 = threadIdx.x * run, i1 = min(i0 + run, bins);
  int sum = 0;
  for (int i = i0; i < i1; ++i) sum += at[i];
  int up = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kAll, up, o);
    if (lane >= o) up += v;
  }
  if (lane == 31) part[warp] = up;
  __syncthreads();
  int first = up - sum;
  for (int w = 0; w < warp; ++w) first += part[w];
  for (int i = i0; i < i1; ++i) {
    const int n = at[i];
    at[i] = first;
    first += n;
  }
  __syncthreads();
  walk(true);
}

// A tile's positions, one a lane: the row and its adapter (INT_MAX beyond the
// last), and a bit for each position that begins another adapter's run.
struct Tile {
  int id, row;
  uint32_t heads;
};
template <bool FEW>
__device__ __forceinline__ Tile tile_at(const LowRankParams& p, int64_t pos0, int* scratch, bool report) {
  const int lane = threadIdx.x & 31;
  Tile t;
  t.id = INT_MAX;
  t.row = 0;
  if constexpr (FEW) {
    const int id = lane < p.M ? adapter_of(p, lane, report) : INT_MAX;
    int rank = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int o = __shfl_sync(kAll, id, i);
      rank += o < id || (o == id && i < lane);
    }
    scratch[rank] = lane;
    __syncwarp();
    t.row = scratch[lane];
    t.id = __shfl_sync(kAll, id, t.row);
    if (t.id == INT_MAX) t.row = 0;
  } else if (pos0 + lane < p.M) {
    t.id = p.sid[pos0 + lane];
    t.row = p.perm[pos0 + lane];
  }
  const int before = __shfl_up_sync(kAll, t.id, 1);
  t.heads = __ballot_sync(kAll, t.id != INT_MAX && (lane == 0 || before != t.id));
  return t;
}
// The run that begins at bit `first` of a tile: its length.
__device__ __forceinline__ int run_length(const Tile& t, int first) {
  const uint32_t live = __ballot_sync(kAll, t.id != INT_MAX);
  const uint32_t later = t.heads & ~((2u << first) - 1);
  return (later != 0 ? __ffs(later) - 1 : __popc(live)) - first;
}

// v as the second product takes it: for each position and four ranks PARTS times
// four bf16.
template <int PARTS>
__device__ __forceinline__ void store_parts(const LowRankParams& p, int64_t pos, int r, float (&v)[4]) {
  uint2* o = reinterpret_cast<uint2*>(p.v) + (pos * (p.R / 4) + r / 4) * PARTS;
#pragma unroll
  for (int s = 0; s < PARTS; ++s) {
    const uint2 w = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    o[s] = w;
    v[0] = rest(v[0], w.x << 16), v[1] = rest(v[1], w.x & 0xFFFF0000u);
    v[2] = rest(v[2], w.y << 16), v[3] = rest(v[3], w.y & 0xFFFF0000u);
  }
}

// v of one tile.  Grid: tiles x slots x splits; slot s takes the tile's runs s,
// s + slots, ...; a cluster of `splits` CTAs and their warps share K, and their
// sums meet in shared memory in a fixed order.  RT: tiles of eight ranks at a time.
template <bool FEW, bool INT8, int RT, int PARTS>
__global__ void __launch_bounds__(kWarps * 32, 2) shrink_kernel(const LowRankParams p) {
  namespace cg = cooperative_groups;
  next_may_start();
  if (!FEW) before_done();
  if (p.mode_dev != nullptr && SIXBIT_MODE_OF(*p.mode_dev) != SIXBIT_MODE_INT8) return;
  extern __shared__ float part[];  // [kWarps][kTile][kP]
  __shared__ int scratch[kWarps][32];
  constexpr int kP = 8 * RT + 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, q = lane & 3;
  const int64_t pos0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const Tile t = tile_at<FEW>(p, pos0, scratch[warp], blockIdx.y == 0 && blockIdx.z == 0 && warp == 0);
  uint32_t left = t.heads;
  for (int turn = 0; left != 0; ++turn, left &= left - 1) {
    const int first = __ffs(left) - 1, id = __shfl_sync(kAll, t.id, first);
    if (turn % gridDim.y != blockIdx.y || id < 0) continue;
    const int count = run_length(t, first);
    size_t at[4];
    bool live[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      live[i] = g8 + 8 * i < count;
      at[i] = static_cast<size_t>(__shfl_sync(kAll, t.row, (first + g8 + 8 * i) & 31)) * p.K;
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
          for (int i = 0; i < 4; i += 2)
            *reinterpret_cast<float2*>(&part[(warp * kTile + 16 * m + 4 * i + g8) * kP + 8 * j + 2 * q]) =
                make_float2(acc[m][j][i], acc[m][j][i + 1]);
      const auto cluster = cg::this_cluster();
      if (gridDim.z > 1)
        cluster.sync();
      else
        __syncthreads();
      const int quads = 2 * tiles;  // four ranks each
      for (int i = blockIdx.z * kWarps * 32 + threadIdx.x; i < count * quads; i += gridDim.z * kWarps * 32) {
        const int n = i / quads, r = i % quads * 4;
        float v[4] = {};
        for (int z = 0; z < static_cast<int>(gridDim.z); ++z) {
          const float* from = gridDim.z > 1 ? cluster.map_shared_rank(part, z) : part;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float4 f = *reinterpret_cast<const float4*>(&from[(w * kTile + n) * kP + r]);
            v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
          }
        }
        const int row = FEW ? scratch[0][first + n] : p.perm[pos0 + first + n];
        const float f = (INT8 ? __ldg(p.row_scale + row) : 1.f) * (p.alpha != nullptr ? __ldg(p.alpha + id) : 1.f);
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] *= f;
        store_parts<PARTS>(p, pos0 + first + n, r0 + r, v);
      }
      if (gridDim.z > 1)
        cluster.sync();
      else
        __syncthreads();
    }
  }
}

// Eight consecutive values of one row of a bf16 or FP32 matrix.
struct Eight {
  uint4 a, b;
};
__device__ __forceinline__ void add_bf16(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] += __uint_as_float(u[i] << 16);
    v[2 * i + 1] += __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ Eight load_base(const LowRankParams& p, size_t at) {
  Eight e;
  e.a = e.b = make_uint4(0, 0, 0, 0);
  if (p.base_f32 != nullptr) {
    e.a = *reinterpret_cast<const uint4*>(p.base_f32 + at);
    e.b = *reinterpret_cast<const uint4*>(p.base_f32 + at + 4);
  } else if (p.base != nullptr) {
    e.a = *reinterpret_cast<const uint4*>(p.base + at);
  }
  return e;
}

// Eight consecutive outputs of one row from column n on: base, epilogue, store.
// `base` holds the base's where VEC.
template <bool VEC>
__device__ __forceinline__ void finish(const LowRankParams& p, size_t at, int n, const Eight& base, float (&v)[8]) {
  if constexpr (VEC) {
    if (p.base_f32 != nullptr) {
      const uint32_t u[8] = {base.a.x, base.a.y, base.a.z, base.a.w, base.b.x, base.b.y, base.b.z, base.b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += __uint_as_float(u[i]);
    } else {
      add_bf16(base.a, v);
    }
    if (p.epilogue == SIXBIT_EPI_GELU) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t g = gelu_pair(f2_pack(v[2 * i], v[2 * i + 1]));
        v[2 * i] = f2_lo(g);
        v[2 * i + 1] = f2_hi(g);
      }
    } else if (p.epilogue == SIXBIT_EPI_RESIDUAL) {
      add_bf16(*reinterpret_cast<const uint4*>(p.residual + at), v);
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

// base + B_l v and the epilogue.  Grid: strips of 32 columns, one a warp, x chunks
// of tiles_per_cta tiles x slots (of a tile's runs, as above).  Ranks and columns
// may stand in any order as long as the operands agree: a lane keeps four
// consecutive ranks of an MMA's 16, and column c of MMA j stands for
// n0 + 8 (c / 2) + 2 j + c % 2, so that a lane ends up with eight consecutive
// outputs of each of its rows.  B_l's strip stays in registers from run to run of
// one adapter (KS: 16-rank steps of them).
template <bool FEW, bool VEC, int PARTS, int KS>
__global__ void __launch_bounds__(kWarps * 32, 2) expand_kernel(const LowRankParams p) {
  __shared__ int scratch[kWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, q = lane & 3;
  const int n0 = (blockIdx.x * (blockDim.x >> 5) + warp) * 32, n = n0 + 8 * q;
  before_done();
  if (p.mode_dev != nullptr && SIXBIT_MODE_OF(*p.mode_dev) != SIXBIT_MODE_INT8) return;
  if (n0 >= p.N) return;
  const int steps = p.R / 16;
  int held = -1;  // the adapter whose strip is in b
  uint2 b[KS][4];
  for (int i = 0; i < p.tiles_per_cta; ++i) {
    const int64_t pos0 = (static_cast<int64_t>(blockIdx.y) * p.tiles_per_cta + i) * kTile;
    if (pos0 >= p.M) return;
    const Tile t = tile_at<FEW>(p, pos0, scratch[warp], false);
    uint32_t left = t.heads;
    for (int turn = 0; left != 0; ++turn, left &= left - 1) {
      if (turn % gridDim.z != blockIdx.z) continue;
      const int first = __ffs(left) - 1, id = __shfl_sync(kAll, t.id, first), count = run_length(t, first);
      for (int m = 0; m < count; m += 16) {
        size_t at[2];
        bool live[2];
        Eight base[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          live[h] = g8 + 8 * h < count - m;
          at[h] = static_cast<size_t>(__shfl_sync(kAll, t.row, (first + m + g8 + 8 * h) & 31)) * p.N + n;
          if constexpr (VEC) {
            live[h] = live[h] && n < p.N;
            if (live[h]) base[h] = load_base(p, at[h]);
          }
        }
        float acc[4][4] = {};
        if (id >= 0) {
          const int64_t pos = pos0 + first + m + g8;
          for (int s0 = 0; s0 < steps; s0 += KS) {
            if (held != id || steps > KS) {
              const uint16_t* bl = p.b + static_cast<size_t>(id) * p.N * p.R;
#pragma unroll
              for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int c = n0 + 8 * (g8 >> 1) + 2 * j + (g8 & 1);
                  b[s][j] = make_uint2(0, 0);
                  if (c < p.N && s0 + s < steps)
                    b[s][j] = __ldg(reinterpret_cast<const uint2*>(bl + static_cast<size_t>(c) * p.R + (s0 + s) * 16 + 4 * q));
                }
              held = id;
            }
#pragma unroll
            for (int s = 0; s < KS; ++s) {
              if (s0 + s >= steps) break;
              uint2 v[2][PARTS];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int w = 0; w < PARTS; ++w) v[h][w] = make_uint2(0, 0);
                if (g8 + 8 * h < count - m) {
                  const uint2* from = reinterpret_cast<const uint2*>(p.v) + ((pos + 8 * h) * (p.R / 4) + (s0 + s) * 4 + q) * PARTS;
                  if constexpr (PARTS == 2) {
                    const uint4 f = *reinterpret_cast<const uint4*>(from);
                    v[h][0] = make_uint2(f.x, f.y);
                    v[h][1] = make_uint2(f.z, f.w);
                  } else {
#pragma unroll
                    for (int w = 0; w < PARTS; ++w) v[h][w] = from[w];
                  }
                }
              }
#pragma unroll
              for (int w = PARTS - 1; w >= 0; --w) {
                const uint32_t a[4] = {v[0][w].x, v[1][w].x, v[0][w].y, v[1][w].y};
#pragma unroll
                for (int j = 0; j < 4; ++j) mma(acc[j], a, b[s][j].x, b[s][j].y);
              }
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!live[h]) continue;
          float y[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            y[2 * j] = acc[j][2 * h];
            y[2 * j + 1] = acc[j][2 * h + 1];
          }
          finish<VEC>(p, at[h], n, base[h], y);
        }
      }
    }
  }
}

// A launch that may start while the one before it on the stream runs.
struct Early {
  cudaLaunchAttribute attrs[2];
  cudaLaunchConfig_t cfg;
  Early(dim3 grid, int threads, int smem, cudaStream_t st, bool early, int cluster_z = 1) : cfg{} {
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attrs;
    if (early) {
      attrs[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attrs[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster_z > 1) {
      attrs[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
      attrs[cfg.numAttrs].val.clusterDim.x = 1;
      attrs[cfg.numAttrs].val.clusterDim.y = 1;
      attrs[cfg.numAttrs++].val.clusterDim.z = cluster_z;
    }
  }
};

template <bool FEW, bool INT8, int RT, int PARTS>
cudaError_t launch_shrink(const LowRankParams& p, int tiles, cudaStream_t st) {
  constexpr int smem = kWarps * kTile * (8 * RT + 4) * 4;
  if (smem > 48 * 1024) {
    const cudaError_t e = set_smem_once<shrink_kernel<FEW, INT8, RT, PARTS>>(smem);
    if (e != cudaSuccess) return e;
  }
  // about two CTAs an SM: first a CTA for each of a tile's runs, then K over clusters
  const int rows = p.M < 32 ? p.M : FEW ? 32 : 4;
  const int most = 304 / tiles > 0 ? 304 / tiles : 1, slots = most < rows ? most : rows;
  const int turns = (p.K / kUnit + kWarps - 1) / kWarps, left = most / slots > 0 ? most / slots : 1;
  int splits = turns < left ? turns : left;
  if (splits > 8) splits = 8;
  Early l(dim3(tiles, slots, splits), kWarps * 32, smem, st, !FEW, splits);
  note_launch();
  return cudaLaunchKernelEx(&l.cfg, shrink_kernel<FEW, INT8, RT, PARTS>, p);
}

template <bool FEW, bool INT8, int PARTS>
cudaError_t launch_shrink(const LowRankParams& p, int tiles, cudaStream_t st) {
  if (p.R <= 16) return launch_shrink<FEW, INT8, 2, PARTS>(p, tiles, st);
  if (p.R <= 32) return launch_shrink<FEW, INT8, 4, PARTS>(p, tiles, st);
  return launch_shrink<FEW, INT8, 8, PARTS>(p, tiles, st);
}

template <bool FEW, bool VEC, int PARTS, int KS>
cudaError_t launch_expand(LowRankParams p, int tiles, cudaStream_t st) {
  const int strips = (p.N + 31) / 32;
  int warps = kWarps, slots = 1;
  p.tiles_per_cta = 1;
  if (FEW) {
    warps = 4;
    slots = p.M;
  } else {
    p.tiles_per_cta = tiles > 4 * 65535 ? (tiles + 65534) / 65535 : 4;
  }
  const dim3 grid((strips + warps - 1) / warps, (tiles + p.tiles_per_cta - 1) / p.tiles_per_cta, slots);
  Early l(grid, warps * 32, 0, st, true);
  note_launch();
  return cudaLaunchKernelEx(&l.cfg, expand_kernel<FEW, VEC, PARTS, KS>, p);
}

template <bool FEW, bool VEC, int PARTS>
cudaError_t launch_both(const LowRankParams& p, int tiles, cudaStream_t st) {
  const cudaError_t e = p.codes != nullptr ? launch_shrink<FEW, true, PARTS>(p, tiles, st)
                                           : launch_shrink<FEW, false, PARTS>(p, tiles, st);
  if (e != cudaSuccess) return e;
  if (p.R <= 16) return launch_expand<FEW, VEC, PARTS, 1>(p, tiles, st);
  if (p.R <= 32) return launch_expand<FEW, VEC, PARTS, 2>(p, tiles, st);
  return launch_expand<FEW, VEC, PARTS, 4>(p, tiles, st);
}

template <bool FEW>
cudaError_t launch_form(const LowRankParams& p, int tiles, cudaStream_t st) {
  const auto a16 = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; };
  const bool vec = p.N % 8 == 0 && a16(p.base) && a16(p.base_f32) && a16(p.residual) && a16(p.Y) && a16(p.Yf);
  if (p.Yf != nullptr) return vec ? launch_both<FEW, true, 3>(p, tiles, st) : launch_both<FEW, false, 3>(p, tiles, st);
  return vec ? launch_both<FEW, true, 2>(p, tiles, st) : launch_both<FEW, false, 2>(p, tiles, st);
}

}  // namespace lowrank

size_t lowrank_workspace(int M, int R) {
  // v in up to three parts; above kFew rows the rows' order and their adapters
  const size_t rows = static_cast<size_t>(M), order = (rows * 4 + 15) / 16 * 16;
  return rows * R * 6 + (M > lowrank::kFew ? 2 * order : 0);
}

cudaError_t launch_lowrank(LowRankParams p, void* workspace, cudaStream_t st) {
  const int tiles = (p.M + lowrank::kTile - 1) / lowrank::kTile;
  if (p.M <= lowrank::kFew) {
    p.v = workspace;
    return lowrank::launch_form<true>(p, tiles, st);
  }
  const size_t order = (static_cast<size_t>(p.M) * 4 + 15) / 16 * 16;
  p.perm = static_cast<int32_t*>(workspace);
  p.sid = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + order);
  p.v = static_cast<uint8_t*>(workspace) + 2 * order;
  const int smem = (p.L + 1) * 4;
  if (smem > 48 * 1024) {
    const cudaError_t e = set_smem_once<lowrank::plan_kernel>((SIXBIT_MAX_ADAPTERS + 1) * 4);
    if (e != cudaSuccess) return e;
  }
  note_launch();
  lowrank::plan_kernel<<<1, lowrank::kPlanThreads, smem, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : lowrank::launch_form<false>(p, tiles, st);
}

}  // namespace sixbit
