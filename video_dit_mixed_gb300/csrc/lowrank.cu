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
// second product as three bf16 parts, v to 2^-24 whatever the result's type.  (Of two,
// 2^-16, the error passed a bf16 output's rounding where the base cancels the product,
// and one output in 1,400 of 17,776 x 7680 was rounded to its other neighbour, where
// now one in 5,600 is; GELU over them took 222 us.)
//
// Rows are taken in the order of their adapters, 32 positions a tile, so that an
// MMA's rows share one however requests are mixed.  Of few rows (up to 64 or 128)
// every warp sorts 32 by itself, and one launch does both products; of more a
// counting sort goes first.  The order of rows of one adapter is not fixed (atomics),
// and does not matter: a row's sums do not depend on its place.
//
// The floor is bytes, of which base and result are nearly all for many rows.
// 17,776 x 7680 outputs, bf16 base and result: rank 16 119 us (floor 84), rank 64
// with GELU 248 (GELU takes 80 us of the FP32 pipe by itself, the 48 MMAs of a tile of
// 16 x 32 some 88 of theirs); 1920 outputs of K 7680, rank 64, residual: 126 (A's
// product 70 of it).  One row beside 7680 x 1920 5.1 us, 32 rows of 32 requests beside
// 1920 x 7680 9.5, 226 rows 20, 2000 mixed rows of 32 adapters 47.
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
// Rows that need no sorting kernel.  (7680 x 1920, rank 16: 33 mixed rows 11 us against
// 35, 128 21 against 24; rank 64: 64 rows 28 against 39, 128 51 against 31.)
constexpr int few_rows(int R) { return R > 32 ? 64 : 128; }
constexpr int kChunk = 256;      // positions of a CTA that applies B, at most
constexpr int kManyBytes = 113 * 1024;  // its shared memory: two on an SM
constexpr unsigned kAll = 0xFFFFFFFFu;

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four s8 codes as bf16, exact: under the exponent of 2^23 a byte is 2^23 + 128 + the
// code in FP32, and the high half of an integer below 256 is its bf16.  (bf16
// arithmetic on pairs is three or more instructions here.)
__device__ __forceinline__ void codes_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  w ^= 0x80808080u;
  const uint64_t less = f2_pack(-8388736.f, -8388736.f);
  const auto pair = [&](uint32_t first) {
    const uint64_t f = f2_add(f2_pack(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440u + first)),
                                      __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7441u + first))), less);
    return __byte_perm(static_cast<uint32_t>(f), static_cast<uint32_t>(f >> 32), 0x7632);
  };
  lo = pair(0);
  hi = pair(2);
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

// Counting sort of the rows by adapter: perm[pos] = row, sid[pos] = its adapter.  One
// CTA, or a cluster of them that each count a part of the rows and read each
// other's counts (17776 rows: 19 us by one).
constexpr int kPlanThreads = 1024, kPlanAtOnce = 4, kPlanCluster = 8;
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const LowRankParams p) {
  namespace cg = cooperative_groups;
  next_may_start();
  if (p.mode_dev != nullptr && SIXBIT_MODE_OF(*p.mode_dev) != SIXBIT_MODE_INT8) return;
  extern __shared__ int count[];  // [L + 1] rows of adapter i - 1 in this CTA's part, [L + 1] where they go
  __shared__ int part[kPlanThreads / 32];
  const int bins = p.L + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int* at = count + bins;
  const auto cluster = cg::this_cluster();
  const int ctas = gridDim.x, me = blockIdx.x;
  for (int i = threadIdx.x; i < bins; i += kPlanThreads) count[i] = 0;
  __syncthreads();
  const int64_t per = (static_cast<int64_t>(p.M) + ctas - 1) / ctas, end = min(static_cast<int64_t>(p.M), per * (me + 1));
  auto walk = [&](int* to, bool place) {
    for (int64_t r0 = per * me + threadIdx.x - lane; r0 < end; r0 += kPlanThreads * kPlanAtOnce) {
      int id[kPlanAtOnce], first[kPlanAtOnce];
      uint32_t same[kPlanAtOnce];
#pragma unroll
      for (int u = 0; u < kPlanAtOnce; ++u) {
        const int64_t row = r0 + u * kPlanThreads + lane;
        id[u] = row < end ? adapter_of(p, static_cast<int>(row), !place) : INT_MAX;
      }
#pragma unroll
      for (int u = 0; u < kPlanAtOnce; ++u) {
        same[u] = __match_any_sync(kAll, id[u]);
        first[u] = 0;
        if (id[u] != INT_MAX && lane == __ffs(same[u]) - 1) first[u] = atomicAdd(&to[id[u] + 1], __popc(same[u]));
      }
      if (place) {
#pragma unroll
        for (int u = 0; u < kPlanAtOnce; ++u) {
          const int pos = __shfl_sync(kAll, first[u], __ffs(same[u]) - 1) + __popc(same[u] & ((1u << lane) - 1));
          if (id[u] != INT_MAX) {
            p.perm[pos] = static_cast<int>(r0 + u * kPlanThreads + lane);
            p.sid[pos] = id[u];
          }
        }
      }
    }
  };
  walk(count, false);
  if (ctas > 1)
    cluster.sync();
  else
    __syncthreads();
  // exclusive sums over the bins, each thread a run of them, and the earlier CTAs' share of each
  const int run = (bins + kPlanThreads - 1) / kPlanThreads;
  const int i0 = min(static_cast<int>(threadIdx.x) * run, bins), i1 = min(i0 + run, bins);
  int sum = 0;
  for (int i = i0; i < i1; ++i) {
    int before = 0, all = 0;
    for (int c = 0; c < ctas; ++c) {
      const int n = ctas > 1 ? cluster.map_shared_rank(count, c)[i] : count[i];
      if (c < me) before += n;
      all += n;
    }
    at[i] = sum + before;
    sum += all;
  }
  int up = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kAll, up, o);
    if (lane >= o) up += v;
  }
  if (lane == 31) part[warp] = up;
  if (ctas > 1)
    cluster.sync();  // (no CTA leaves while another reads its counts)
  else
    __syncthreads();
  int first = up - sum;
  for (int w = 0; w < warp; ++w) first += part[w];
  for (int i = i0; i < i1; ++i) at[i] += first;
  __syncthreads();
  walk(at, true);
}

// A tile's positions, one a lane: the row and its adapter (INT_MAX beyond the
// last), and a bit for each position that begins another adapter's run.
struct Tile {
  int id, row;
  uint32_t heads;
};
__device__ __forceinline__ void mark_heads(Tile& t) {
  const int lane = threadIdx.x & 31, before = __shfl_up_sync(kAll, t.id, 1);
  t.heads = __ballot_sync(kAll, t.id != INT_MAX && (lane == 0 || before != t.id));
}
__device__ __forceinline__ Tile tile_at(const LowRankParams& p, int64_t pos0) {
  const int64_t pos = pos0 + (threadIdx.x & 31);
  Tile t;
  t.id = pos < p.M ? p.sid[pos] : INT_MAX;
  t.row = pos < p.M ? p.perm[pos] : 0;
  mark_heads(t);
  return t;
}
// 32 rows from row0 on, sorted by the warp; scratch: 32 words of its own, which then
// hold the rows.
__device__ __forceinline__ Tile tile_of_few(const LowRankParams& p, int row0, int* scratch, bool report) {
  const int lane = threadIdx.x & 31, id = row0 + lane < p.M ? adapter_of(p, row0 + lane, report) : INT_MAX;
  int rank = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const int o = __shfl_sync(kAll, id, i);
    rank += o < id || (o == id && i < lane);
  }
  scratch[rank] = lane;
  __syncwarp();
  Tile t;
  const int from = scratch[lane];
  t.id = __shfl_sync(kAll, id, from);
  t.row = t.id == INT_MAX ? 0 : row0 + from;
  scratch[lane] = t.row;
  __syncwarp();
  mark_heads(t);
  return t;
}
// The run that begins at bit `first` of a tile: its length.
__device__ __forceinline__ int run_length(const Tile& t, int first) {
  const uint32_t live = __ballot_sync(kAll, t.id != INT_MAX);
  const uint32_t later = t.heads & ~((2u << first) - 1);
  return (later != 0 ? __ffs(later) - 1 : __popc(live)) - first;
}

// v as the second product takes it, three bf16 parts of four ranks at a time: for
// each position and four ranks 16 bytes of the first two parts, and in an array
// behind them 8 of the third.
constexpr int kParts = 3;
struct Parts {
  uint4 first;  // [2][4]
  uint2 last;   // [4]
};
__device__ __forceinline__ Parts parts_of(float (&v)[4]) {
  uint2 w[kParts];
#pragma unroll
  for (int s = 0; s < kParts; ++s) {
    w[s] = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    v[0] = rest(v[0], w[s].x << 16), v[1] = rest(v[1], w[s].x & 0xFFFF0000u);
    v[2] = rest(v[2], w[s].y << 16), v[3] = rest(v[3], w[s].y & 0xFFFF0000u);
  }
  return {make_uint4(w[0].x, w[0].y, w[1].x, w[1].y), w[2]};
}
// v of ranks r .. r + 3 of a position, to the workspace.
__device__ __forceinline__ void store_v(const LowRankParams& p, int64_t pos, int r, float (&v)[4]) {
  const Parts w = parts_of(v);
  const int64_t at = pos * (p.R / 4) + r / 4;
  static_cast<uint4*>(p.v)[at] = w.first;
  static_cast<uint2*>(p.v_last)[at] = w.last;
}

// One warp's share of A_l x for up to 32 rows: k units first, first + step, ..., 8 RT
// ranks from `a` (rank g8 of them) on, of which `tiles` times eight exist.  The sums
// go to `to` [kTile][8 RT + 4].
template <bool INT8, int RT>
__device__ __forceinline__ void sums_of(const LowRankParams& p, const uint16_t* a, int tiles, const size_t (&at)[4],
                                        const bool (&live)[4], int count, int first, int step, float* to) {
  constexpr int kP = 8 * RT + 4;
  const int lane = threadIdx.x & 31, g8 = lane >> 2, q = lane & 3;
  float acc[2][RT][4] = {};
  for (int u = first; u < p.K / kUnit; u += step) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // 32 k; a lane keeps eight of them, four for each MMA
      const int k = u * kUnit + 32 * h + 8 * q;
      uint4 b[RT];
#pragma unroll
      for (int j = 0; j < RT; ++j)
        b[j] = j < tiles ? __ldg(reinterpret_cast<const uint4*>(a + static_cast<size_t>(8 * j) * p.K + k))
                         : make_uint4(0, 0, 0, 0);
      uint32_t x[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0;
        if (live[i]) {
          if constexpr (INT8) {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(p.codes + at[i] + k));
            codes_bf16(w.x, x[i][0], x[i][1]);
            codes_bf16(w.y, x[i][2], x[i][3]);
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
        for (int j = 0; j < RT; ++j) {
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
        *reinterpret_cast<float2*>(&to[(16 * m + 4 * i + g8) * kP + 8 * j + 2 * q]) =
            make_float2(acc[m][j][i], acc[m][j][i + 1]);
}

// v of one tile.  Grid: tiles x slots x splits; slot s takes the tile's runs s,
// s + slots, ...; a cluster of `splits` CTAs and their warps share K, and their
// sums meet in shared memory in a fixed order.  RT: tiles of eight ranks at a time.
template <bool INT8, int RT>
__global__ void __launch_bounds__(kWarps * 32, 2) shrink_kernel(const LowRankParams p) {
  namespace cg = cooperative_groups;
  next_may_start();
  before_done();
  if (p.mode_dev != nullptr && SIXBIT_MODE_OF(*p.mode_dev) != SIXBIT_MODE_INT8) return;
  extern __shared__ float part[];  // [kWarps][kTile][kP]
  constexpr int kP = 8 * RT + 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, q = lane & 3;
  const int64_t pos0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const Tile t = tile_at(p, pos0);
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
      sums_of<INT8, RT>(p, a, tiles, at, live, count, blockIdx.z * kWarps + warp, gridDim.z * kWarps, part + warp * kTile * kP);
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
        const int row = p.perm[pos0 + first + n];
        const float f = (INT8 ? __ldg(p.row_scale + row) : 1.f) * (p.alpha != nullptr ? __ldg(p.alpha + id) : 1.f);
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] *= f;
        store_v(p, pos0 + first + n, r0 + r, v);
      }
      if (gridDim.z > 1)
        cluster.sync();
      else
        __syncthreads();
    }
  }
}

// 16 bytes from global to shared memory without a register round trip; zeros
// where !valid (src must still be an address).
__device__ __forceinline__ void copy16(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// v of 64 positions, for many rows: x and A_l pass through shared memory, 128 k a
// stage, and are read there by four pairs of warps, 32 rows a warp, a pair for each
// quarter of the stage's k.  A run of one adapter within the block is a pass over
// K.  Grid: blocks of positions x blocks of 8 RT ranks x 2 (the block's runs in
// turn).  (Two CTAs an SM, so that
// one's MMAs run while the other waits at its stage's barrier.)
constexpr int kBlock = 64, kStageK = 128, kStagedThreads = 256;
template <bool INT8, int RT>
struct Staged {
  static constexpr int kXRow = INT8 ? 128 : 256;  // bytes of a row's stage
  static constexpr int kX = kBlock * kXRow, kA = 8 * RT * 256, kStage = kX + kA;
  static constexpr int kStages = INT8 ? 4 : 3;
  static constexpr int kP = 8 * RT + 4;           // floats of a row's sums
  static constexpr int kSums = kBlock * kP * 4;
  static constexpr int kBytes = kStages * kStage > kSums ? kStages * kStage : kSums;
};
// Where chunk `ch` (16 bytes) of a row lies.  A quarter warp's 16-byte reads take
// four neighbouring chunks of two rows, a half warp's 8-byte ones two of four.
__device__ __forceinline__ int chunk256(int row, int ch) { return row * 256 + ((ch ^ ((row & 1) << 2)) << 4); }
__device__ __forceinline__ int chunk128(int row, int ch) { return row * 128 + ((ch ^ ((row & 3) << 1)) << 4); }
template <bool INT8, int RT>
__global__ void __launch_bounds__(kStagedThreads, 2) staged_kernel(const LowRankParams p) {
  using S = Staged<INT8, RT>;
  constexpr int kStages = S::kStages;
  next_may_start();
  before_done();
  if (p.mode_dev != nullptr && SIXBIT_MODE_OF(*p.mode_dev) != SIXBIT_MODE_INT8) return;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int rows[kBlock], ids[kBlock];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, q = lane & 3;
  const int wr = warp & 1, wk = warp >> 1;
  const int64_t pos0 = static_cast<int64_t>(blockIdx.x) * kBlock;
  const int r0 = blockIdx.y * 8 * RT, tiles = min(RT, (p.R - r0) / 8);
  if (tid < kBlock) {
    const bool in = pos0 + tid < p.M;
    rows[tid] = in ? p.perm[pos0 + tid] : 0;
    ids[tid] = in ? p.sid[pos0 + tid] : INT_MAX;
  }
  __syncthreads();
  const int stages = p.K / kStageK;
  for (int first = 0, turn = 0; first < kBlock; ) {
    const int id = ids[first];
    if (id == INT_MAX) break;
    int end = kBlock;
#pragma unroll
    for (int b = kBlock / 32 - 1; b >= 0; --b) {
      const uint32_t other = __ballot_sync(kAll, 32 * b + lane > first && ids[32 * b + lane] != id);
      if (other != 0) end = 32 * b + __ffs(other) - 1;
    }
    if (id < 0 || turn++ % gridDim.z != blockIdx.z) {
      first = end;
      continue;
    }
    // this thread's chunks of a stage: of x, and of A (bytes from the adapter's first)
    constexpr int kXC = S::kXRow / 16, kNX = kBlock * kXC / kStagedThreads;
    constexpr int kNA = (8 * RT * 16 + kStagedThreads - 1) / kStagedThreads;
    const unsigned char* x_from[kNX];
    const unsigned char* a_from = reinterpret_cast<const unsigned char*>(p.a + (static_cast<size_t>(id) * p.R + r0) * p.K);
    int a_at[kNA];
    unsigned live = 0;  // bit i: x chunk i; ranks beyond R are zeros too
#pragma unroll
    for (int i = 0; i < kNX; ++i) {
      const int c = tid + i * kStagedThreads, row = c / kXC, ch = c % kXC;
      if (row >= first && row < end) live |= 1u << i;
      const size_t at = static_cast<size_t>(rows[row]) * p.K;
      x_from[i] = (INT8 ? reinterpret_cast<const unsigned char*>(p.codes + at) : reinterpret_cast<const unsigned char*>(p.x + at)) + ch * 16;
    }
#pragma unroll
    for (int i = 0; i < kNA; ++i) {
      const int c = tid + i * kStagedThreads, row = c >> 4, ch = c & 15;
      if (row < 8 * tiles) live |= 1u << (kNX + i);
      a_at[i] = row < 8 * tiles ? row * p.K * 2 + ch * 16 : 0;
    }
    auto fetch = [&](int st) {
      unsigned char* to = smem + (st % kStages) * S::kStage;
#pragma unroll
      for (int i = 0; i < kNX; ++i) {
        const int c = tid + i * kStagedThreads, row = c / kXC, ch = c % kXC;
        copy16(to + (INT8 ? chunk128(row, ch) : chunk256(row, ch)), x_from[i] + st * S::kXRow, (live >> i) & 1);
      }
#pragma unroll
      for (int i = 0; i < kNA; ++i) {
        const int c = tid + i * kStagedThreads;
        if (8 * RT * 16 % kStagedThreads == 0 || c < 8 * RT * 16)
          copy16(to + S::kX + chunk256(c >> 4, c & 15), a_from + a_at[i] + st * 256, (live >> (kNX + i)) & 1);
      }
    };
    for (int st = 0; st < kStages - 1; ++st) {
      if (st < stages) fetch(st);
      copies_commit();
    }
    const bool mine = wr * 32 < end && wr * 32 + 32 > first;
    float acc[2][RT][4] = {};
    for (int st = 0; st < stages; ++st) {
      copies_wait<kStages - 2>();
      __syncthreads();  // (the stage is here, and the one before it is free)
      if (st + kStages - 1 < stages) fetch(st + kStages - 1);
      copies_commit();
      if (!mine) continue;
      const unsigned char* xs = smem + (st % kStages) * S::kStage;
      const unsigned char* as = xs + S::kX;
      uint4 b[RT];
#pragma unroll
      for (int j = 0; j < RT; ++j)
        b[j] = *reinterpret_cast<const uint4*>(as + chunk256(8 * j + g8, 4 * wk + q));
      uint32_t x[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = wr * 32 + g8 + 8 * i;
        if constexpr (INT8) {
          const uint2 w = *reinterpret_cast<const uint2*>(xs + chunk128(row, 2 * wk + (q >> 1)) + (q & 1) * 8);
          codes_bf16(w.x, x[i][0], x[i][1]);
          codes_bf16(w.y, x[i][2], x[i][3]);
        } else {
          const uint4 w = *reinterpret_cast<const uint4*>(xs + chunk256(row, 4 * wk + q));
          x[i][0] = w.x, x[i][1] = w.y, x[i][2] = w.z, x[i][3] = w.w;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < RT; ++j)
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const uint32_t a[4] = {x[2 * m][2 * h], x[2 * m + 1][2 * h], x[2 * m][2 * h + 1], x[2 * m + 1][2 * h + 1]};
            mma(acc[m][j], a, h == 0 ? b[j].x : b[j].z, h == 0 ? b[j].y : b[j].w);
          }
    }
    // the quarters of k, joined in the stages' place
    copies_wait<0>();
    __syncthreads();
    float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int quarter = 3; quarter >= 0; --quarter) {
      if (wk == quarter && mine) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int j = 0; j < RT; ++j)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              float2* at = reinterpret_cast<float2*>(&sums[(wr * 32 + 16 * m + 4 * i + g8) * S::kP + 8 * j + 2 * q]);
              const float2 v = make_float2(acc[m][j][i], acc[m][j][i + 1]);
              *at = quarter == 3 ? v : make_float2(v.x + at->x, v.y + at->y);
            }
      }
      __syncthreads();
    }
    const int quads = 2 * tiles;
    const float alpha = p.alpha != nullptr ? __ldg(p.alpha + id) : 1.f;
    for (int i = tid; i < (end - first) * quads; i += kStagedThreads) {
      const int n = first + i / quads, r = i % quads * 4;
      const float4 f = *reinterpret_cast<const float4*>(&sums[n * S::kP + r]);
      const float by = (INT8 ? __ldg(p.row_scale + rows[n]) : 1.f) * alpha;
      float v[4] = {f.x * by, f.y * by, f.z * by, f.w * by};
      store_v(p, pos0 + n, r0 + r, v);
    }
    __syncthreads();
    first = end;
  }
}

// Eight consecutive values of the base, which is FP32 (F32) or bf16.
template <bool F32>
struct Eight {
  uint4 w[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const LowRankParams& p, size_t at) {
    if constexpr (F32) {
      w[0] = *reinterpret_cast<const uint4*>(p.base_f32 + at);
      w[1] = *reinterpret_cast<const uint4*>(p.base_f32 + at + 4);
    } else {
      w[0] = p.base != nullptr ? *reinterpret_cast<const uint4*>(p.base + at) : make_uint4(0, 0, 0, 0);
    }
  }
};
__device__ __forceinline__ void add_bf16(const uint4& w, uint64_t* v) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = f2_add(v[i], f2_from_bf16x2(u[i]));
}
__device__ __forceinline__ void add_f32(const uint4& w, uint64_t* v) {
  v[0] = f2_add(v[0], f2_pack(__uint_as_float(w.x), __uint_as_float(w.y)));
  v[1] = f2_add(v[1], f2_pack(__uint_as_float(w.z), __uint_as_float(w.w)));
}

// Eight consecutive outputs of one row, 16-byte aligned.
__device__ __forceinline__ void store8(const LowRankParams& p, size_t at, const uint64_t* v) {
  if (p.Yf != nullptr) {
    reinterpret_cast<float4*>(p.Yf + at)[0] = make_float4(f2_lo(v[0]), f2_hi(v[0]), f2_lo(v[1]), f2_hi(v[1]));
    reinterpret_cast<float4*>(p.Yf + at)[1] = make_float4(f2_lo(v[2]), f2_hi(v[2]), f2_lo(v[3]), f2_hi(v[3]));
  } else {
    *reinterpret_cast<uint4*>(p.Y + at) =
        make_uint4(f2_to_bf16x2(v[0]), f2_to_bf16x2(v[1]), f2_to_bf16x2(v[2]), f2_to_bf16x2(v[3]));
  }
}
// base + B_l v and the epilogue, a warp a strip of 32 columns from n0 on.  Ranks and
// columns may stand in any order as long as the operands agree: a lane keeps four
// consecutive ranks of an MMA's 16, and column c of MMA j stands for
// n0 + 8 (c / 2) + 2 j + c % 2, so that a lane ends up with eight consecutive
// outputs of each of its two rows of a 16-row tile.  KS: 16-rank steps that are
// held in registers; R is 16 KS, or with BIG taken KS steps at a time.
template <int KS>
struct Strip {
  uint2 b[KS][4];
  __device__ __forceinline__ void load(const LowRankParams& p, int id, int n0, int s0) {
    const int lane = threadIdx.x & 31, g8 = lane >> 2, q = lane & 3, steps = p.R / 16;
    const int c0 = n0 + 8 * (g8 >> 1) + (g8 & 1);
    const uint16_t* bl = p.b + (static_cast<size_t>(id) * p.N + c0) * p.R + s0 * 16 + 4 * q;
#pragma unroll
    for (int j = 0; j < 4; ++j, bl += 2 * p.R)
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        b[s][j] = make_uint2(0, 0);
        if (c0 + 2 * j < p.N && s0 + s < steps) b[s][j] = __ldg(reinterpret_cast<const uint2*>(bl + s * 16));
      }
  }
};
// acc += the strip times a step of v, the smallest part first: lo, hi: this lane's
// parts of rows g8 and g8 + 8.
__device__ __forceinline__ void step_mma(float (&acc)[4][4], const Parts& lo, const Parts& hi, const uint2 (&b)[4]) {
  const uint32_t a[kParts][4] = {{lo.last.x, hi.last.x, lo.last.y, hi.last.y},
                                 {lo.first.z, hi.first.z, lo.first.w, hi.first.w},
                                 {lo.first.x, hi.first.x, lo.first.y, hi.first.y}};
#pragma unroll
  for (int w = 0; w < kParts; ++w)
#pragma unroll
    for (int j = 0; j < 4; ++j) mma(acc[j], a[w], b[j].x, b[j].y);
}
// The outputs of a tile of 16 rows, columns n .. n + 7 of this lane's two.
template <bool F32, bool RES>
__device__ __forceinline__ void finish_rows(const LowRankParams& p, const float (&acc)[4][4], const size_t (&row)[2],
                                            const bool (&live)[2], int n, const Eight<F32> (&base)[2],
                                            const uint4 (&res)[2]) {
  uint64_t y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = f2_pack(acc[i & 3][2 * (i >> 2)], acc[i & 3][2 * (i >> 2) + 1]);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (F32) {
      add_f32(base[h].w[0], y + 4 * h);
      add_f32(base[h].w[1], y + 4 * h + 2);
    } else {
      add_bf16(base[h].w[0], y + 4 * h);
    }
    if constexpr (RES) add_bf16(res[h], y + 4 * h);
  }
  if (!RES && p.epilogue == SIXBIT_EPI_GELU) gelu_pairs(y);
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (live[h] && n < p.N) store8(p, row[h] * p.N + n, y + 4 * h);
}
// The same for rows that are not 16-byte aligned: through the warp's `turn` [16][33],
// so that a lane has one column of all 16 rows, rows[0 .. count) of them.  What is
// added to them, the base and the residual, is loaded in front of the products.
__device__ __forceinline__ void turn_load(const LowRankParams& p, const int* rows, int count, int n, float (&add)[16]) {
  // (dead rows read the first one's place: loads under a condition would wait for each other)
  size_t at[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    at[i] = i < count && n < p.N ? static_cast<size_t>(rows[i]) * p.N + n : 0;
    add[i] = 0.f;
  }
  if (p.base_f32 != nullptr) {
#pragma unroll
    for (int i = 0; i < 16; ++i) add[i] = p.base_f32[at[i]];
  } else if (p.base != nullptr) {
    uint16_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = p.base[at[i]];
#pragma unroll
    for (int i = 0; i < 16; ++i) add[i] = __uint_as_float(static_cast<uint32_t>(w[i]) << 16);
  }
  if (p.epilogue == SIXBIT_EPI_RESIDUAL) {
    uint16_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = p.residual[at[i]];
#pragma unroll
    for (int i = 0; i < 16; ++i) add[i] += __uint_as_float(static_cast<uint32_t>(w[i]) << 16);
  }
}
__device__ __forceinline__ void turn_rows(const LowRankParams& p, const float (&acc)[4][4], const int* rows, int count,
                                          int n0, const float (&add)[16], float* turn) {
  const int lane = threadIdx.x & 31, g8 = lane >> 2, q = lane & 3, n = n0 + lane;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      turn[(g8 + 8 * h) * 33 + 8 * q + 2 * j] = acc[j][2 * h];
      turn[(g8 + 8 * h) * 33 + 8 * q + 2 * j + 1] = acc[j][2 * h + 1];
    }
  __syncwarp();
  uint64_t y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    y[i] = f2_add(f2_pack(turn[2 * i * 33 + lane], turn[(2 * i + 1) * 33 + lane]), f2_pack(add[2 * i], add[2 * i + 1]));
  if (p.epilogue == SIXBIT_EPI_GELU) gelu_pairs(y);
  if (n < p.N) {
    if (p.Yf != nullptr) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < count) p.Yf[static_cast<size_t>(rows[i]) * p.N + n] = (i & 1) ? f2_hi(y[i / 2]) : f2_lo(y[i / 2]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < count)
          p.Y[static_cast<size_t>(rows[i]) * p.N + n] =
              __bfloat16_as_ushort(__float2bfloat16_rn((i & 1) ? f2_hi(y[i / 2]) : f2_lo(y[i / 2])));
    }
  }
  __syncwarp();
}

// Rows of v in shared memory, the first two parts and the third apart: a quarter warp
// reads 64 bytes of each of two rows, then a half warp 32 of each of four, and with
// these strides no two lie in the same banks (but for rank 128, whose rows have to
// leave room for the base's and the residual's pieces).
__host__ __device__ constexpr int first_stride(int R) { return R * 4 % 128 == 64 ? R * 4 : R * 4 + 64; }
__host__ __device__ constexpr int last_stride(int R) { return R * 2 % 64 == 32 ? R * 2 : R * 2 + (R < 128 ? 32 : 16); }
struct Held {  // v of some rows in shared memory
  unsigned char *first, *last;
  int first_row, last_row;
  __device__ __forceinline__ Held(unsigned char* at, int rows, int R)
      : first(at), last(at + rows * first_stride(R)), first_row(first_stride(R)), last_row(last_stride(R)) {}
  // four ranks, quad q of step s
  __device__ __forceinline__ uint4* first_of(int row, int s, int q) const {
    return reinterpret_cast<uint4*>(first + row * first_row + s * 64 + q * 16);
  }
  __device__ __forceinline__ uint2* last_of(int row, int s, int q) const {
    return reinterpret_cast<uint2*>(last + row * last_row + s * 32 + q * 8);
  }
  __device__ __forceinline__ Parts get(int row, int s, int q, bool live) const {
    Parts w = {make_uint4(0, 0, 0, 0), make_uint2(0, 0)};
    if (live) w = {*first_of(row, s, q), *last_of(row, s, q)};
    return w;
  }
};
__host__ __device__ constexpr int held_bytes(int rows, int R) { return rows * (first_stride(R) + last_stride(R)); }
// Few rows: everything in one launch.  A cluster of eight CTAs takes one of a
// tile's runs and a share of the columns: its 64 warps split K, their sums meet in
// shared memory (the warps' of a CTA, then the CTAs' through the cluster), every CTA
// keeps v in parts, and its warps go through their strips.  Grid: 8 shares of the
// columns x slots (of a tile's runs; a cluster without one ends) x tiles.
constexpr int kCluster = 8;
template <int RT>
constexpr int few_bytes(int R) {
  return kWarps * kTile * (8 * RT + 4) * 4 + held_bytes(kTile, R);
}
template <bool VEC, bool INT8, int KS, bool BIG>
__global__ void __launch_bounds__(kWarps * 32) few_kernel(const LowRankParams p) {
  namespace cg = cooperative_groups;
  if (p.mode_dev != nullptr && SIXBIT_MODE_OF(*p.mode_dev) != SIXBIT_MODE_INT8) return;
  extern __shared__ __align__(16) float part[];  // [kWarps][kTile][kP], then v's parts
  __shared__ int scratch[kWarps][32];
  __shared__ float turns[VEC ? 1 : kWarps][16 * 33];
  constexpr int RT = 2 * KS, kP = 8 * RT + 4;
  const Held vs(reinterpret_cast<unsigned char*>(part + kWarps * kTile * kP), kTile, p.R);
  const auto cluster = cg::this_cluster();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, q = lane & 3;
  const int rank = blockIdx.x % kCluster;
  const Tile t = tile_of_few(p, blockIdx.z * kTile, scratch[warp], blockIdx.x == 0 && blockIdx.y == 0 && warp == 0);
  uint32_t left = t.heads;
  for (int turn = 0; left != 0; ++turn, left &= left - 1) {  // (the same in the whole cluster)
    if (turn % gridDim.y != blockIdx.y) continue;
    const int first = __ffs(left) - 1, id = __shfl_sync(kAll, t.id, first), count = run_length(t, first);
    if (id >= 0) {
      size_t at[4];
      bool live[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        live[i] = g8 + 8 * i < count;
        at[i] = static_cast<size_t>(__shfl_sync(kAll, t.row, (first + g8 + 8 * i) & 31)) * p.K;
      }
      const float alpha = p.alpha != nullptr ? __ldg(p.alpha + id) : 1.f;
      for (int r0 = 0; r0 < p.R; r0 += 8 * RT) {
        const int tiles = min(RT, (p.R - r0) / 8), quads = 2 * tiles;
        sums_of<INT8, RT>(p, p.a + (static_cast<size_t>(id) * p.R + r0 + g8) * p.K, tiles, at, live, count,
                          rank * kWarps + warp, kCluster * kWarps, part + warp * kTile * kP);
        __syncthreads();
        for (int i = threadIdx.x; i < count * quads; i += kWarps * 32) {
          float4* mine = reinterpret_cast<float4*>(&part[(i / quads) * kP + i % quads * 4]);
          float4 v = *mine;
#pragma unroll
          for (int w = 1; w < kWarps; ++w) {
            const float4 f = mine[w * kTile * kP / 4];
            v.x += f.x, v.y += f.y, v.z += f.z, v.w += f.w;
          }
          *mine = v;
        }
        cluster.sync();
        for (int i = threadIdx.x; i < count * quads; i += kWarps * 32) {
          const int n = i / quads, r = i % quads * 4, row = scratch[0][first + n];
          float v[4] = {};
#pragma unroll
          for (int z = 0; z < kCluster; ++z) {
            const float4 f = *reinterpret_cast<const float4*>(&cluster.map_shared_rank(part, z)[n * kP + r]);
            v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
          }
          const float f = (INT8 ? __ldg(p.row_scale + row) : 1.f) * alpha;
#pragma unroll
          for (int c = 0; c < 4; ++c) v[c] *= f;
          const Parts w = parts_of(v);
          *vs.first_of(n, 0, (r0 + r) / 4) = w.first;
          *vs.last_of(n, 0, (r0 + r) / 4) = w.last;
        }
        cluster.sync();  // (no CTA writes its sums again, or leaves, while another reads them)
      }
    }
    for (int n0 = (blockIdx.x * kWarps + warp) * 32; n0 < p.N; n0 += gridDim.x * kWarps * 32) {
      const int n = n0 + 8 * q;
      for (int m = 0; m < count; m += 16) {
        size_t row[2];
        bool live[2];
        Eight<true> wide[2] = {};
        Eight<false> base[2] = {};
        uint4 res[2] = {};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          live[h] = g8 + 8 * h < count - m;
          row[h] = static_cast<size_t>(__shfl_sync(kAll, t.row, (first + m + g8 + 8 * h) & 31));
          if (VEC && live[h] && n < p.N) {
            if (p.base_f32 != nullptr)
              wide[h].load(p, row[h] * p.N + n);
            else
              base[h].load(p, row[h] * p.N + n);
            if (p.epilogue == SIXBIT_EPI_RESIDUAL) res[h] = *reinterpret_cast<const uint4*>(p.residual + row[h] * p.N + n);
          }
        }
        float add[16];
        if constexpr (!VEC) turn_load(p, scratch[warp] + first + m, count - m, n0 + lane, add);
        float acc[4][4] = {};
        if (id >= 0) {
          for (int s0 = 0; s0 < (BIG ? p.R / 16 : KS); s0 += KS) {
            Strip<KS> strip;
            strip.load(p, id, n0, s0);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
              if (BIG && s0 + s >= p.R / 16) break;
              step_mma(acc, vs.get(m + g8, s0 + s, q, live[0]), vs.get(m + g8 + 8, s0 + s, q, live[1]), strip.b[s]);
            }
          }
        }
        if constexpr (VEC) {
          if (p.epilogue == SIXBIT_EPI_RESIDUAL) {
            if (p.base_f32 != nullptr)
              finish_rows<true, true>(p, acc, row, live, n, wide, res);
            else
              finish_rows<false, true>(p, acc, row, live, n, base, res);
          } else if (p.base_f32 != nullptr) {
            finish_rows<true, false>(p, acc, row, live, n, wide, res);
          } else {
            finish_rows<false, false>(p, acc, row, live, n, base, res);
          }
        } else {
          turn_rows(p, acc, scratch[warp] + first + m, count - m, n0, add, turns[warp]);
        }
      }
    }
  }
}

// More rows.  Grid: groups of eight strips x chunks of positions, whose v, rows and
// tiles (up to 16 positions of one adapter) the CTA keeps in shared memory.  Each
// lane copies the base, and the residual, of its outputs some tiles ahead into
// pieces of its own: with one tile ahead, in registers, 16 KB an SM were on their
// way, a quarter of what it takes.  Four tiles for rank 16, whose v is small, and two
// above it, which leaves room for longer chunks (17,776 x 7680: rank 16 119 us and 124
// with three; rank 32 to GELU 215, and 225 with three).
__host__ __device__ constexpr int ahead_of(int KS) { return KS == 1 ? 4 : 2; }
// Pieces of 16 bytes a lane has of each row: base, residual.
template <bool VEC, bool F32>
__host__ __device__ constexpr int pieces_of(bool residual) {
  return !VEC ? 0 : (F32 ? 2 : 1) + (residual ? 1 : 0);
}
template <bool VEC, bool F32, int KS>
constexpr int many_bytes(int chunk, int R, bool residual) {
  return (3 * chunk + 48) * 4 + held_bytes(chunk + 16, R) + kWarps * ahead_of(KS) * 1024 * pieces_of<VEC, F32>(residual);
}
static_assert(many_bytes<true, true, 4>(kTile, SIXBIT_MAX_RANK, true) <= kManyBytes, "the smallest chunk fits");
template <bool VEC, bool F32, bool RES, int KS, bool BIG>
__global__ void __launch_bounds__(kWarps * 32, 2) many_kernel(const LowRankParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float turns[VEC ? 1 : kWarps][16 * 33];
  __shared__ int counts[kWarps];
  constexpr int kPieces = pieces_of<VEC, F32>(RES), kAhead = ahead_of(KS);
  const int padded = p.chunk + 16;
  int* rows = reinterpret_cast<int*>(smem);
  int* ids = rows + padded;
  int* tiles = ids + padded;  // where each begins, and the last ends
  const Held vs(smem + (3 * p.chunk + 48) * 4, padded, p.R);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, q = lane & 3;
  const int n0 = (blockIdx.x * kWarps + warp) * 32, n = n0 + 8 * q;
  unsigned char* ring = vs.last + padded * vs.last_row + warp * kAhead * 1024 * kPieces + lane * 16;
  before_done();
  if (p.mode_dev != nullptr && SIXBIT_MODE_OF(*p.mode_dev) != SIXBIT_MODE_INT8) return;
  for (int chunk = 0; chunk < p.chunks_per_cta; ++chunk) {
    const int64_t pos0 = (static_cast<int64_t>(blockIdx.y) * p.chunks_per_cta + chunk) * p.chunk;
    if (pos0 >= p.M) break;
    const int live_rows = static_cast<int>(min(static_cast<int64_t>(p.chunk), p.M - pos0));
    if (chunk > 0) __syncthreads();
    const int quads = p.R / 4;  // (a piece of 16 bytes each of the first parts, half of one of the last)
    const uint4* first = static_cast<const uint4*>(p.v) + pos0 * quads;
    const uint4* last = static_cast<const uint4*>(p.v_last) + pos0 * (quads / 2);
    for (int i = threadIdx.x; i < live_rows * quads; i += kWarps * 32) copy16(vs.first_of(i / quads, 0, i % quads), first + i, true);
    for (int i = threadIdx.x; i < live_rows * (quads / 2); i += kWarps * 32)
      copy16(vs.last_of(i / (quads / 2), 0, i % (quads / 2) * 2), last + i, true);
    copies_commit();
    for (int i = threadIdx.x; i < padded; i += kWarps * 32) {
      rows[i] = i < live_rows ? p.perm[pos0 + i] : 0;
      ids[i] = i < live_rows ? p.sid[pos0 + i] : INT_MAX;
    }
    __syncthreads();
    {
      const int i = threadIdx.x;  // (a chunk has no more positions than the CTA threads)
      bool begins = false;
      if (i < live_rows) {
        int lo = 0, hi = i;  // the first position of this one's adapter: they ascend
        while (lo < hi) {
          const int mid = (lo + hi) / 2;
          if (ids[mid] < ids[i])
            lo = mid + 1;
          else
            hi = mid;
        }
        begins = ((i - lo) & 15) == 0;
      }
      const uint32_t mask = __ballot_sync(kAll, begins);
      if (lane == 0) counts[warp] = __popc(mask);
      __syncthreads();
      int at = __popc(mask & ((1u << lane) - 1));
      for (int w = 0; w < warp; ++w) at += counts[w];
      if (begins) tiles[at] = i;
      if (i == kWarps * 32 - 1) tiles[at + (begins ? 1 : 0)] = live_rows;
    }
    copies_wait<0>();
    __syncthreads();
    if (n0 >= p.N) continue;
    int many = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) many += counts[w];
    auto ask = [&](int t) {
      if constexpr (VEC) {
        if (t < many && n < p.N) {
          const int at = tiles[t], end = tiles[t + 1];
          unsigned char* to = ring + (t % kAhead) * 1024 * kPieces;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int pos = at + g8 + 8 * h;
            if (pos >= end) continue;
            const size_t from = static_cast<size_t>(rows[pos]) * p.N + n;
            if constexpr (F32) {
              copy16(to + h * 512 * kPieces, p.base_f32 + from, true);
              copy16(to + h * 512 * kPieces + 512, p.base_f32 + from + 4, true);
            } else {
              if (p.base != nullptr) copy16(to + h * 512 * kPieces, p.base + from, true);
            }
            if constexpr (RES) copy16(to + h * 512 * kPieces + 512 * (kPieces - 1), p.residual + from, true);
          }
        }
        copies_commit();
      }
    };
#pragma unroll
    for (int t = 0; t < kAhead; ++t) ask(t);
    Strip<KS> strip;
    int held = -1;
    for (int t = 0; t < many; ++t) {
      const int at = tiles[t], count = tiles[t + 1] - at, id = ids[at];
      const bool live[2] = {g8 < count, g8 + 8 < count};
      const size_t row[2] = {static_cast<size_t>(rows[at + g8]), static_cast<size_t>(rows[at + g8 + 8])};
      float add[16];
      if constexpr (!VEC) turn_load(p, rows + at, count, n0 + lane, add);
      float acc[4][4] = {};
      if (id >= 0) {
        // (rows of the MMA that are not live hold anything: they stay apart)
        for (int s0 = 0; s0 < (BIG ? p.R / 16 : KS); s0 += KS) {
          if (BIG || held != id) strip.load(p, id, n0, s0);
          held = id;
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            if (BIG && s0 + s >= p.R / 16) break;
            step_mma(acc, vs.get(at + g8, s0 + s, q, true), vs.get(at + g8 + 8, s0 + s, q, true), strip.b[s]);
          }
        }
      }
      if constexpr (VEC) {
        copies_wait<kAhead - 1>();
        const unsigned char* mine = ring + (t % kAhead) * 1024 * kPieces;
        Eight<F32> base[2] = {};
        uint4 res[2] = {};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (F32 || p.base != nullptr) {
#pragma unroll
            for (int i = 0; i < (F32 ? 2 : 1); ++i)
              base[h].w[i] = *reinterpret_cast<const uint4*>(mine + h * 512 * kPieces + i * 512);
          }
          if constexpr (RES) res[h] = *reinterpret_cast<const uint4*>(mine + h * 512 * kPieces + 512 * (kPieces - 1));
        }
        ask(t + kAhead);
        finish_rows<F32, RES>(p, acc, row, live, n, base, res);
      } else {
        turn_rows(p, acc, rows + at, count, n0, add, turns[warp]);
      }
    }
    copies_wait<0>();
  }
}

// A launch that may start while the one before it on the stream runs (early), of
// clusters of this shape.
struct Launch {
  cudaLaunchAttribute attrs[2];
  cudaLaunchConfig_t cfg;
  Launch(dim3 grid, int threads, int smem, cudaStream_t st, bool early, dim3 cluster = dim3(1)) : cfg{} {
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attrs;
    if (early) {
      attrs[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attrs[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster.x * cluster.y * cluster.z > 1) {
      attrs[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
      attrs[cfg.numAttrs].val.clusterDim.x = cluster.x;
      attrs[cfg.numAttrs].val.clusterDim.y = cluster.y;
      attrs[cfg.numAttrs++].val.clusterDim.z = cluster.z;
    }
  }
};

template <bool VEC, bool INT8, int KS, bool BIG>
cudaError_t launch_few(const LowRankParams& p, cudaStream_t st) {
  const int smem = few_bytes<2 * KS>(p.R);
  const cudaError_t e =
      set_smem_once<few_kernel<VEC, INT8, KS, BIG>>(few_bytes<2 * KS>(BIG ? SIXBIT_MAX_RANK : 16 * KS));
  if (e != cudaSuccess) return e;
  // a cluster for each run there may be and a strip a warp, as far as all clusters come to about two CTAs an SM (above
  // rank 32 a CTA's 162 to 240 registers a thread leave room for one at a time, and the second follows it)
  const int strips = (p.N + 31) / 32, shares = (strips + kCluster * kWarps - 1) / (kCluster * kWarps);
  const int tiles = (p.M + kTile - 1) / kTile, all = 2 * sm_count() / kCluster / tiles, rows = p.M < kTile ? p.M : kTile;
  const int slots = rows < all || tiles == 1 ? rows : all, most = all / slots > 0 ? all / slots : 1;
  Launch l(dim3(kCluster * (shares < most ? shares : most), slots, tiles), kWarps * 32, smem, st, false, dim3(kCluster));
  note_launch();
  return cudaLaunchKernelEx(&l.cfg, few_kernel<VEC, INT8, KS, BIG>, p);
}

template <bool VEC, bool INT8>
cudaError_t launch_few(const LowRankParams& p, cudaStream_t st) {
  switch (p.R) {
    case 16: return launch_few<VEC, INT8, 1, false>(p, st);
    case 32: return launch_few<VEC, INT8, 2, false>(p, st);
    case 48: return launch_few<VEC, INT8, 3, false>(p, st);
    case 64: return launch_few<VEC, INT8, 4, false>(p, st);
    default: return launch_few<VEC, INT8, 4, true>(p, st);
  }
}

template <bool INT8, int RT>
cudaError_t launch_shrink(const LowRankParams& p, cudaStream_t st) {
  // For many rows x and A pass through shared memory: K 1920, rank 64, 2047 rows 44 us
  // against 56, but 1024 mixed ones 50 against 42; rank 16, 2047 rows 30.6 against 30.2,
  // 4096 44.1 against 44.0, 8192 69 against 70.  (The border lies where mixed rows need
  // it: rows in runs would gain from 1024 on at K 7680, 56 against 60, mixed ones lose,
  // 96 against 64.)
  if (p.M >= (p.R > 32 ? 1536 : 4096)) {
    constexpr int smem = Staged<INT8, RT>::kBytes;
    const cudaError_t e = set_smem_once<staged_kernel<INT8, RT>>(smem);
    if (e != cudaSuccess) return e;
    Launch l(dim3((p.M + kBlock - 1) / kBlock, (p.R + 8 * RT - 1) / (8 * RT), 2), kStagedThreads, smem, st, true);
    note_launch();
    return cudaLaunchKernelEx(&l.cfg, staged_kernel<INT8, RT>, p);
  }
  constexpr int smem = kWarps * kTile * (8 * RT + 4) * 4;
  const cudaError_t e = set_smem_once<shrink_kernel<INT8, RT>>(smem);
  if (e != cudaSuccess) return e;
  // about two CTAs an SM: first up to four for a tile's runs, then K over clusters
  const int tiles = (p.M + kTile - 1) / kTile, ctas = 2 * sm_count();
  const int most = ctas / tiles > 0 ? ctas / tiles : 1, slots = most < 4 ? most : 4;
  const int turns = (p.K / kUnit + kWarps - 1) / kWarps, left = most / slots > 0 ? most / slots : 1;
  int splits = turns < left ? turns : left;
  if (splits > kCluster) splits = kCluster;
  Launch l(dim3(tiles, slots, splits), kWarps * 32, smem, st, true, dim3(1, 1, splits));
  note_launch();
  return cudaLaunchKernelEx(&l.cfg, shrink_kernel<INT8, RT>, p);
}

template <bool INT8>
cudaError_t launch_shrink(const LowRankParams& p, cudaStream_t st) {
  if (p.R <= 16) return launch_shrink<INT8, 2>(p, st);
  if (p.R <= 32) return launch_shrink<INT8, 4>(p, st);
  if (p.R == 48 || p.R == 96) return launch_shrink<INT8, 6>(p, st);
  return launch_shrink<INT8, 8>(p, st);
}

template <bool VEC, bool F32, bool RES, int KS, bool BIG>
cudaError_t launch_many(LowRankParams p, cudaStream_t st) {
  // the largest chunks that let two CTAs share an SM (rank 64, residual: 160 positions), smaller ones where they would leave SMs idle
  const int groups = ((p.N + 31) / 32 + kWarps - 1) / kWarps;
  p.chunk = kChunk;
  while (many_bytes<VEC, F32, KS>(p.chunk, p.R, RES) > kManyBytes) p.chunk -= kTile;
  while (p.chunk > kTile && static_cast<int64_t>(groups) * ((p.M + p.chunk - 1) / p.chunk) < 2 * sm_count())
    p.chunk = p.chunk / 2 > kTile ? (p.chunk / 2 + 15) / 16 * 16 : kTile;
  const int chunks = (p.M + p.chunk - 1) / p.chunk;
  p.chunks_per_cta = (chunks + 65534) / 65535;
  const cudaError_t e = set_smem_once<many_kernel<VEC, F32, RES, KS, BIG>>(kManyBytes);
  if (e != cudaSuccess) return e;
  Launch l(dim3(groups, (chunks + p.chunks_per_cta - 1) / p.chunks_per_cta), kWarps * 32,
           many_bytes<VEC, F32, KS>(p.chunk, p.R, RES), st, true);
  note_launch();
  return cudaLaunchKernelEx(&l.cfg, many_kernel<VEC, F32, RES, KS, BIG>, p);
}

template <bool VEC, bool F32, bool RES>
cudaError_t launch_many(const LowRankParams& p, cudaStream_t st) {
  switch (p.R) {
    case 16: return launch_many<VEC, F32, RES, 1, false>(p, st);
    case 32: return launch_many<VEC, F32, RES, 2, false>(p, st);
    case 48: return launch_many<VEC, F32, RES, 3, false>(p, st);
    case 64: return launch_many<VEC, F32, RES, 4, false>(p, st);
    default: return launch_many<VEC, F32, RES, 4, true>(p, st);
  }
}

cudaError_t launch(const LowRankParams& p, cudaStream_t st) {
  const auto a16 = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; };
  const bool vec = p.N % 8 == 0 && a16(p.base) && a16(p.base_f32) && a16(p.residual) && a16(p.Y) && a16(p.Yf);
  const bool int8 = p.codes != nullptr, f32 = p.base_f32 != nullptr;
  if (p.M <= few_rows(p.R)) {
    if (vec) return int8 ? launch_few<true, true>(p, st) : launch_few<true, false>(p, st);
    return int8 ? launch_few<false, true>(p, st) : launch_few<false, false>(p, st);
  }
  const cudaError_t e = int8 ? launch_shrink<true>(p, st) : launch_shrink<false>(p, st);
  if (e != cudaSuccess) return e;
  if (!vec) return launch_many<false, false, false>(p, st);
  if (p.epilogue == SIXBIT_EPI_RESIDUAL)
    return f32 ? launch_many<true, true, true>(p, st) : launch_many<true, false, true>(p, st);
  return f32 ? launch_many<true, true, false>(p, st) : launch_many<true, false, false>(p, st);
}

}  // namespace lowrank

size_t lowrank_workspace(int M, int R) {
  // v in three parts, the rows' order and their adapters
  const size_t rows = static_cast<size_t>(M), order = (rows * 4 + 15) / 16 * 16;
  return M > lowrank::few_rows(R) ? rows * R * 6 + 2 * order : 0;
}

cudaError_t launch_lowrank(LowRankParams p, void* workspace, cudaStream_t st) {
  if (p.M > lowrank::few_rows(p.R)) {
    const size_t order = (static_cast<size_t>(p.M) * 4 + 15) / 16 * 16;
    p.perm = static_cast<int32_t*>(workspace);
    p.sid = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + order);
    p.v = static_cast<uint8_t*>(workspace) + 2 * order;
    p.v_last = static_cast<uint8_t*>(p.v) + static_cast<size_t>(p.M) * p.R * 4;
    const int smem = 2 * (p.L + 1) * 4;
    cudaError_t e = set_smem_once<lowrank::plan_kernel>(2 * (SIXBIT_MAX_ADAPTERS + 1) * 4);
    if (e != cudaSuccess) return e;
    // (a cluster where one CTA would go around more than once)
    const int ctas = p.M > lowrank::kPlanAtOnce * lowrank::kPlanThreads ? lowrank::kPlanCluster : 1;
    lowrank::Launch l(dim3(ctas), lowrank::kPlanThreads, smem, st, false, dim3(ctas));
    note_launch();
    e = cudaLaunchKernelEx(&l.cfg, lowrank::plan_kernel, p);
    if (e != cudaSuccess) return e;
  }
  return lowrank::launch(p, st);
}

}  // namespace sixbit
