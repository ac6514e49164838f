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
//
// A team of W warps takes a row, V chunks of 16 elements a lane, which stay in
// registers from the load to the store; each warp's part of the next row is copied
// to shared memory in the meantime.  (A warp has what it does for a row as such
// -- three reductions, the factors, the addresses -- once for 512 V elements; with
// four warps of one chunk a lane that was a third of all instructions.)  Up to
// three factors a channel remain when those of the same place are joined: post_w .
// gate, w . (1 + scale) and shift.  A CTA takes neighbouring rows and keeps those of
// a window of segments, as many as fit, in shared memory; where its rows leave the
// window it is filled anew, unless few rows would use it: they join them as they go.
// An absent operand is a factor of 1 or a shift of 0, so that nothing branches.
//
// The floor is bytes: 7 an element, 8 with bf16 rows.  17,776 x 1920 with every
// operand 51 us (4.7 TB/s, 69% of a copy; 47 without gate, scale and shift), 4,444
// x 7680 67, 2,777 x 12288 79; 1,003 x 7680 gated, to bf16, 23 (floor 9); one row
// 3.5, 226 rows 4.8.  It is bound by issue and dependence: some 385 instructions a
// warp for 512 elements, which issue in half of the cycles.  (A CTA a row, one chunk
// a lane: 66 us, 730 instructions; two rows a CTA at once spilled and took 74.  Four
// chunks a lane spill too, 60 to 200 bytes a thread, read again in L1.)
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "ctx_cache.h"
#include "internal.h"
#include "row_norm.cuh"

namespace sixbit {
namespace gnorm {

constexpr int kWarps = 16;              // of a CTA
constexpr int kSmemBytes = 224 * 1024;  // copies and factors

struct Params {
  GatedNormParams g;
  float inv_sqrt_b, inv_k;
  int b;     // of the rotation
  int wide;  // x, res, sum_out, y are 32-byte aligned
  int held;  // segments whose factors are in shared memory
  int rows;  // of a CTA
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Sums and maxima of a team's warps; two buffers, so that the next row's writes need
// no barrier of their own.
template <int W>
struct Joint {
  float ss[2][W];
  uint32_t mx[2][W];
};
template <int W>
__device__ __forceinline__ void team_sync(int team) {
  asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(32 * W) : "memory");
}
template <int W>
__device__ __forceinline__ float team_sum(float v, Joint<W>& j, int buf, int team, int rank) {
  v = warp_sum(v);
  if constexpr (W > 1) {
    if ((threadIdx.x & 31) == 0) j.ss[buf][rank] = v;
    team_sync<W>(team);
    v = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) v += j.ss[buf][i];
  }
  return v;
}
// 1 / sqrt(ss / K + eps); NaN for a sum that is not finite.
__device__ __forceinline__ float row_factor(float ss, float inv_k, float eps) {
  const float r = rsqrtf(fmaf(ss, inv_k, eps));
  return finite_sum(ss) ? r : __uint_as_float(0x7FC00000u);
}
// max over |u|, a NaN above all
__device__ __forceinline__ float max_abs(const uint64_t (&u)[8], float m) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(f2_lo(u[i])), "f"(f2_hi(u[i])));
  return m;
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

// The joined factors of segment `seg`, channels k .. k + 15: 0 the branch's, 1 the
// norm's, 2 the shift.
__device__ __forceinline__ void join(const GatedNormParams& g, int which, int seg, int k, uint64_t (&a)[8]) {
  const size_t at = static_cast<size_t>(seg) * g.K + k;
  if (which == 2) {
    load16f(g.shift != nullptr ? g.shift + at : nullptr, 0.f, a);
    return;
  }
  uint64_t b[8];
  if (which == 0) {
    load16f(g.post_w != nullptr ? g.post_w + k : nullptr, 1.f, a);
    load16f(g.gate != nullptr ? g.gate + at : nullptr, 1.f, b);
  } else {
    load16f(g.w != nullptr ? g.w + k : nullptr, 1.f, a);
    load16f(g.scale != nullptr ? g.scale + at : nullptr, 0.f, b);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = which == 0 ? f2_mul(a[i], b[i]) : f2_fma(a[i], b[i], a[i]);
}
// They lie in shared memory as [segment][3][4][chunks] pieces of 16 bytes.
__device__ __forceinline__ void put(float4* to, int chunks, const uint64_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    to[i * chunks] = make_float4(f2_lo(w[2 * i]), f2_hi(w[2 * i]), f2_lo(w[2 * i + 1]), f2_hi(w[2 * i + 1]));
}
__device__ __forceinline__ void get(const float4* from, int chunks, uint64_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 f = from[i * chunks];
    w[2 * i] = f2_pack(f.x, f.y);
    w[2 * i + 1] = f2_pack(f.z, f.w);
  }
}

// The unscaled butterfly of blocks of b (0: none) across a warp's chunks.
template <int V>
__device__ __forceinline__ void rotate(uint64_t (&u)[V][8], int b) {
  if (b == 0) return;
#pragma unroll
  for (int v = 0; v < V; ++v) fwht<16>(u[v]);
  const int lane = threadIdx.x & 31;
  for (int h = 1; h < b / kChunk; h <<= 1) {
    const float sg = (lane & h) ? -1.f : 1.f;  // upper lane: other - mine
    const uint64_t s2 = f2_pack(sg, sg);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t o = __shfl_xor_sync(0xFFFFFFFFu, static_cast<unsigned long long>(u[v][i]), h);
        u[v][i] = f2_fma(u[v][i], s2, o);
      }
  }
}

template <int V, int W, bool STAGE>
__global__ void __launch_bounds__(kWarps * 32, 1) row_kernel(const Params p) {
  const GatedNormParams& g = p.g;
  if (g.mode_dev != nullptr && SIXBIT_MODE_OF(*g.mode_dev) != SIXBIT_MODE_INT8) return;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Joint<W> post[kWarps / W], pre[kWarps / W], top[kWarps / W];
  __shared__ uint64_t arrived[kWarps];
  constexpr int kPart = V * 32 * 32;  // bytes of a warp's part of a row
  constexpr int kTeams = kWarps / W, kFillRows = kTeams > 4 ? kTeams / 2 : 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, team = warp / W, rank = warp % W;
  const int chunks = g.K / kChunk, c0 = rank * 32 * V + lane;  // this lane's: c0 + 32 v
  unsigned char* part = smem + warp * (2 * kPart);             // x, then the residual
  float4* vec = reinterpret_cast<float4*>(smem + (STAGE ? kWarps * 2 * kPart : 0));
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.rows;
  const int64_t row1 = min(row0 + p.rows, static_cast<int64_t>(g.M));
  auto segment_of = [&](int64_t row) {
    return g.segment != nullptr ? __ldg(g.segment + row) : g.S > 1 ? static_cast<int>(row) / g.rows_per_seg : 0;
  };
  // this warp's part of a row on its way to shared memory (one lane; the others are past their last reads of it)
  auto fetch = [&](int64_t row) {
    const int bytes = min(32 * V, chunks - rank * 32 * V) * 32;
    const size_t at = static_cast<size_t>(row) * g.K + static_cast<size_t>(rank) * 32 * V * kChunk;
    mbar_expect_tx(&arrived[warp], g.res != nullptr ? 2 * bytes : bytes);
    bulk_load(part, g.x + at, bytes, &arrived[warp]);
    if (g.res != nullptr) bulk_load(part + kPart, g.res + at, bytes, &arrived[warp]);
  };
  const bool copies = STAGE && rank * 32 * V < chunks;
  if (STAGE) {
    if (g.res == nullptr)
      for (int i = lane; i < kPart / 16; i += 32) reinterpret_cast<uint4*>(part + kPart)[i] = make_uint4(0, 0, 0, 0);
    if (lane == 0) {
      mbar_init(&arrived[warp], 1);
      fence_barrier_init();
      if (copies && row0 + team < row1 && !g.withhold_first) fetch(row0 + team);
    }
    __syncwarp();
  }
  uint32_t buf = 0, lost = 0;
  bool dead = false;  // a copy did not arrive in time: reported, waited for no more, and this and later rows NaN

  // One row; HELD: its factors are in shared memory from `mine` on.
  auto process = [&](auto held, int64_t row, int seg, const float4* mine) {
    constexpr bool HELD = decltype(held)::value;
    auto factors = [&](int which, int v, uint64_t (&w)[8]) {
      if constexpr (HELD)
        get(mine + which * 4 * chunks + 32 * v, chunks, w);
      else
        join(g, which, seg, (c0 + 32 * v) * kChunk, w);
    };
    const size_t base = static_cast<size_t>(row) * g.K;
    uint32_t xr[V][8], rr[V][8];
    if (STAGE) {
      if (copies && !dead && !mbar_wait(&arrived[warp], buf, nullptr, g.wait_ns)) {
        dead = true;
        lost = buf;
        set_error(g.err, SIXBIT_ETIMEOUT);
      }
      if (dead) seg = -1;  // (what shared memory holds is another row's, or nothing)
    }
    auto part_of = [&](const unsigned char* from, int v, uint32_t (&r)[8]) {
      const uint4* q = reinterpret_cast<const uint4*>(from + (v * 32 + lane) * 32);
      const uint4 a = q[0], b = q[1];
      r[0] = a.x, r[1] = a.y, r[2] = a.z, r[3] = a.w, r[4] = b.x, r[5] = b.y, r[6] = b.z, r[7] = b.w;
    };
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = c0 + 32 * v;
#pragma unroll
      for (int i = 0; i < 8; ++i) xr[v][i] = rr[v][i] = 0;
      if (c < chunks) {
        if (STAGE)
          part_of(part, v, xr[v]);
        else
          load32(g.x + base + static_cast<size_t>(c) * kChunk, p.wide, xr[v]);
      }
    }
    if (!STAGE && g.res != nullptr) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (c0 + 32 * v < chunks) load32(g.res + base + static_cast<size_t>(c0 + 32 * v) * kChunk, p.wide, rr[v]);
    }
    if (seg < 0 || seg >= g.S) {
      seg = 0;
      if (lane == 0 && !dead) set_error(g.err, SIXBIT_EDEVICE);
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) xr[v][i] = 0x7FC07FC0u;  // (NaN)
    }
    uint64_t u[V][8], ss = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) u[v][i] = f2_from_bf16x2(xr[v][i]);
    float rpost = 1.f;
    if (g.post_w != nullptr) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = f2_fma(u[v][i], u[v][i], ss);
      rpost = row_factor(team_sum<W>(f2_lo(ss) + f2_hi(ss), post[team], buf, team, rank), p.inv_k, g.eps);
      ss = 0;
    }
    const uint64_t rp = f2_pack(rpost, rpost), rs = f2_pack(g.res_scale, g.res_scale);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = c0 + 32 * v;
      if (c >= chunks) continue;  // (u is 0)
      uint64_t w[8];
      factors(0, v, w);
      if (STAGE) part_of(part + kPart, v, rr[v]);
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        u[v][i] = f2_fma(f2_from_bf16x2(rr[v][i]), rs, f2_mul(f2_mul(u[v][i], rp), w[i]));
        o[i] = f2_to_bf16x2(u[v][i]);
        ss = f2_fma(u[v][i], u[v][i], ss);
      }
      if (g.sum_out != nullptr) store32(g.sum_out + base + static_cast<size_t>(c) * kChunk, p.wide, o);
    }
    if (STAGE) {
      __syncwarp();
      if (lane == 0 && copies && !dead && row + kTeams < row1) fetch(row + kTeams);
    }
    const float rpre = row_factor(team_sum<W>(f2_lo(ss) + f2_hi(ss), pre[team], buf, team, rank), p.inv_k, g.eps);
    const uint64_t r2 = f2_pack(rpre, rpre);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (c0 + 32 * v >= chunks) continue;
      uint64_t w[8], t[8];
      factors(1, v, w);
      factors(2, v, t);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[v][i] = f2_fma(f2_mul(u[v][i], r2), w[i], t[i]);
    }
    if (g.y != nullptr) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = c0 + 32 * v;
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = f2_to_bf16x2(u[v][i]);
        if (c < chunks) store32(g.y + base + static_cast<size_t>(c) * kChunk, p.wide, o);
      }
      return;
    }
    float m = 0.f;
    rotate<V>(u, p.b);  // (every lane of the warp takes part)
#pragma unroll
    for (int v = 0; v < V; ++v) m = max_abs(u[v], m);
    uint32_t mb = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m) & 0x7FFFFFFFu);
    if constexpr (W > 1) {
      if (lane == 0) top[team].mx[buf][rank] = mb;
      team_sync<W>(team);
      mb = 0;
#pragma unroll
      for (int i = 0; i < W; ++i) mb = max(mb, top[team].mx[buf][i]);
    }
    const RowOut o = row_out(p.inv_sqrt_b, true, mb);
    if (lane == 0 && rank == 0) g.row_scale[row] = o.scale;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = c0 + 32 * v;
      if (c < chunks) store_codes(g.codes + base + static_cast<size_t>(c) * kChunk, o, u[v]);
    }
  };

  int64_t row = row0 + team;
  for (int64_t from = row0; from < row1;) {  // (the same windows in every warp)
    int64_t to = row1;
    int seg0 = 0;
    bool fill = p.held > 0 && to - from >= kFillRows;
    if (p.held > 0 && p.held < g.S) {
      seg0 = min(max(segment_of(from), 0), g.S - p.held);
      for (int64_t r = from; r < row1; r += 32) {
        const int s = r + lane < row1 ? segment_of(r + lane) : seg0;
        const uint32_t out = __ballot_sync(0xFFFFFFFFu, s >= 0 && s < g.S && (s < seg0 || s >= seg0 + p.held));
        if (out != 0) {
          to = r + __ffs(out) - 1;
          break;
        }
      }
      fill = to - from >= kFillRows;
    }
    if (fill) {
      __syncthreads();  // (the last window's rows are done)
      for (int i = threadIdx.x; i < p.held * chunks; i += blockDim.x) {
        const int seg = i / chunks, c = i % chunks;
        uint64_t a[8];
#pragma unroll
        for (int which = 0; which < 3; ++which) {
          join(g, which, seg0 + seg, c * kChunk, a);
          put(vec + (static_cast<size_t>(seg) * 3 + which) * 4 * chunks + c, chunks, a);
        }
      }
      __syncthreads();
    }
    for (; row < to; row += kTeams, buf ^= 1) {
      const int seg = segment_of(row);
      if (fill && seg >= seg0 && seg < seg0 + p.held)
        process(std::true_type{}, row, seg, vec + static_cast<size_t>(seg - seg0) * 12 * chunks + c0);
      else
        process(std::false_type{}, row, seg, vec);
    }
    from = to;
  }
  if (STAGE && dead) mbar_wait(&arrived[warp], lost, nullptr, g.wait_ns);  // (the copy in flight, once more with a limit)
}

template <int V, int W, bool STAGE>
cudaError_t launch_rows(Params& p, int64_t grid, cudaStream_t st) {
  static_assert(kWarps % W == 0 && (W == 1 || kWarps / W <= 15), "a named barrier a team");
  const cudaError_t e = set_smem_once<row_kernel<V, W, STAGE>>(kSmemBytes);
  if (e != cudaSuccess) return e;
  const GatedNormParams& g = p.g;
  p.rows = static_cast<int>((static_cast<int64_t>(g.M) + grid - 1) / grid);
  int smem = STAGE ? kWarps * 2 * V * 1024 : 0;
  const int of_segment = 3 * g.K * 4;
  p.held = 0;
  if (p.rows > 1) {
    p.held = std::min(g.S, (kSmemBytes - smem) / of_segment);
    smem += p.held * of_segment;
  }
  note_launch();
  const int threads = p.rows == 1 ? 32 * W : 32 * kWarps;  // (one team has nothing to share a CTA with)
  row_kernel<V, W, STAGE><<<static_cast<unsigned>((g.M + p.rows - 1) / p.rows), threads, smem, st>>>(p);
  return cudaGetLastError();
}

// One chunk a lane and a row a CTA, the shortest way through a row, while all rows are
// resident at once, four CTAs an SM at most (1920: 304 rows 5.1 us against 10.3, 599
// 6.8 against 10.6, but 1200 12.3 against 9.6; 7680, a CTA an SM: 152 rows 7.2 against
// 11.0, 304 14.0 against 12.6).  Else teams of warps with four chunks a lane.
cudaError_t launch(Params& p, cudaStream_t st) {
  const int chunks = p.g.K / kChunk, sms = sm_count(), warps = (chunks + 31) / 32;
  if (p.g.M <= sms * (warps <= 4 ? 4 : warps <= 8 ? 2 : 1)) {
    if (warps == 1) return launch_rows<1, 1, false>(p, p.g.M, st);
    if (warps == 2) return launch_rows<1, 2, false>(p, p.g.M, st);
    if (warps <= 4) return launch_rows<1, 4, false>(p, p.g.M, st);
    if (warps <= 8) return launch_rows<1, 8, false>(p, p.g.M, st);
    if (warps <= 16) return launch_rows<1, 16, false>(p, p.g.M, st);
    return launch_rows<2, 16, false>(p, p.g.M, st);
  }
  if (warps == 1) return launch_rows<1, 1, true>(p, sms, st);
  if (warps == 2) return launch_rows<2, 1, true>(p, sms, st);
  if (warps <= 4) return launch_rows<4, 1, true>(p, sms, st);
  if (warps <= 8) return launch_rows<4, 2, true>(p, sms, st);
  if (warps <= 16) return launch_rows<4, 4, true>(p, sms, st);
  return launch_rows<4, 8, false>(p, sms, st);  // (copies and three factors of a row do not fit)
}

}  // namespace gnorm

cudaError_t launch_gated_norm(const GatedNormParams& g, int b, cudaStream_t st) {
  gnorm::Params p{};
  p.g = g;
  p.inv_k = 1.f / static_cast<float>(g.K);
  p.inv_sqrt_b = b == 16 ? 0.25f : b == 64 ? 0.125f : b == 256 ? 0.0625f : 1.f;
  const auto a32 = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 31u) == 0; };
  p.wide = a32(g.x) && a32(g.res) && a32(g.sum_out) && a32(g.y);
  p.b = b;
  return gnorm::launch(p, st);
}

}  // namespace sixbit
