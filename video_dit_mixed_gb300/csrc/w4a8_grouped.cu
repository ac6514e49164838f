// W4A8 product grouped by expert on the tcgen05 tensor cores of sm_103a:
// ragged row counts on the device, INT4 weights read as they are stored
// (technical summary sections 2.A and 4; the dense GEMM is qgemm_w4a8.cu).
//
//   rows m of expert e:  Y[m, n] = s_m[m] * sum_g s_w[e][g][n] * acc_g[m, n]
//   acc_g[m, n] = sum_{k in group g} qa[m, k] * qw[e][n, k]   (exact integers)
//
// Integers run through kind::f8f6f4 as E4M3, whose codes 0 .. 15 are the
// integers 0 .. 15 in units of 2^-9.  A weight is one such code with its sign;
// a token's code q is two digits, q = 16 h + l, l a code 0 .. 15 and h (-8 .. 7)
// the E4M3 of h 2^-5.  Both products go into one FP32 accumulator, whose 2^18
// fold is the group's exact integer (below 2^18); the group's scale is applied
// when it is read back.  Two E4M3 MMAs take as long as one in fp16, and the
// operands half the tensor memory and, for a weight, a third of the conversion.
//
// The operands' roles are the dense GEMM's swapped.  There the weights are
// expanded to fp16 in memory once per call, which many rows pay for; an expert
// with few rows cannot pay 4.5 bytes of traffic for a weight that holds half
// of one.  Here the 128 weight rows of a tile are the A operand in tensor
// memory: converter warps take the nibbles from shared memory, turn them into
// E4M3 in registers and store them into the row's tensor-memory lane.  The
// tokens are the B operand in shared memory; their codes are expanded to
// digits once per call (2 bytes a code, written and read mostly in L2).  A
// byte's two nibbles go to different words, so within each eight inputs both
// operands hold the order 0 2 4 6 1 3 5 7.  An accumulator lane is a weight
// row, so a group's scale is one number a thread.
//
// Work.  A tile is 128 weight rows by up to NT rows of one expert; tiles are
// numbered expert by expert, weight tiles fastest, and a persistent CTA per SM
// takes every gridDim-th one, finding its expert by bisection in the prefix
// sums that each CTA takes of the row counts on entry.  All rings move by
// batches of GB groups.  The MMA's token count is the tile's own (rounded up
// to 16), as are the rows copied, so a ragged end costs what it holds.
//
// Two forms, by the mean rows of an expert:
//   NT = 96, GB = 2   24 warps.  17,776 tokens in two experts each of eight:
//                     up 7680 x 1920 920 us, down 1920 x 7680 450 us, 1.14
//                     PFLOP/s, 58% of what bf16 GEMMs reach here; 512 rows an
//                     expert 121 us.  Bound by the round of an accumulator
//                     (MMAs 700 - 800 cycles, fold 1,000, and some 700 of
//                     barriers between them, two in flight), not by the tensor
//                     cores (768 cycles a batch), the converters (850) or
//                     memory.  Larger tiles spill in the fold (128: 1066 us),
//                     one fold team leaves the epilogue alone (1070 us), two
//                     teams that share a tile as well (1295 us).
//   NT = 32, GB = 4   20 warps.  452 rows over 64 experts of 7680 x 1920 92 us
//                     (5.1 TB/s of the weights' bytes, 76% of a copy), 32 rows
//                     over 64 39 us, 16 over 8 16.5 us.  Bound by the weights'
//                     bytes and, close behind, by the fold.  Its weights are
//                     v + 8 (no sign to convert: the integer pipe bound it
//                     before, 102 us), which the fold takes out with the sums of
//                     the tokens' codes.  Tiles of up to 16 rows take both
//                     digits in one MMA, as 32 columns that the fold adds (32
//                     over 64 experts: 52 -> 43 us).
//
// Warps:
//   0       TMA producer: 128 x 128-byte nibble tiles (two groups each); asks
//           L2 for the scales
//   2       TMA producer: a batch of tokens in one 3-D box (eight copies a batch
//           paced the narrow form)
//   1, 3    MMA issuers, even and odd batches (one issuer's waits leave the
//           tensor core idle, as measured in the dense GEMM); warp 1 also
//           allocates tensor memory
//   4 ..    converters, one warp per 32-lane quarter and two groups
//   ..      two fold teams, alternate tiles, so that one team's epilogue runs
//           beside the other's batches
// A batch's MMAs are followed by three commits: onto its accumulator's barrier
// of the team that folds the tile (each team has barriers of its own, so that
// it sees every phase of those it waits on), its A slot's and its token slot's.
//
// Every mbarrier wait is bounded; on expiry the kernel records
// SIXBIT_ETIMEOUT, raises the abort flag, waits (bounded) for its copies and
// tensor-core work in flight, frees tensor memory and returns.
#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "ctx_cache.h"
#include "gemm_common.cuh"
#include "internal.h"
#include "w4a8_common.cuh"

namespace sixbit {
namespace grouped {

constexpr int kBM = 128;           // weight rows of a tile
constexpr int kConvWarp0 = 4;
constexpr int kPairBytes = kBM * 128;  // nibbles of two groups: 128 rows of 128 bytes, 128-byte swizzle

// NT: tokens of a tile.  GB: groups of a batch, the unit of every ring.  SW, SX,
// NA, NB: slots of the nibble, token, A and accumulator rings.
template <bool NARROW>
struct Cfg;
template <>
struct Cfg<false> {
  static constexpr int NT = 96, GB = 2, SW = 2, SX = 3, NA = 2, NB = 2, kTeams = 2, kTeamWarps = 8;
  // Registers: 24 warps launch with 80 each; warps 0 - 3 keep 48, the converters
  // 80, the fold warps get 88.  (With 64 sums a thread they need 96 and more,
  // and the spilled ones cost each batch a round trip to L2.)
  static constexpr int kRegs = 80, kRegsLow = 48, kRegsConv = 80, kRegsFold = 88;
};
template <>
struct Cfg<true> {
  static constexpr int NT = 32, GB = 4, SW = 3, SX = 3, NA = 2, NB = 2, kTeams = 2, kTeamWarps = 4;
  // 20 warps of 96; 32 sums and two groups' loads in flight
  static constexpr int kRegs = 96, kRegsLow = 56, kRegsConv = 64, kRegsFold = 144;
};
template <bool NARROW>
struct Smem {
  using C = Cfg<NARROW>;
  static constexpr int kConv = 4 * (C::GB / 2), kFold = C::kTeamWarps * C::kTeams;  // warps
  static constexpr int kWarps = kConvWarp0 + kConv + kFold, kThreads = 32 * kWarps;
  static constexpr int kCols = C::NT / (C::kTeamWarps / 4);  // tokens of a fold thread
  static constexpr int kBox = token_box(NARROW);
  static constexpr int kXSlot = C::GB * C::NT * 256, kWSlot = (C::GB / 2) * kPairBytes;
  // a fold warp's row scales, and the narrow form's sums of codes
  static constexpr int kWarpArea = kCols * 4 * (NARROW ? 1 + C::GB : 1);
  static constexpr int kBars = 2 * C::SW + 2 * C::SX + 2 * C::NA + (C::kTeams + 1) * C::NB + 3;
  static constexpr int kX = 0, kW = C::SX * kXSlot, kFoldArea = kW + C::SW * kWSlot,
                       kBarAt = kFoldArea + kFold * kWarpArea, kTables = kBarAt + kBars * 8 + 16;
  static constexpr int kAccCols = C::GB * C::NT, kACol0 = C::NB * kAccCols, kACols = C::GB * 32;
  static_assert(C::NT == token_maps(NARROW) * kBox && 2 * C::GB == token_chunks(NARROW), "the token maps' boxes");
  static_assert(kACol0 + C::NA * kACols <= 512, "tensor memory columns");
  // The register split must fit in what the CTA is launched with;
  // setmaxnreg.dec may not raise a warp's count, nor .inc lower it.
  static_assert(4 * C::kRegsLow + kConv * C::kRegsConv + kFold * C::kRegsFold <= kWarps * C::kRegs &&
                    C::kRegsLow <= C::kRegs && C::kRegsConv <= C::kRegs && C::kRegsFold >= C::kRegs,
                "register split");
  // tables: prefix [E + 1], first row [E], rows [E]
  static size_t bytes(int E) { return 1024 + kTables + static_cast<size_t>(3 * E + 1) * 4; }
};
static_assert(Smem<false>::kTables + 1024 + (3 * SIXBIT_MAX_EXPERTS + 1) * 4 <= 227 * 1024, "shared memory per CTA");
static_assert(Smem<true>::kTables + 1024 + (3 * SIXBIT_MAX_EXPERTS + 1) * 4 <= 227 * 1024, "shared memory per CTA");

// Eight nibbles -> E4M3 of v 2^-9, or OFFSET, of (v + 8) 2^-9, even k in
// `even`, odd k in `odd`.  E4M3 codes 0 .. 15 (its subnormals and first binade)
// are the value in units of 2^-9, so a byte needs only sign and magnitude:
// v >= 0 stays, v < 0 becomes 0x90 - (v + 16) = ((v + 16) ^ 15) + 0x81.  With
// the offset it needs no more than the nibble, its sign bit flipped: three
// instructions instead of eleven, for which the fold takes the offset out.
template <bool OFFSET>
__device__ __forceinline__ void nibbles(uint32_t w, uint32_t& even, uint32_t& odd) {
  if (OFFSET) {
    even = (w & 0x0F0F0F0Fu) ^ 0x08080808u;
    odd = ((w >> 4) & 0x0F0F0F0Fu) ^ 0x08080808u;
  } else {
    const uint32_t ne = (w >> 3) & 0x01010101u, no = (w >> 7) & 0x01010101u;  // negative
    even = ((w & 0x0F0F0F0Fu) ^ (ne * 15u)) + ne * 0x81u;
    odd = (((w >> 4) & 0x0F0F0F0Fu) ^ (no * 15u)) + no * 0x81u;
  }
}

// The kernel may start while the digits' kernel runs (programmatic dependent
// launch): what reads its results waits for its end here.  The producer of
// every CTA does, so that this kernel never ends first.
__device__ __forceinline__ void digits_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// One lane of the (converged) warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// D[tmem] (+)= A[tmem] * B[smem]^T, E4M3 inputs, fp32 accumulate.  The first
// of two MMAs with the same A leaves it in the collector buffer, the second
// takes it from there.
__device__ __forceinline__ void mma_e4m3_fill(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4.collector::a::fill [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_e4m3_lastuse(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, 1, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4.collector::a::lastuse [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc)
      : "memory");
}

// How a tile's outputs are written.  kPair*: bf16, N even and below 2^30 (two
// rows' bytes are a 32-bit step there), Y and residual 4-byte aligned:
// neighbouring lanes exchange one value of each two tokens, so that a lane
// holds two outputs of one token and a store writes 4 bytes.  kAny:
// whatever else, one output at a time.  They are forms of the kernel: one code
// path a kernel, since its instruction fetch (92% hits) paced the epilogue.
enum Out { kPair, kPairGelu, kPairResidual, kAny };

__device__ __forceinline__ void gelu16(float (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    const uint64_t g = gelu_pair(f2_pack(v[j], v[j + 1]));
    v[j] = f2_lo(g);
    v[j + 1] = f2_hi(g);
  }
}

// The epilogue and the store of 16 tokens (rows row .. row + 15 of Y, the first
// `left` of them valid) of output column n, one column a lane.
template <Out OUT>
__device__ __forceinline__ void store16(const RowsParams& p, size_t row, int n, int left, int lane, float (&v)[16]) {
  if constexpr (OUT != kAny) {
    if constexpr (OUT == kPairGelu) gelu16(v);
    const int odd = lane & 1, nb = n & ~1;
    const uint32_t sel = odd ? 0x3276u : 0x5410u;  // own and other -> columns (n, n + 1) of token j, or of j + 1
    const int some = nb < p.N ? left - odd : 0;    // token 2 i + odd is there when 2 i < some
    const uint32_t step = 4u * static_cast<uint32_t>(p.N);  // bytes of two rows
    const size_t at = 2 * ((row + odd) * p.N + nb);
    const char* in = reinterpret_cast<const char*>(p.residual) + at;
    char* out = reinterpret_cast<char*>(p.Y) + at;
    if constexpr (OUT == kPairResidual) {
      uint32_t r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        r[i] = 2 * i < some ? *reinterpret_cast<const uint32_t*>(in + static_cast<uint64_t>(i) * step) : 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // the exchange below, backwards
        const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, r[i], 1);
        r[i] = __byte_perm(r[i], o, sel);
        v[2 * i] = __fadd_rn(v[2 * i], __uint_as_float(r[i] << 16));
        v[2 * i + 1] = __fadd_rn(v[2 * i + 1], __uint_as_float(r[i] & 0xFFFF0000u));
      }
    }
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = f2_to_bf16x2(f2_pack(v[2 * i], v[2 * i + 1]));  // tokens 2 i, 2 i + 1 of column n
      w[i] = __byte_perm(w[i], __shfl_xor_sync(0xFFFFFFFFu, w[i], 1), sel);
    }
    if (some >= 15) {
#pragma unroll
      for (int i = 0; i < 8; ++i) *reinterpret_cast<uint32_t*>(out + static_cast<uint64_t>(i) * step) = w[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (2 * i < some) *reinterpret_cast<uint32_t*>(out + static_cast<uint64_t>(i) * step) = w[i];
    }
  } else {
    if (p.epilogue == SIXBIT_EPI_GELU) gelu16(v);
    if (n >= p.N) return;
    size_t at = row * p.N + n;
#pragma unroll
    for (int i = 0; i < 16; ++i, at += p.N) {
      if (i >= left) break;
      if (p.epilogue == SIXBIT_EPI_RESIDUAL)
        v[i] = __fadd_rn(v[i], __uint_as_float(static_cast<uint32_t>(p.residual[at]) << 16));
      if (p.Yf != nullptr)
        p.Yf[at] = v[i];
      else
        p.Y[at] = static_cast<uint16_t>(f2_to_bf16x2(f2_pack(v[i], 0.f)) & 0xFFFFu);
    }
  }
}

// A load that stays where it is written (moved down to its use, it cost the
// fold an L2 latency a batch).
__device__ __forceinline__ float load_now(const float* p) {
  float v;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}

// sum += s * accumulator columns
__device__ __forceinline__ void fold16(float s, const uint32_t (&r)[16], float* sum) {
  const uint64_t s2 = f2_pack(s, s);
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const uint64_t v = f2_fma(s2, f2_pack(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), f2_pack(sum[i], sum[i + 1]));
    sum[i] = f2_lo(v);
    sum[i + 1] = f2_hi(v);
  }
}
// The narrow form's: sum += s * (columns + less) for 32 tokens, or, APART, for
// 16 with the high digits' columns before the low ones'.
template <bool APART>
__device__ __forceinline__ void fold32(float s, const uint32_t (&r)[32], const float* less, float* sum) {
  const uint64_t s2 = f2_pack(s, s);
#pragma unroll
  for (int i = 0; i < (APART ? 16 : 32); i += 4) {
    const float4 l = *reinterpret_cast<const float4*>(less + i);
#pragma unroll
    for (int j = i; j < i + 4; j += 2) {
      uint64_t d = f2_pack(__uint_as_float(r[j]), __uint_as_float(r[j + 1]));
      if (APART) d = f2_add(d, f2_pack(__uint_as_float(r[(16 + j) % 32]), __uint_as_float(r[(17 + j) % 32])));
      d = f2_add(d, j == i ? f2_pack(l.x, l.y) : f2_pack(l.z, l.w));
      const uint64_t v = f2_fma(s2, d, f2_pack(sum[j], sum[j + 1]));
      sum[j] = f2_lo(v);
      sum[j + 1] = f2_hi(v);
    }
  }
}

struct Tile {
  int e, row, rows, n0;  // expert, first row of Y, rows of the tile, first weight row
};

template <bool NARROW, Out OUT>
__global__ void __launch_bounds__(Smem<NARROW>::kThreads, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ TokenMaps tmX, const RowsParams p) {
  if (p.mode_dev != nullptr && SIXBIT_MODE_OF(*p.mode_dev) != SIXBIT_MODE_INT8) {
    digits_wait();
    return;
  }
  using C = Cfg<NARROW>;
  using L = Smem<NARROW>;
  constexpr int NT = C::NT, GB = C::GB, SW = C::SW, SX = C::SX, NA = C::NA, NB = C::NB;
  constexpr int kFoldWarp0 = kConvWarp0 + L::kConv, kBox = L::kBox;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarAt);
  uint64_t* w_full = bars;                      // [SW] a batch's nibbles landed
  uint64_t* w_empty = w_full + SW;              // [SW] the converter warps have read them
  uint64_t* x_full = w_empty + SW;              // [SX] a token slot landed
  uint64_t* x_empty = x_full + SX;              // [SX] its MMAs are complete
  uint64_t* a_full = x_empty + SX;              // [NA] the converter warps stored a batch's A
  uint64_t* a_empty = a_full + NA;              // [NA] the batch's MMAs are complete
  uint64_t* acc_full = a_empty + NA;            // [team][NB] an accumulator of the team's tile is complete
  uint64_t* afree = acc_full + C::kTeams * NB;  // [NB] it has been read back by all of the team's warps
  uint64_t* turns = afree + NB;                 // [2] the other issuer has issued its batch
  uint64_t* drain = turns + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* total = tmem_slot + 2;  // tiles of the call
  uint32_t* prefix = reinterpret_cast<uint32_t*>(smem + L::kTables);  // [E + 1] token tiles of the experts before e
  int* first = reinterpret_cast<int*>(prefix) + p.E + 1;              // [E]
  int* count = first + p.E;                                           // [E]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nk = p.K / 128, np = (nk + GB - 1) / GB;  // groups, batches of a tile
  const uint32_t tiles_n = (p.N + kBM - 1) / kBM;

  if (threadIdx.x == 0) {
    for (int s = 0; s < SW; ++s) {
      mbar_init(&w_full[s], 1);
      mbar_init(&w_empty[s], L::kConv);
    }
    for (int s = 0; s < SX; ++s) {
      mbar_init(&x_full[s], 1);
      mbar_init(&x_empty[s], 1);
    }
    for (int a = 0; a < NA; ++a) {
      mbar_init(&a_full[a], L::kConv);
      mbar_init(&a_empty[a], 1);
    }
    for (int b = 0; b < C::kTeams * NB; ++b) mbar_init(&acc_full[b], 1);
    for (int b = 0; b < NB; ++b) mbar_init(&afree[b], C::kTeamWarps);
    for (int i = 0; i < 2; ++i) mbar_init(&turns[i], 1);
    mbar_init(drain, 2);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmW);
    for (int i = 0; i < NT / L::kBox; ++i) prefetch_tmap(&tmX.map[i]);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == 2) {  // row counts and the prefix sums of token tiles, 32 experts at a time
    uint32_t before = 0;  // (no sum passes 32 bits, whatever the offsets: checked on the host)
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int f = 0, c = 0;
      if (e < p.E) {
        expert_rows(p, e, blockIdx.x == 0, &f, &c);
        first[e] = f;
        count[e] = c;
      }
      int t = (c + NT - 1) / NT;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, t, o);
        if (lane >= o) t += u;
      }
      if (e < p.E) prefix[e + 1] = before + t;
      before += __shfl_sync(0xFFFFFFFFu, t, 31);
    }
    if (lane == 0) {
      prefix[0] = 0;
      *total = tile_count(before, tiles_n);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t ntiles = *total;

  auto tile_at = [&](uint32_t id) {
    const uint32_t q = id / tiles_n;
    int lo = 0, hi = p.E;  // prefix[lo] <= q < prefix[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= q)
        lo = mid;
      else
        hi = mid;
    }
    const int r = (q - prefix[lo]) * NT;
    return Tile{lo, first[lo] + r, min(NT, count[lo] - r), static_cast<int>(id - q * tiles_n) * kBM};
  };

  if (warp < kConvWarp0) {
    setmaxnreg_dec<C::kRegsLow>();
    if (warp == 0) {
      // ---------------------------------------------------- nibble producer --
      // Lane 0 copies; the others ask L2 for the batch's scales, which the fold
      // reads some five batches later.
      uint32_t bi = 0;
      bool ok = true;
      for (uint32_t id = blockIdx.x; id < ntiles && ok; id += gridDim.x) {
        const Tile t = tile_at(id);
        const int wrow = t.e * p.N + t.n0;
        const float* sw = p.w4_scale + static_cast<size_t>(t.e) * nk * p.N + min(t.n0 + 32 * (lane & 3), p.N - 1);
        for (int j = 0; j < np; ++j, ++bi) {
          const int s = bi % SW;
          if (bi >= SW && !mbar_wait(&w_empty[s], ((bi / SW) - 1) & 1, abort_flag, p.wait_ns)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            const int boxes = min(GB / 2, (nk - j * GB + 1) / 2);  // (a last, odd group's box is half past the row: zeros)
            mbar_expect_tx(&w_full[s], boxes * kPairBytes);
            for (int h = 0; h < boxes; ++h)
              tma_load_2d(smem + L::kW + s * L::kWSlot + h * kPairBytes, &tmW, &w_full[s], (j * GB + 2 * h) * 64, wrow);
          }
          const int g = j * GB + (lane >> 2);
          if ((lane >> 2) < GB && g < nk) prefetch_l2(sw + static_cast<size_t>(g) * p.N);
        }
      }
      if (lane == 0) {
        if (!ok) {
          set_error(p.err, SIXBIT_ETIMEOUT);
          *abort_flag = 1;
        }
        // every copy this warp started lands before it can exit
        for (uint32_t j = (bi > SW ? bi - SW : 0); j < bi; ++j)
          (void)mbar_wait(&w_full[j % SW], (j / SW) & 1, nullptr, p.wait_ns);
      }
    } else if (warp == 2) {
      if (lane == 0) {
        // --------------------------------------------------- token producer --
        digits_wait();
        uint32_t it = 0;
        bool ok = true;
        for (uint32_t id = blockIdx.x; id < ntiles && ok; id += gridDim.x) {
          const Tile t = tile_at(id);
          const int box = (t.rows - 1) / kBox;
          const CUtensorMap* map = &tmX.map[box];
          for (int j = 0; j < np; ++j, ++it) {
            const int s = it % SX;
            if (it >= SX && !mbar_wait(&x_empty[s], ((it / SX) - 1) & 1, abort_flag, p.wait_ns)) {
              ok = false;
              break;
            }
            if (p.withhold_first && it == 0) continue;  // failure-path test: slot 0 never lands
            // (chunks past K are filled with zeros and counted like the others)
            mbar_expect_tx(&x_full[s], 2 * GB * (box + 1) * kBox * 128);
            tma_load_3d(smem + L::kX + s * L::kXSlot, map, &x_full[s], 0, t.row, 2 * j * GB);
          }
        }
        if (!ok) {
          set_error(p.err, SIXBIT_ETIMEOUT);
          *abort_flag = 1;
        }
        for (uint32_t j = (it > SX ? it - SX : 0); j < it; ++j)
          (void)mbar_wait(&x_full[j % SX], (j / SX) & 1, nullptr, p.wait_ns);
      }
    } else {
      // --------------------------------------------------------- MMA issuers --
      // Warp 1 issues the even batches, warp 3 the odd ones (the whole warp
      // keeps the loop, so that the operands stay in uniform registers; one
      // elected lane issues: with the loop in one lane, an MMA took some 100
      // cycles of issue).  They take strict turns, so that no MMA comes between
      // two that share the collector buffer, and a wait that an issuer meets
      // at every second phase only cannot mistake an older phase for its own:
      // the batch three before was issued before this warp's last turn.  All
      // waits (some 130 cycles each when the phase is there) come before the
      // turn and the commits after it, beside the other issuer's MMAs.
      const uint32_t par = warp == 1 ? 0u : 1u;
      uint32_t bi = 0, turn = 0;  // batches, tiles so far
      bool ok = true;
      for (uint32_t id = blockIdx.x; id < ntiles && ok; id += gridDim.x, ++turn) {
        const Tile t = tile_at(id);
        uint64_t* done = acc_full + (turn & 1) * NB;
        const bool few = NARROW && t.rows <= 16;
        const uint32_t nt = few ? 32 : static_cast<uint32_t>((t.rows + 15) & ~15);
        const uint32_t chunk = ((t.rows - 1) / kBox + 1) * kBox * 128;  // bytes of the tile's digits of a group
        const uint32_t idesc = (1u << 4) | ((nt >> 3) << 17) | (static_cast<uint32_t>(kBM >> 4) << 24);
        for (int j = 0; j < np; ++j, ++bi) {
          if ((bi & 1) != par) continue;
          const int groups = min(GB, nk - j * GB);
          ok = mbar_wait(&x_full[bi % SX], (bi / SX) & 1, abort_flag, p.wait_ns);
          if (ok && bi >= NB) ok = mbar_wait(&afree[bi % NB], ((bi / NB) - 1) & 1, abort_flag, p.wait_ns);
          if (ok) ok = mbar_wait(&a_full[bi % NA], (bi / NA) & 1, abort_flag, p.wait_ns);
          if (ok && bi > 0) ok = mbar_wait(&turns[par], ((bi - 1) >> 1) & 1, abort_flag, p.wait_ns);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d_tmem = tmem + (bi % NB) * L::kAccCols, a_tmem = tmem + L::kACol0 + (bi % NA) * L::kACols;
          const uint32_t b_base = smem_u32(smem + L::kX) + (bi % SX) * L::kXSlot;
          if (elect_one()) {
            auto issue = [&](uint32_t step, bool apart) {  // (the narrow form's are constants)
#pragma unroll
              for (int g = 0; g < GB; ++g) {
                if (g < groups) {
#pragma unroll
                  for (int k = 0; k < 4; ++k) {  // 32 k: the high digits, then the low ones
                    const uint32_t b = b_base + 2 * g * step + 32 * k, a = a_tmem + g * 32 + 8 * k;
                    mma_e4m3_fill(d_tmem + g * NT, a, sdesc_sw128(b), idesc, k == 0 ? 0u : 1u);
                    if (apart) mma_e4m3_lastuse(d_tmem + g * NT, a, sdesc_sw128(b + step), idesc);
                  }
                }
              }
            };
            if (!NARROW)
              issue(chunk, true);
            else if (few)
              issue(L::kBox * 128, false);
            else
              issue(2 * L::kBox * 128, true);
            tc_fence_before();
            mbar_arrive(&turns[par ^ 1]);
            tc_commit(&done[bi % NB]);
            tc_commit(&a_empty[bi % NA]);
            tc_commit(&x_empty[bi % SX]);
          }
          __syncwarp();
        }
      }
      if (!ok && lane == 0) {
        set_error(p.err, SIXBIT_ETIMEOUT);
        *abort_flag = 1;
      }
      __syncwarp();
      if (elect_one()) {
        tc_commit(drain);  // both issuers: all tensor-core work completes before exit
        (void)mbar_wait(drain, 0, nullptr, p.wait_ns);
      }
      __syncwarp();
    }
  } else if (warp < kFoldWarp0) {
    setmaxnreg_dec<C::kRegsConv>();
    // ------------------------------------------------------------ converters --
    // Thread `lane` of the warp of quarter q converts weight row 32 q + lane,
    // the row of its tensor-memory lane; each set of four warps takes two
    // groups of every batch (one group at a time, the barriers and fences took
    // the converters 1,100 cycles a group, more than its MMAs).  A nibble slot
    // goes back once every lane's reads have returned (`zero` needs them) and
    // behind a proxy fence: the refill is an async-proxy write.
    const int q = warp & 3, myrow = 32 * q + lane, pair = (warp - kConvWarp0) >> 2;
    const int swz = myrow & 7;
    const uint32_t total = blockIdx.x < ntiles ? ((ntiles - blockIdx.x - 1) / gridDim.x + 1) * np : 0;
    const uint32_t acol = tmem + (static_cast<uint32_t>(32 * q) << 16) + L::kACol0;
    const uint8_t* row = smem + L::kW + pair * kPairBytes + myrow * 128;
    bool ok = true;
    for (uint32_t bi = 0; bi < total; ++bi) {
      const int s = bi % SW, a = bi % NA;
      if (!mbar_wait(&w_full[s], (bi / SW) & 1, abort_flag, p.wait_ns)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 in[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          in[c] = *reinterpret_cast<const uint4*>(row + s * L::kWSlot + (((4 * h + c) ^ swz) << 4));
        if (h == 1) {
          uint32_t zero;
          asm volatile("and.b32 %0, %1, 0;" : "=r"(zero) : "r"(in[0].x ^ in[1].x ^ in[2].x ^ in[3].x));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&w_empty[s]);
        }
        uint32_t v[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4& u = in[c];
          nibbles<NARROW>(u.x, v[8 * c], v[8 * c + 1]);
          nibbles<NARROW>(u.y, v[8 * c + 2], v[8 * c + 3]);
          nibbles<NARROW>(u.z, v[8 * c + 4], v[8 * c + 5]);
          nibbles<NARROW>(u.w, v[8 * c + 6], v[8 * c + 7]);
        }
        if (h == 0) {
          if (bi >= NA && !mbar_wait(&a_empty[a], ((bi / NA) - 1) & 1, abort_flag, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
        }
        tmem_st32(acol + a * L::kACols + pair * 64 + 32 * h, v);
      }
      if (!ok) break;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&a_full[a]);
    }
    if (!ok && lane == 0) {
      set_error(p.err, SIXBIT_ETIMEOUT);
      *abort_flag = 1;
    }
  } else {
    setmaxnreg_inc<C::kRegsFold>();
    // -------------------------------------------------------- fold + epilogue --
    // A team takes a whole tile, every second one of the CTA's; a thread one
    // weight row and kCols tokens of it.
    static_assert(C::kTeams == 2, "teams take turns");
    constexpr int kCols = L::kCols, kChunks = kCols / 16;
    const int ew = warp - kFoldWarp0, q = warp & 3;
    const uint32_t team = static_cast<uint32_t>(ew / C::kTeamWarps);
    const int cs = (ew % C::kTeamWarps) / 4 * kCols;  // first token of this thread
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * q) << 16) + cs;
    float* my_rs = reinterpret_cast<float*>(smem + L::kFoldArea + ew * L::kWarpArea);
    uint64_t* full = acc_full + team * NB;
    if (NARROW) digits_wait();
    uint32_t phases = 0;  // bit b: parity of this team's next wait for buffer b
    uint32_t bi = 0, turn = 0;
    bool ok = true;
    for (uint32_t id = blockIdx.x; id < ntiles && ok; id += gridDim.x, ++turn) {
      if ((turn & 1) != team) {
        bi += np;
        continue;
      }
      const Tile t = tile_at(id);
      const int n = t.n0 + 32 * q + lane;  // output column
      const float* sw = p.w4_scale + static_cast<size_t>(t.e) * nk * p.N + min(n, p.N - 1);
      float next[GB];  // the next batch's scales, asked for a batch ahead
      auto fetch_sw = [&](int left) {
#pragma unroll
        for (int g = 0; g < GB; ++g, sw += p.N)
          if (g < left) next[g] = load_now(sw);
      };
      fetch_sw(nk);
      // The narrow form's weights stand 8 too high: -8 of the sums of the codes
      // goes onto every accumulator column.  A lane fetches its token's.
      float* my_less = my_rs + kCols;
      const float* less = NARROW ? p.less + t.row + min(lane, t.rows - 1) : nullptr;
      float next_less[GB];
      auto fetch_less = [&](int left) {
#pragma unroll
        for (int g = 0; g < GB; ++g, less += p.M)
          if (g < left)  // (not .nc: the digits' kernel may write while this one runs)
            asm volatile("ld.global.f32 %0, [%1];" : "=f"(next_less[g]) : "l"(less));
      };
      if (NARROW) fetch_less(nk);
      __syncwarp();  // every lane is done with the last tile's row scales
      const int mine = min(t.rows - cs, kCols);  // tokens of this thread (none: <= 0)
#pragma unroll
      for (int j = lane; j < kCols; j += 32) my_rs[j] = j < mine ? __ldg(p.row_scale + t.row + cs + j) : 0.f;
      float sum[kCols];
#pragma unroll
      for (int j = 0; j < kCols; ++j) sum[j] = 0.f;
      for (int j = 0; j < np; ++j, ++bi) {
        const int left = nk - j * GB;
        const uint32_t b = bi % NB;
        if (!mbar_wait(&full[b], (phases >> b) & 1, abort_flag, p.wait_ns)) {
          ok = false;
          break;
        }
        phases ^= 1u << b;
        tc_fence_after();
        if (mine <= 0) {
          release_acc(&afree[b], lane);
          continue;
        }
        const uint32_t acc = lane_addr + b * L::kAccCols;
        float s[GB];
        // The batch's scales and the loads of the next one's, while the first
        // accumulator columns are on their way.
        auto scales = [&] {
#pragma unroll
          for (int g = 0; g < GB; ++g) s[g] = next[g] * 262144.f;  // (2^18: both operands stand in units of 2^-9)
          if (NARROW) {
#pragma unroll
            for (int g = 0; g < GB; ++g) my_less[g * NT + lane] = next_less[g];
            __syncwarp();
            fetch_less(left - GB);
          }
          fetch_sw(left - GB);
        };
        if constexpr (!NARROW) {
#pragma unroll
          for (int g = 0; g < GB; ++g) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              uint32_t r[16];
              tmem_ld16(acc + g * NT + 16 * c, r);
              if (g == 0 && c == 0) scales();
              tmem_ld_wait(r);
              if (g + 1 == GB && c + 1 == kChunks) release_acc(&afree[b], lane);
              if (g < left) fold16(s[g], r, sum + 16 * c);
            }
          }
        } else {
          // Two groups' loads are in flight together (one at a time, the
          // round trips made the fold the slowest role).
#pragma unroll
          for (int g = 0; g < GB; g += 2) {
            uint32_t r0[32], r1[32];
            tmem_ld32(acc + g * NT, r0);
            tmem_ld32(acc + (g + 1) * NT, r1);
            if (g == 0) scales();
            tmem_ld_wait(r0);
            tmem_ld_wait(r1);
            if (g + 2 >= GB) release_acc(&afree[b], lane);
            if (mine > 16) {
              if (g < left) fold32<false>(s[g], r0, my_less + g * NT, sum);
              if (g + 1 < left) fold32<false>(s[g + 1], r1, my_less + (g + 1) * NT, sum);
            } else {
              if (g < left) fold32<true>(s[g], r0, my_less + g * NT, sum);
              if (g + 1 < left) fold32<true>(s[g + 1], r1, my_less + (g + 1) * NT, sum);
            }
          }
          __syncwarp();  // every lane is done with this batch's sums of codes
        }
      }
      __syncwarp();
      if (!ok) break;
      // One copy of the epilogue's code, 32 tokens a turn, the sums moved down
      // in between.
#pragma unroll 1
      for (int c = 0; c < kCols; c += 32) {
        if (c >= mine) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (mine <= c + 16 * h) break;
          float v[16];
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 rv = *reinterpret_cast<const float4*>(my_rs + c + 16 * h + j);
            v[j] = __fmul_rn(sum[16 * h + j], rv.x);
            v[j + 1] = __fmul_rn(sum[16 * h + j + 1], rv.y);
            v[j + 2] = __fmul_rn(sum[16 * h + j + 2], rv.z);
            v[j + 3] = __fmul_rn(sum[16 * h + j + 3], rv.w);
          }
          store16<OUT>(p, static_cast<size_t>(t.row + cs + c + 16 * h), n, mine - c - 16 * h, lane, v);
        }
#pragma unroll
        for (int j = 0; j + 32 < kCols; ++j) sum[j] = sum[j + 32];
      }
    }
    if (!ok && lane == 0) {
      set_error(p.err, SIXBIT_ETIMEOUT);
      *abort_flag = 1;
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// s8 [M, K] -> the token operand, 2 K bytes a row: per group of 128 the high
// digits h of q = 16 h + l as E4M3 of h 2^-5, then the low ones (0 .. 15) as
// E4M3 of l 2^-9, each eight in the order 0 2 4 6 1 3 5 7.
__device__ __forceinline__ uint32_t high_digits(uint32_t q) {
  const uint32_t n = (q >> 7) & 0x01010101u;                         // negative
  const uint32_t mag = (((q >> 4) & 0x0F0F0F0Fu) ^ (n * 15u)) + n;   // |h|, 0 .. 8
  const uint32_t t = mag | (mag >> 4);
  const uint32_t code = __byte_perm(0x1C181000u, 0x26242220u, __byte_perm(t, 0u, 0x4420));  // |h| = 0 .. 7 (8 -> 0)
  return code + ((mag >> 3) & 0x01010101u) * 0x28u + n * 0x80u;
}
// less, if not NULL: [K/128][M], -8 of the sum of a group's codes in units of 2^-18.
__global__ void __launch_bounds__(256) digits_kernel(const int8_t* __restrict__ codes, int64_t n16, int M, int groups,
                                                     uint8_t* __restrict__ out, float* __restrict__ less,
                                                     const int32_t* mode_dev) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (mode_dev != nullptr && SIXBIT_MODE_OF(*mode_dev) != SIXBIT_MODE_INT8) return;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n16;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const uint4 c = __ldg(reinterpret_cast<const uint4*>(codes) + i);
    const uint4 s = make_uint4(__byte_perm(c.x, c.y, 0x6420), __byte_perm(c.x, c.y, 0x7531),
                               __byte_perm(c.z, c.w, 0x6420), __byte_perm(c.z, c.w, 0x7531));
    uint4* o = reinterpret_cast<uint4*>(out) + (i >> 3) * 16 + (i & 7);  // (128 codes are 8 reads; K % 128 == 0)
    o[0] = make_uint4(high_digits(s.x), high_digits(s.y), high_digits(s.z), high_digits(s.w));
    o[8] = make_uint4(s.x & 0x0F0F0F0Fu, s.y & 0x0F0F0F0Fu, s.z & 0x0F0F0F0Fu, s.w & 0x0F0F0F0Fu);
    if (less != nullptr) {  // eight neighbouring lanes hold a group, all of them or none
      const uint32_t eight = 0xFFu << (threadIdx.x & 24);
      int q = __dp4a(static_cast<int>(c.x), 0x01010101, __dp4a(static_cast<int>(c.y), 0x01010101, 0));
      q = __dp4a(static_cast<int>(c.z), 0x01010101, __dp4a(static_cast<int>(c.w), 0x01010101, q));
#pragma unroll
      for (int m = 1; m < 8; m <<= 1) q += __shfl_xor_sync(eight, q, m);
      if ((i & 7) == 0) {
        const int64_t row = (i >> 3) / groups, g = (i >> 3) % groups;
        less[g * M + row] = static_cast<float>(q) * (-8.f / 262144.f);
      }
    }
  }
}

template <bool NARROW, Out OUT>
cudaError_t launch(const CUtensorMap& w, const TokenMaps& x, const RowsParams& p,
                   cudaStream_t st) {
  cudaError_t e = set_smem_once<grouped_kernel<NARROW, OUT>>(static_cast<int>(Smem<NARROW>::bytes(SIXBIT_MAX_EXPERTS)));
  if (e != cudaSuccess) return e;
  static ContextCache<int> regs_cache;
  int regs = 0;
  e = regs_cache.get(&regs, [](int* o) {
    cudaFuncAttributes fa;
    const cudaError_t r = cudaFuncGetAttributes(&fa, grouped_kernel<NARROW, OUT>);
    *o = fa.numRegs;
    return r;
  });
  if (e != cudaSuccess) return e;
  // setmaxnreg.inc waits until the block's own registers cover the increase:
  // launch only with the register count the split was sized for.
  if (regs != Cfg<NARROW>::kRegs) return cudaErrorInvalidConfiguration;
  // at most one token tile per row, and one more per expert than rows / NT
  const int64_t tiles_n = (p.N + kBM - 1) / kBM;
  const int64_t tiles_t = std::min<int64_t>(p.M, p.M / Cfg<NARROW>::NT + static_cast<int64_t>(p.E));
  // (neither is reached by arrays that fit the GPU's memory)
  if (tiles_t * tiles_n > INT32_MAX || most_token_tiles(p.M, Cfg<NARROW>::NT, p.E) > UINT32_MAX)
    return cudaErrorInvalidValue;
  const int grid = static_cast<int>(std::min<int64_t>(tiles_t * tiles_n, sm_count()));
  // The CTAs' set-up and first weights beside the digits' kernel: 16 rows over 8
  // experts 17.2 -> 16.5 us, 32 over 64 40.4 -> 38.8, 1024 over 8 49.1 -> 47.4,
  // 35552 over 8 928 -> 922; but in the narrow form 1024 rows over 32 78 -> 82
  // and 2560 over 64 173 -> 185 (768 over 64 96.7 -> 95.5).  (The limit lies
  // between these sizes; why the narrow form loses above it is not known.)
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(Smem<NARROW>::kThreads);
  cfg.dynamicSmemBytes = Smem<NARROW>::bytes(p.E);
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = NARROW && p.M > 768 ? 0 : 1;
  note_launch();
  return cudaLaunchKernelEx(&cfg, grouped_kernel<NARROW, OUT>, w, x, p);
}

template <bool NARROW>
cudaError_t launch_form(const CUtensorMap& w, const TokenMaps& x, const RowsParams& p,
                        cudaStream_t st) {
  const bool pairs = p.Yf == nullptr && (p.N & 1) == 0 && p.N < (1 << 30) &&
                     ((reinterpret_cast<uintptr_t>(p.Y) | reinterpret_cast<uintptr_t>(p.residual)) & 3) == 0;
  if (!pairs) return launch<NARROW, kAny>(w, x, p, st);
  if (p.epilogue == SIXBIT_EPI_GELU) return launch<NARROW, kPairGelu>(w, x, p, st);
  if (p.epilogue == SIXBIT_EPI_RESIDUAL) return launch<NARROW, kPairResidual>(w, x, p, st);
  return launch<NARROW, kPair>(w, x, p, st);
}

}  // namespace grouped

cudaError_t launch_digits(const int8_t* codes, int M, int K, const int32_t* mode_dev, uint8_t* out, float* less,
                          cudaStream_t st) {
  const int64_t n16 = static_cast<int64_t>(M) * K / 16;
  const int64_t want = (n16 + 255) / 256, cap = static_cast<int64_t>(sm_count()) * 8;
  grouped::digits_kernel<<<static_cast<int>(want < cap ? want : cap), 256, 0, st>>>(codes, n16, M, K / 128, out, less,
                                                                                   mode_dev);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_w4a8_grouped(const CUtensorMap& w, const TokenMaps& x, const RowsParams& p, bool narrow,
                                cudaStream_t st) {
  return narrow ? grouped::launch_form<true>(w, x, p, st) : grouped::launch_form<false>(w, x, p, st);
}

}  // namespace sixbit
