// Internal interface between the C-ABI layer and the kernel translation units.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "sixbit.h"

namespace sixbit {

// SIXBIT_OK when the current device is a compute capability 10.3 GPU (checked
// once per context), else SIXBIT_EUNSUPPORTED.
sixbit_status check_device();
// Device address of the allocation-free entry point's scratch array in the
// current context (resolved once per context).
sixbit_status noalloc_scratch(void** out);

struct GemmParams {
  int M, N, K;
  const int32_t* mode_dev;
  int want_mode;
  int epilogue;
  const uint8_t* sfa;      // NVFP4 tiled scales of A
  const uint8_t* sfb;      // NVFP4 tiled scales of B
  const float* s_a;        // NVFP4 tensor scale of A
  const float* s_b;        // NVFP4 tensor scale of B
  const float* row_scale;  // INT8: s_m [M]
  const float* grp_scale;  // INT8: s_w [K/128][N]
  const uint16_t* residual;
  uint16_t* Y;
  float* Yf;
  int32_t* acc_dbg;
  int32_t* err;
  int n_fastest;           // tile order: 1 = output column tiles fastest, 0 = row tiles fastest
  float* rot_amax;         // NVFP4 epilogue: atomicMax of |bf16(Y) . blockdiag(H_b / sqrt b)| (or NULL)
  int had_block;           // b of rot_amax (16 or 64)
  int y_tma;               // bf16-operand kinds: bf16 Y is written by TMA stores through the Y tensor map
  uint64_t wait_ns;        // limit of every bounded wait (kWaitLimitNs unless a test shortens it)
  int withhold_first;      // test of the failure path: each CTA's producer skips its first stage
  uint16_t* bs_delta;      // residual epilogue: the block's Delta cache (Delta_prev in, Delta out), or NULL
  void* bs_parts;          // ... and its statistics, one partial row per epilogue warp (see gemm_common.cuh)
};

// Partial rows of a GEMM epilogue's block statistics: a uint32 row count at
// byte 0, then one row per CTA of kBsSums float-float values {hi, lo} from
// byte 16, in the order sum Delta^2, sum x_in^2, sum Delta Delta_prev,
// sum Delta_prev^2, max |x_out| (lo = 0), sum |x_out|.  At most sm_count
// rows; a CTA has at most kBsMaxWarps epilogue warps.
constexpr int kBsSums = 6;
constexpr int kBsMaxWarps = 16;
size_t bs_parts_bytes();
cudaError_t launch_block_stats_parts(const void* parts, int64_t n, sixbit_stats* stats, cudaStream_t st);
cudaError_t launch_dit_block_end_parts(const sixbit_policy_cfg& cfg, const sixbit_dit_blocks& B, int l,
                                       const void* parts, cudaStream_t st);

// Test setting of the GEMMs' failure path (sixbit_debug_gemm_timeout).
void gemm_debug_params(GemmParams& p);

cudaError_t launch_hq_amax(const uint16_t* X, int M, int K, int b, const int32_t* mode_dev, float* amax_out,
                           cudaStream_t st);
cudaError_t launch_hq_nvfp4(const uint16_t* X, int M, int K, int b, const int32_t* mode_dev, const float* amax_src,
                            const sixbit_qact* o, cudaStream_t st);
cudaError_t launch_hq_int8(const uint16_t* X, int M, int K, int b, const int32_t* mode_dev, const sixbit_qact* o,
                           cudaStream_t st);
cudaError_t launch_pack_weights(const float* W, int N, int K, int b, const sixbit_weights* o, cudaStream_t st);

size_t stats_scratch_bytes(int64_t n);
cudaError_t launch_tensor_stats(const uint16_t* x, int64_t n, double* out, void* scratch, cudaStream_t st);
cudaError_t launch_block_stats(const uint16_t* x_in, const uint16_t* x_out, uint16_t* delta, int64_t n,
                               const int32_t* mode_dev, sixbit_stats* stats, void* scratch, cudaStream_t st);
// Elements one CTA of the fixed-grid statistics launch covers.
constexpr int64_t kFixedElemsPerCta = 65536;
cudaError_t launch_block_stats_fixed_grid(const uint16_t* x_in, const uint16_t* x_out, uint16_t* delta, int64_t n,
                                          const int32_t* mode_dev, sixbit_stats* stats, void* scratch,
                                          cudaStream_t st);
cudaError_t launch_skip_apply(const uint16_t* x_in, const uint16_t* delta, uint16_t* x_out, int64_t n,
                              const int32_t* mode_dev, sixbit_stats* stats, void* scratch, cudaStream_t st);
cudaError_t launch_block_stats_mx(const uint16_t* x_in, const uint16_t* x_out, uint8_t* codes, uint8_t* scales,
                                  int64_t n, const int32_t* mode_dev, sixbit_stats* stats, void* scratch,
                                  cudaStream_t st);
cudaError_t launch_skip_apply_mx(const uint16_t* x_in, const uint8_t* codes, const uint8_t* scales, uint16_t* x_out,
                                 int64_t n, const int32_t* mode_dev, sixbit_stats* stats, void* scratch,
                                 cudaStream_t st);
cudaError_t launch_dit_begin(const sixbit_policy_cfg& cfg, const sixbit_dit_blocks& B, void* scratch, int32_t* err,
                             cudaStream_t st);
cudaError_t launch_dit_block_end(const sixbit_policy_cfg& cfg, const sixbit_dit_blocks& B, int l, void* scratch,
                                 int32_t* err, cudaStream_t st);
cudaError_t launch_dit_skip_run(const sixbit_policy_cfg& cfg, const sixbit_dit_blocks& B, int l, void* scratch,
                                int32_t* err, cudaStream_t st);
cudaError_t launch_policy(const sixbit_policy_cfg& cfg, sixbit_policy_state* st_dev, const sixbit_stats* last,
                          const double* in_stats, int32_t* mode_out, cudaStream_t st);

cudaError_t launch_qgemm_nvf4(const CUtensorMap& a, const CUtensorMap& b, const GemmParams& p, cudaStream_t st);
// y: tensor map of the bf16 output (box 32 x 32, 64-byte swizzle), used when p.y_tma.
cudaError_t launch_qgemm_bf16(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& y, const GemmParams& p,
                              cudaStream_t st);
// W4A8: INT4 codes [N, K/2] -> fp16 [N, K] into ws (w4a8_workspace_bytes(N, K)),
// then the GEMM: a_s8 maps the s8 codes [M, K] (box 128 x 128, 128-byte
// swizzle), w_f16 the expanded weights (box 64 x 192, 128-byte swizzle), y the
// bf16 output.
size_t w4a8_workspace_bytes(int N, int K);
cudaError_t launch_w4_expand(const uint8_t* codes, int N, int K, uint16_t* ws, const int32_t* mode_dev,
                             cudaStream_t st);
cudaError_t launch_qgemm_w4a8(const CUtensorMap& a_s8, const CUtensorMap& w_f16, const CUtensorMap& y,
                              const GemmParams& p, cudaStream_t st);


// Residual add, RMS norm, rotation (b = 0: none) and INT8 quantization of [M, K] rows; res, w and sum_out may be NULL.
cudaError_t launch_add_rmsnorm_quant(const uint16_t* x, const uint16_t* res, const float* w, int M, int K, float eps,
                                     int b, const int32_t* mode_dev, uint16_t* sum_out, int8_t* codes,
                                     float* row_scale, cudaStream_t st);

// A W4A8 product on the stored operands: one weight (offsets NULL, E 1) or
// E of them, expert e's rows [offsets[e], offsets[e + 1]) of [M, K].
struct RowsParams {
  const int8_t* codes;     // [M, K]
  const float* row_scale;  // [M]
  const uint8_t* w4;       // [E][N, K/2]
  const float* w4_scale;   // [E][K/128][N]
  const int32_t* offsets;  // [E + 1] on the device, or NULL
  int M, N, K, E;
  const int32_t* mode_dev;
  int epilogue;
  const uint16_t* residual;
  uint16_t* Y;
  float* Yf;
  int32_t* err;
  uint64_t wait_ns;        // as in GemmParams (grouped kernel)
  int withhold_first;
  const float* less;       // narrow grouped kernel: [K/128][M], -8 x a group's sum of codes x 2^-18
};
cudaError_t launch_w4a8_rows(const RowsParams& p, cudaStream_t st);
// Codes [M, K] -> the grouped kernel's token operand, 2 K bytes a row, and, if
// less is not NULL, its RowsParams::less.
cudaError_t launch_digits(const int8_t* codes, int M, int K, const int32_t* mode_dev, uint8_t* out, float* less,
                          cudaStream_t st);
// Maps of the token operand, seen as [K/64 chunks][M rows][128 bytes], 128-byte
// swizzle: map i has boxes of token_chunks() chunks x (i + 1) token_box() rows,
// so that a copy of any tile's batch is one box.
constexpr int token_box(bool narrow) { return narrow ? 16 : 32; }
constexpr int token_chunks(bool narrow) { return narrow ? 8 : 4; }
constexpr int token_maps(bool narrow) { return narrow ? 2 : 3; }
struct TokenMaps {
  CUtensorMap map[3];
};
// Token tiles that E experts' ranges of M rows can come to: ascending offsets
// claim each row once, others once for each run of ascending ones, of which a
// pair that does not ascend ends each but the last.
constexpr int64_t most_token_tiles(int64_t M, int tile, int E) { return (E + 1) / 2 * (M / tile) + E; }
// Numbers of all tiles are 31 bits: with offsets that claim rows more than once,
// tiles beyond them are left out.
#ifdef __CUDACC__
__host__ __device__
#endif
constexpr uint32_t tile_count(uint32_t tiles_t, uint32_t tiles_n) {
  const uint64_t all = static_cast<uint64_t>(tiles_t) * tiles_n;
  return all < INT32_MAX ? static_cast<uint32_t>(all) : INT32_MAX;
}
// w: map of the INT4 codes [E N, K/2] (box 128 bytes x 128 rows, 128-byte
// swizzle).  narrow: token tiles of 32 instead of 96.
cudaError_t launch_w4a8_grouped(const CUtensorMap& w, const TokenMaps& x, const RowsParams& p, bool narrow,
                                cudaStream_t st);

// The norms around a block's branch (sixbit_gated_rmsnorm_quant): y non-NULL
// takes bf16 rows in place of codes and row_scale.
struct GatedNormParams {
  const uint16_t* x;
  const uint16_t* res;   // or NULL
  const float* w;        // [K], or NULL
  const float* post_w;   // [K], or NULL: no norm of the branch
  const float* gate;     // [S][K], or NULL
  const float* scale;    // [S][K], or NULL
  const float* shift;    // [S][K], or NULL
  const int32_t* segment;  // [M], or NULL: runs of rows_per_seg rows
  float res_scale, eps;
  int M, K, S, rows_per_seg;
  const int32_t* mode_dev;
  uint16_t* sum_out;     // or NULL
  uint16_t* y;
  int8_t* codes;
  float* row_scale;
  int32_t* err;
  uint64_t wait_ns;      // as in GemmParams
  int withhold_first;
};
cudaError_t launch_gated_norm(const GatedNormParams& g, int b, cudaStream_t st);

// Routing (sixbit_moe_route).  counts: workspace, [kRouteRuns][pitch].
constexpr int kRouteTurn = 32;   // tokens of a turn; up to these one CTA does all and needs no workspace
constexpr int kRouteRuns = 304;  // runs of tokens, a CTA each: two for each SM (above 64 experts their registers leave room for one at a time)
struct RouteParams {
  const float* logits;           // [T][E], or
  const uint16_t* logits_bf16;
  const float* bias;             // [E], or NULL
  int T, E, k, score, groups, top_groups, best, renorm;
  float factor;
  int32_t* experts;              // [T][k]
  float* weights;                // [T][k]
  int32_t* rows;                 // [T][k]
  int32_t* token;                // [T k]
  int32_t* offsets;              // [E + 1]
  int32_t* counts;
  // set by the launch: tokens of a run, log2 of the lanes that look through a group, E rounded up to four, and 2^20
  // over a group's size
  int tokens_per_cta, team, pitch;
  uint32_t per;
};
cudaError_t launch_moe_route(RouteParams p, cudaStream_t st);

// The experts' weighted sum (sixbit_moe_combine).
struct CombineParams {
  const void* d;                 // [R][H] bf16, or FP32
  int f32;
  const int32_t* rows;           // [T][k]
  const float* weights;          // [T][k]
  int T, k, H, R;
  uint16_t* Y;
  float* Yf;
  int32_t* err;
  int wide;                      // set by the launch: rows are 32-byte aligned
};
cudaError_t launch_moe_combine(CombineParams p, cudaStream_t st);

// Low-rank adapters (sixbit_lowrank_add).
struct LowRankParams {
  const int8_t* codes;           // [M][K] with row_scale [M], or
  const float* row_scale;
  const uint16_t* x;             // bf16 [M][K]
  const uint16_t* a;             // [L][R][K]
  const uint16_t* b;             // [L][N][R]
  const float* alpha;            // [L], or NULL
  const int32_t* ids;            // [M]
  int M, N, K, R, L;
  const float* base_f32;         // [M][N], or
  const uint16_t* base;          // bf16, or neither
  int epilogue;
  const uint16_t* residual;
  uint16_t* Y;
  float* Yf;
  const int32_t* mode_dev;
  int32_t* err;
  void* v;                       // in the workspace: its first two parts,
  void* v_last;                  // its third, the rows' order and their adapters
  int32_t* perm;
  int32_t* sid;
  int chunk, chunks_per_cta;     // set by the launch
};
size_t lowrank_workspace(int M, int R);
cudaError_t launch_lowrank(LowRankParams p, void* workspace, cudaStream_t st);

}  // namespace sixbit
