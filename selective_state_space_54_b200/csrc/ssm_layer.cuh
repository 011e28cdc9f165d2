// Internal definitions of the layer operators beside the selective scan: the
// gated linear recurrence (ssm_gscan.cu) and layer norm (ssm_norm.cu).  Not
// part of the public interface.
#pragma once

#include "ssm_common.cuh"
#include "ssm_scan.h"

namespace ssm {

// Shared by every entry point (ssm_api.cu).
cudaError_t injected_failure();
ssm_status cuda_status(cudaError_t e);

// Gated recurrence, channel-major: a lane takes 32 bytes of each tensor (16
// bf16 or 8 fp32 steps), a warp 32 lanes of it; the state entering every warp's
// run is what the backward starts from.  Saved [batch][dim][gs_row_chunks] fp32
// (the first of a row is the initial state and is not read).
constexpr int kGsLaneBytes = 32;
__host__ __device__ __forceinline__ int gs_row_steps(int esize) { return 32 * kGsLaneBytes / esize; }
// Rows that are not whole 16-byte pieces are cut where memory is aligned to 32 bytes (as far
// as the tensors are): a row's first chunk begins `row * L mod the lane's steps` steps early.
__host__ __device__ __forceinline__ int gs_row_cut(int64_t L, int esize) {  // mask of that remainder
  return L % (16 / esize) ? kGsLaneBytes / esize - 1 : 0;
}
__host__ __device__ __forceinline__ int64_t gs_row_span(int64_t L, int esize) {  // steps the widest row takes
  const int cut = gs_row_cut(L, esize);
  return cut ? L + cut + 1 - (L & -L) : L;
}
__host__ __device__ __forceinline__ int64_t gs_row_chunks(int64_t L, int esize) {
  return (gs_row_span(L, esize) + gs_row_steps(esize) - 1) / gs_row_steps(esize);
}
constexpr int kGsTileWarps = 8;    // warps, and warp runs of steps, per look-back tile
constexpr int kGsRowGroup = 31;    // tiles between two published states of a row, at most
// Token-major: a tile is 64 channels by gs_tok_steps steps (8 KB of each tensor), a warp's
// run a quarter of it.  Saved [batch][tile][dim] fp32, the state entering every tile.
constexpr int kTokChannels = 64;
constexpr int kTokWarps = 4;
constexpr int kTokGroup = 32;      // tiles between two published states of a channel, at most
__host__ __device__ constexpr int gs_tok_steps(int esize) { return 128 / esize; }
__host__ __device__ __forceinline__ int64_t gs_tok_tiles(int64_t L, int esize) {
  return (L + gs_tok_steps(esize) - 1) / gs_tok_steps(esize);
}
__host__ __device__ __forceinline__ int64_t gs_tok_groups(int64_t dim) { return (dim + kTokChannels - 1) / kTokChannels; }

struct GsParams {
  const void *u, *f, *z;             // [batch][dim][L] (or [batch][L][dim]) io dtype; z nullable
  const float *bias;                 // [dim], nullable
  const uint8_t *starts;             // [batch][L], nullable
  const float *h0;                   // [batch][dim], nullable
  void *y;                           // as u; null: only the saved states are wanted
  float *last;                       // [batch][dim], nullable
  float *ckpt;                       // saved states, nullable (forward writes, backward reads)
  int64_t batch, dim, L;
  int tok, untied;
  int vec;                           // accesses rows allow: 2 = 16 bytes, 1 = 4, 0 = one element
  int cut;                           // channel-major: gs_row_cut
  int v32;                           // channel-major: 32-byte stores; token-major: two channels at once
  int start_vec;                     // starts rows 4-byte aligned
  // look-back schedule (zeroed): error word, ticket counter, tile runs, group states
  unsigned *err, *ticket;
  unsigned long long *runs;
  unsigned *states;
  int64_t tiles;                     // time tiles per row or channel group
  unsigned group, groups;            // tiles between two published states, and how many such groups
  int sms;
  // backward
  const void *dout;
  const float *dlast;                // [batch][dim], nullable
  void *du, *df, *dz;
  float *dbias_part;                 // [part_rows][dim], nullable
  int64_t part_rows;
  float *dbias;                      // [dim], nullable
  float *dh0;                        // [batch][dim], nullable
};
// path: SSM_PATH_PER_GROUP or SSM_PATH_LOOKBACK
cudaError_t launch_gscan_fwd(int io_dtype, int path, const GsParams &p, cudaStream_t s);
cudaError_t launch_gscan_bwd(int io_dtype, int path, const GsParams &p, cudaStream_t s);
cudaError_t launch_gs_rows_fwd(int io_dtype, int path, const GsParams &p, cudaStream_t s);
cudaError_t launch_gs_rows_bwd(int io_dtype, int path, const GsParams &p, cudaStream_t s);
cudaError_t launch_gs_tok_fwd(int io_dtype, const GsParams &p, cudaStream_t s);
cudaError_t launch_gs_tok_bwd(int io_dtype, const GsParams &p, cudaStream_t s);

struct GsStepParams {
  const void *u, *f, *z;             // [batch][dim]; z nullable
  const float *bias;                 // [dim], nullable
  float *state;                      // [batch][dim], updated in place
  void *y;
  int64_t batch, dim;
  int untied;
};
cudaError_t launch_gscan_step(int io_dtype, const GsStepParams &p, cudaStream_t s);
// test hook: the tiles' bounded wait on 8 words that stay 0
cudaError_t launch_gs_wait_probe(const unsigned long long *words, unsigned *err, unsigned long long limit_ns,
                                 cudaStream_t s);

struct NormParams {
  const void *x, *res;               // [rows][dim] io dtype, residual dtype (nullable)
  const float *w, *b;                // [dim]; b nullable
  void *y, *res_out;                 // io dtype, residual dtype (with res)
  int64_t rows, dim;
  float eps;
};
cudaError_t launch_norm(int io_dtype, int res_dtype, const NormParams &p, int sms, cudaStream_t s);

struct NormBwdParams {
  const void *s, *dy, *dres_out;     // residual dtype, io dtype, residual dtype (nullable)
  const float *w;
  void *dx, *dres;                   // io dtype, residual dtype (null where it is the io dtype)
  float *dw, *db;                    // [dim]; db nullable
  float *part;                       // partial sums of dw, then of db
  int64_t rows, dim;
  float eps;
};
size_t norm_bwd_part_floats(int64_t rows, int64_t dim, int sms);
cudaError_t launch_norm_bwd(int io_dtype, int res_dtype, const NormBwdParams &p, int sms, cudaStream_t s);

}  // namespace ssm
