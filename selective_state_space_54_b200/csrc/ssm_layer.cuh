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

// Gated recurrence: steps between two saved states, the state entering every
// kGsCkpt-step chunk laid out [batch][chunk][dim] fp32.
constexpr int kGsCkpt = 64;
__host__ __device__ __forceinline__ int64_t gs_chunks(int64_t L) { return (L + kGsCkpt - 1) / kGsCkpt; }

struct GsParams {
  const void *u, *f, *z;             // [batch][dim][L] (or [batch][L][dim]) io dtype; z nullable
  const float *bias;                 // [dim], nullable
  const uint8_t *starts;             // [batch][L], nullable
  const float *h0;                   // [batch][dim], nullable
  void *y;                           // as u; null: only the saved states are wanted
  float *last;                       // [batch][dim], nullable
  float *ckpt;                       // [batch][gs_chunks(L)][dim], nullable (forward writes, backward reads)
  int64_t batch, dim, L;
  int tok, untied;
  // backward
  const void *dout;
  const float *dlast;                // [batch][dim], nullable
  void *du, *df, *dz;
  float *dbias_part;                 // [batch][dim], nullable
  float *dbias;                      // [dim], nullable
  float *dh0;                        // [batch][dim], nullable
};
cudaError_t launch_gscan_fwd(int io_dtype, const GsParams &p, cudaStream_t s);
cudaError_t launch_gscan_bwd(int io_dtype, const GsParams &p, cudaStream_t s);

struct GsStepParams {
  const void *u, *f, *z;             // [batch][dim]; z nullable
  const float *bias;                 // [dim], nullable
  float *state;                      // [batch][dim], updated in place
  void *y;
  int64_t batch, dim;
  int untied;
};
cudaError_t launch_gscan_step(int io_dtype, const GsStepParams &p, cudaStream_t s);

struct NormParams {
  const void *x, *res;               // [rows][dim] io dtype, residual dtype (nullable)
  const float *w, *b;                // [dim]; b nullable
  void *y, *res_out;                 // io dtype, residual dtype (with res)
  int64_t rows, dim;
  float eps;
};
cudaError_t launch_norm(int io_dtype, int res_dtype, const NormParams &p, cudaStream_t s);

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
