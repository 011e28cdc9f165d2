// C ABI of the layer operators beside the selective scan: the gated linear
// recurrence and layer norm.  Argument checks, workspace layout and launches;
// the public contract is include/ssm_scan.h.
#include <string.h>

#include <cmath>

#include "ssm_layer.cuh"

using namespace ssm;

namespace {

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
bool aligned(const void *p, size_t a) { return p == nullptr || ((uintptr_t)p % a) == 0; }
size_t esize(int32_t dtype) { return dtype == SSM_BF16 ? 2 : 4; }

int device_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return sms;
}

ssm_status check_gscan(const ssm_shape *s) {
  if (!s) return SSM_ERR_INVALID_ARG;
  if (s->batch < 0 || s->dim < 0 || s->seqlen < 0 || s->dstate != 1) return SSM_ERR_INVALID_ARG;
  if (s->io_dtype != SSM_F32 && s->io_dtype != SSM_BF16) return SSM_ERR_UNSUPPORTED;
  if (s->path != SSM_PATH_AUTO && s->path != SSM_PATH_PER_GROUP && s->path != SSM_PATH_LOOKBACK)
    return SSM_ERR_UNSUPPORTED;
  if (s->lanes != 0) return SSM_ERR_UNSUPPORTED;
  if (s->flags & ~(SSM_FLAG_SAVE_STATES | SSM_FLAG_TOKEN_MAJOR | SSM_FLAG_UNTIED)) return SSM_ERR_INVALID_ARG;
  if ((s->flags & SSM_FLAG_TOKEN_MAJOR) && s->path == SSM_PATH_PER_GROUP) return SSM_ERR_UNSUPPORTED;
  // index arithmetic is int64 and a grid dimension 31 bits
  if ((double)s->batch * (double)s->dim * (double)s->seqlen > 4.0e15 || (double)s->batch * (double)s->dim > 2.0e9)
    return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

// Workspace of the forward: header, saved states.  Of the backward: header,
// saved states (its own), per-batch partial sums of df_bias.
struct GsLayout {
  size_t off_ckpt, off_part, total;
};
GsLayout gs_layout(const ssm_shape *s, bool bwd) {
  GsLayout l;
  const size_t ckpt = sizeof(float) * (size_t)s->batch * (size_t)gs_chunks(s->seqlen) * (size_t)s->dim;
  l.off_ckpt = kHeaderBytes;
  l.off_part = l.off_ckpt;
  if (bwd || (s->flags & SSM_FLAG_SAVE_STATES)) l.off_part = round_up(l.off_ckpt + ckpt, 256);
  l.total = l.off_part;
  if (bwd) l.total = round_up(l.off_part + sizeof(float) * (size_t)s->batch * (size_t)s->dim, 256);
  if (!bwd && !(s->flags & SSM_FLAG_SAVE_STATES)) l.total = 0;
  return l;
}

void gs_fill(GsParams &p, const ssm_shape *s, const void *u, const void *f, const void *z, const float *bias,
             const uint8_t *starts, const float *h0) {
  memset(&p, 0, sizeof(p));
  p.u = u; p.f = f; p.z = z; p.bias = bias; p.starts = starts; p.h0 = h0;
  p.batch = s->batch; p.dim = s->dim; p.L = s->seqlen;
  p.tok = (s->flags & SSM_FLAG_TOKEN_MAJOR) ? 1 : 0;
  p.untied = (s->flags & SSM_FLAG_UNTIED) ? 1 : 0;
}

}  // namespace

extern "C" {

size_t ssm_gated_scan_fwd_workspace_bytes(const ssm_shape *shape) {
  if (check_gscan(shape) != SSM_OK || shape->batch * shape->dim == 0 || shape->seqlen == 0) return 0;
  return gs_layout(shape, false).total;
}

size_t ssm_gated_scan_bwd_workspace_bytes(const ssm_shape *shape) {
  if (check_gscan(shape) != SSM_OK || shape->batch * shape->dim == 0 || shape->seqlen == 0) return 0;
  return gs_layout(shape, true).total;
}

int32_t ssm_gated_scan_path(const ssm_shape *shape) {
  if (check_gscan(shape) != SSM_OK) return SSM_PATH_AUTO;
  if (shape->path != SSM_PATH_AUTO) return shape->path;
  return (shape->flags & SSM_FLAG_TOKEN_MAJOR) ? SSM_PATH_LOOKBACK : SSM_PATH_PER_GROUP;
}

ssm_status ssm_gated_scan_fwd(const ssm_shape *shape, const void *u, const void *f, const void *z,
                              const float *f_bias, const uint8_t *starts, const float *initial_state,
                              void *y, float *last_state, void *workspace, size_t ws_bytes,
                              ssm_stream_t stream) {
  const ssm_status st = check_gscan(shape);
  if (st != SSM_OK) return st;
  const int64_t nch = shape->batch * shape->dim;
  if (nch == 0) return SSM_OK;
  if (!aligned(f_bias, 4) || !aligned(initial_state, 4) || !aligned(last_state, 4)) return SSM_ERR_INVALID_ARG;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (shape->seqlen == 0) {  // nothing to scan: last_state = initial state
    if (!last_state || last_state == initial_state) return SSM_OK;
    const size_t bytes = sizeof(float) * (size_t)nch;
    return cuda_status(initial_state
                           ? cudaMemcpyAsync(last_state, initial_state, bytes, cudaMemcpyDeviceToDevice, s)
                           : cudaMemsetAsync(last_state, 0, bytes, s));
  }
  const size_t es = esize(shape->io_dtype);
  if (!u || !f || !y || !aligned(u, es) || !aligned(f, es) || !aligned(z, es) || !aligned(y, es))
    return SSM_ERR_INVALID_ARG;
  if (y == u || y == f || y == z) return SSM_ERR_INVALID_ARG;
  const GsLayout l = gs_layout(shape, false);
  if (l.total && (!workspace || ws_bytes < l.total || !aligned(workspace, 256))) return SSM_ERR_WORKSPACE;
  GsParams p;
  gs_fill(p, shape, u, f, z, f_bias, starts, initial_state);
  p.y = y; p.last = last_state;
  if (shape->flags & SSM_FLAG_SAVE_STATES)
    p.ckpt = reinterpret_cast<float *>(static_cast<char *>(workspace) + l.off_ckpt);
  const cudaError_t inj = injected_failure();
  if (inj != cudaSuccess) return cuda_status(inj);
  return cuda_status(launch_gscan_fwd(shape->io_dtype, p, s));
}

ssm_status ssm_gated_scan_bwd(const ssm_shape *shape, const void *u, const void *f, const void *z,
                              const float *f_bias, const uint8_t *starts, const float *initial_state,
                              const void *dout, const float *dlast_state, const void *fwd_workspace,
                              void *du, void *df, void *dz, float *df_bias, float *dinitial_state,
                              void *workspace, size_t ws_bytes, ssm_stream_t stream) {
  const ssm_status st = check_gscan(shape);
  if (st != SSM_OK) return st;
  if (fwd_workspace && (!(shape->flags & SSM_FLAG_SAVE_STATES) || !aligned(fwd_workspace, 256)))
    return SSM_ERR_INVALID_ARG;
  if ((z == nullptr) != (dz == nullptr) || (f_bias == nullptr) != (df_bias == nullptr)) return SSM_ERR_INVALID_ARG;
  if (!aligned(f_bias, 4) || !aligned(initial_state, 4) || !aligned(dlast_state, 4) || !aligned(df_bias, 4) ||
      !aligned(dinitial_state, 4))
    return SSM_ERR_INVALID_ARG;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t nch = shape->batch * shape->dim;
  if (nch == 0 || shape->seqlen == 0) {  // no step: the state's gradient passes through
    cudaError_t e = cudaSuccess;
    if (shape->dim > 0 && df_bias) e = cudaMemsetAsync(df_bias, 0, sizeof(float) * (size_t)shape->dim, s);
    if (e == cudaSuccess && nch > 0 && dinitial_state && dinitial_state != dlast_state)
      e = dlast_state ? cudaMemcpyAsync(dinitial_state, dlast_state, sizeof(float) * (size_t)nch,
                                        cudaMemcpyDeviceToDevice, s)
                      : cudaMemsetAsync(dinitial_state, 0, sizeof(float) * (size_t)nch, s);
    return cuda_status(e);
  }
  const size_t es = esize(shape->io_dtype);
  if (!u || !f || !dout || !du || !df || !aligned(u, es) || !aligned(f, es) || !aligned(z, es) ||
      !aligned(dout, es) || !aligned(du, es) || !aligned(df, es) || !aligned(dz, es))
    return SSM_ERR_INVALID_ARG;
  const void *in[] = {u, f, z, dout}, *out[] = {du, df, dz};
  for (int i = 0; i < 3; ++i) {
    if (!out[i]) continue;
    for (const void *q : in)
      if (out[i] == q) return SSM_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (out[i] == out[j]) return SSM_ERR_INVALID_ARG;
  }
  const GsLayout l = gs_layout(shape, true);
  if (!workspace || ws_bytes < l.total || !aligned(workspace, 256)) return SSM_ERR_WORKSPACE;
  char *ws = static_cast<char *>(workspace);
  GsParams p;
  gs_fill(p, shape, u, f, z, f_bias, starts, initial_state);
  const cudaError_t inj = injected_failure();
  if (inj != cudaSuccess) return cuda_status(inj);
  if (fwd_workspace) {
    p.ckpt = reinterpret_cast<float *>(const_cast<char *>(static_cast<const char *>(fwd_workspace)) + kHeaderBytes);
  } else {  // the forward once more, for the saved states alone
    p.ckpt = reinterpret_cast<float *>(ws + l.off_ckpt);
    const cudaError_t e = launch_gscan_fwd(shape->io_dtype, p, s);
    if (e != cudaSuccess) return cuda_status(e);
  }
  p.dout = dout; p.dlast = dlast_state; p.du = du; p.df = df; p.dz = dz;
  p.dbias = df_bias; p.dh0 = dinitial_state;
  if (df_bias) p.dbias_part = reinterpret_cast<float *>(ws + l.off_part);
  return cuda_status(launch_gscan_bwd(shape->io_dtype, p, s));
}

ssm_status ssm_gated_scan_step(const ssm_shape *shape, const void *u, const void *f, const void *z,
                               const float *f_bias, float *state, void *y, ssm_stream_t stream) {
  const ssm_status st = check_gscan(shape);
  if (st != SSM_OK) return st;
  if (shape->seqlen != 1) return SSM_ERR_INVALID_ARG;
  if (shape->path != SSM_PATH_AUTO || (shape->flags & SSM_FLAG_SAVE_STATES)) return SSM_ERR_UNSUPPORTED;
  if (shape->batch * shape->dim == 0) return SSM_OK;
  const size_t es = esize(shape->io_dtype);
  if (!u || !f || !state || !y || !aligned(u, es) || !aligned(f, es) || !aligned(z, es) || !aligned(y, es) ||
      !aligned(f_bias, 4) || !aligned(state, 4))
    return SSM_ERR_INVALID_ARG;
  if (y == u || y == f || y == z || y == state || state == u || state == f || state == z) return SSM_ERR_INVALID_ARG;
  GsStepParams p;
  memset(&p, 0, sizeof(p));
  p.u = u; p.f = f; p.z = z; p.bias = f_bias; p.state = state; p.y = y;
  p.batch = shape->batch; p.dim = shape->dim;
  p.untied = (shape->flags & SSM_FLAG_UNTIED) ? 1 : 0;
  const cudaError_t inj = injected_failure();
  if (inj != cudaSuccess) return cuda_status(inj);
  return cuda_status(launch_gscan_step(shape->io_dtype, p, reinterpret_cast<cudaStream_t>(stream)));
}

static ssm_status check_norm(int64_t rows, int64_t dim, int32_t io_dtype, int32_t residual_dtype, float eps) {
  if (rows < 0 || dim < 0 || !(eps >= 0.f) || std::isinf(eps)) return SSM_ERR_INVALID_ARG;
  if (io_dtype != SSM_F32 && io_dtype != SSM_BF16) return SSM_ERR_UNSUPPORTED;
  if (residual_dtype != io_dtype && residual_dtype != SSM_F32) return SSM_ERR_UNSUPPORTED;
  // a grid dimension is 31 bits; column indexes are 32
  if (rows > 2000000000 || dim > 1000000000 || (double)rows * (double)dim > 4.0e15) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

ssm_status ssm_layer_norm(int64_t rows, int64_t dim, int32_t io_dtype, int32_t residual_dtype, const void *x,
                          const void *residual, const float *weight, const float *bias, float eps, void *y,
                          void *residual_out, ssm_stream_t stream) {
  const ssm_status st = check_norm(rows, dim, io_dtype, residual_dtype, eps);
  if (st != SSM_OK) return st;
  if ((residual == nullptr) != (residual_out == nullptr)) return SSM_ERR_INVALID_ARG;
  if (rows == 0 || dim == 0) return SSM_OK;
  const size_t es = esize(io_dtype), rs = esize(residual_dtype);
  if (!x || !weight || !y || !aligned(x, es) || !aligned(y, es) || !aligned(residual, rs) ||
      !aligned(residual_out, rs) || !aligned(weight, 4) || !aligned(bias, 4))
    return SSM_ERR_INVALID_ARG;
  if (y == x || (residual && (y == residual || y == residual_out || residual_out == x))) return SSM_ERR_INVALID_ARG;
  NormParams p;
  memset(&p, 0, sizeof(p));
  p.x = x; p.res = residual; p.w = weight; p.b = bias; p.y = y; p.res_out = residual_out;
  p.rows = rows; p.dim = dim; p.eps = eps;
  const cudaError_t inj = injected_failure();
  if (inj != cudaSuccess) return cuda_status(inj);
  return cuda_status(launch_norm(io_dtype, residual ? residual_dtype : io_dtype, p,
                                 reinterpret_cast<cudaStream_t>(stream)));
}

size_t ssm_layer_norm_bwd_workspace_bytes(int64_t rows, int64_t dim) {
  if (check_norm(rows, dim, SSM_F32, SSM_F32, 0.f) != SSM_OK) return 0;
  const int sms = device_sms();
  if (sms <= 0) return 0;
  return round_up(kHeaderBytes + sizeof(float) * norm_bwd_part_floats(rows, dim, sms), 256);
}

ssm_status ssm_layer_norm_bwd(int64_t rows, int64_t dim, int32_t io_dtype, int32_t residual_dtype, const void *sum,
                              const float *weight, float eps, const void *dy, const void *dresidual_out, void *dx,
                              void *dresidual, float *dweight, float *dbias, void *workspace, size_t ws_bytes,
                              ssm_stream_t stream) {
  const ssm_status st = check_norm(rows, dim, io_dtype, residual_dtype, eps);
  if (st != SSM_OK) return st;
  if (dim == 0) return SSM_OK;
  if (!weight || !dweight || !aligned(weight, 4) || !aligned(dweight, 4) || !aligned(dbias, 4))
    return SSM_ERR_INVALID_ARG;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (rows == 0) {  // no row: parameter gradients are zero
    cudaError_t e = cudaMemsetAsync(dweight, 0, sizeof(float) * (size_t)dim, s);
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, sizeof(float) * (size_t)dim, s);
    return cuda_status(e);
  }
  const size_t es = esize(io_dtype), rs = esize(residual_dtype);
  if (!sum || !dy || !dx || !aligned(sum, rs) || !aligned(dy, es) || !aligned(dx, es) ||
      !aligned(dresidual_out, rs) || !aligned(dresidual, rs))
    return SSM_ERR_INVALID_ARG;
  if ((dresidual != nullptr) != (residual_dtype != io_dtype)) return SSM_ERR_INVALID_ARG;
  if (dx == sum || dx == dy || dx == dresidual_out || dx == dresidual ||
      (dresidual && (dresidual == sum || dresidual == dy)))
    return SSM_ERR_INVALID_ARG;
  const int sms = device_sms();
  if (sms <= 0) return SSM_ERR_CUDA;
  const size_t need = round_up(kHeaderBytes + sizeof(float) * norm_bwd_part_floats(rows, dim, sms), 256);
  if (!workspace || ws_bytes < need || !aligned(workspace, 256)) return SSM_ERR_WORKSPACE;
  NormBwdParams p;
  memset(&p, 0, sizeof(p));
  p.s = sum; p.dy = dy; p.dres_out = dresidual_out; p.w = weight; p.dx = dx; p.dres = dresidual;
  p.dw = dweight; p.db = dbias;
  p.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + kHeaderBytes);
  p.rows = rows; p.dim = dim; p.eps = eps;
  const cudaError_t inj = injected_failure();
  if (inj != cudaSuccess) return cuda_status(inj);
  return cuda_status(launch_norm_bwd(io_dtype, residual_dtype, p, sms, s));
}

}  // extern "C"
