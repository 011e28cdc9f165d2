// C ABI of the layer operators beside the selective scan: the gated linear
// recurrence and layer norm.  Argument checks, workspace layout and launches;
// the public contract is include/ssm_scan.h.
#include <string.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>

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

// Schedule and workspace of a call: header (error word), saved states, then for the
// look-back schedule the ticket counter, the tiles' runs and the groups' states (zeroed
// before each launch), then the partial sums of df_bias.
struct GsPlan {
  int path = SSM_PATH_PER_GROUP;
  int64_t tiles = 1, group = 1, groups = 1, part_rows = 0;
  int sms = 0;
  size_t ckpt_bytes = 0;
  size_t off_ctl = 0, off_runs = 0, off_states = 0, end_ctl = 0;  // look-back
  size_t off_part = 0, total = 0;
};

// AUTO, channel-major: a warp per row needs enough rows to keep the memory system busy
// (each holds two passes of its row in flight); with fewer, rows longer than one tile
// are split into tiles.  Measured with z, rows as they are and in tiles, forward + backward:
// 256 x 65536 bf16 117 + 193 us and 45 + 81 us, 768 x 262144 532 + 944 and 382 + 785 us,
// 1024 x 2^20 2104 + 3747 and 1987 + 4135 us (fp32 x 65536: 213 + 379 and 221 + 447 us).
constexpr int64_t kRowsPerSm = 8;

ssm_status gs_plan(const ssm_shape *s, bool bwd, GsPlan *out) {
  GsPlan l;
  const bool tok = (s->flags & SSM_FLAG_TOKEN_MAJOR) != 0;
  const int es = (int)esize(s->io_dtype);
  const int64_t rows = s->batch * s->dim, L = s->seqlen;
  const int64_t row_tiles = L == 0 ? 0 : (gs_row_chunks(L, es) + kGsTileWarps - 1) / kGsTileWarps;
  l.path = tok ? SSM_PATH_LOOKBACK : s->path;
  if (l.path == SSM_PATH_AUTO && row_tiles <= 1) l.path = SSM_PATH_PER_GROUP;
  if (l.path != SSM_PATH_PER_GROUP) {
    l.sms = device_sms();
    if (l.sms <= 0) return SSM_ERR_CUDA;
    if (l.path == SSM_PATH_AUTO) l.path = rows < kRowsPerSm * l.sms ? SSM_PATH_LOOKBACK : SSM_PATH_PER_GROUP;
  }
  const int64_t chains = tok ? s->batch * gs_tok_groups(s->dim) : rows;  // sequences of tiles
  const int64_t width = tok ? kTokChannels : 1;
  if (l.path == SSM_PATH_LOOKBACK) l.tiles = tok ? gs_tok_tiles(L, es) : row_tiles;
  if ((double)chains * (double)l.tiles > 2.0e9) return SSM_ERR_UNSUPPORTED;  // a grid dimension
  // Tiles between two published states (a group).  One where there are enough chains: a
  // chain's state then takes about 1.2 us from tile to tile, which the tiles of the other
  // chains fill.  With fewer the chain itself would set the pace, and the tiles of a group
  // hand on their runs first (a state every group), which costs each tile a look at all of
  // them.  Measured forward, bf16: channel-major 64 x 262144 66 us with single tiles, 85 us
  // with groups of 8; token-major 64 chains (4096 channels x 32768) 444 and 362 us (groups
  // of 8), 128 chains equal, 4 chains (256 x 65536) 658 and 85 us (groups of 32).
  if (l.path == SSM_PATH_LOOKBACK && chains > 0 && chains < (tok ? 96 : 48))
    l.group = std::min<int64_t>(tok ? kTokGroup : kGsRowGroup, (512 + chains - 1) / chains);
  l.groups = (l.tiles + l.group - 1) / l.group;
  l.part_rows = s->batch * (l.path == SSM_PATH_LOOKBACK ? l.tiles : 1);
  // in the backward always: with the flag too fwd_workspace may be null, which no query sees
  const bool save = bwd || (s->flags & SSM_FLAG_SAVE_STATES);
  if (save)
    l.ckpt_bytes = round_up(sizeof(float) * (size_t)rows * (size_t)(tok ? gs_tok_tiles(L, es) : gs_row_chunks(L, es)), 256);
  size_t at = kHeaderBytes + l.ckpt_bytes;
  const bool handoff = l.path == SSM_PATH_LOOKBACK && !(tok && l.tiles == 1);
  if (handoff) {
    l.off_ctl = at;
    l.off_runs = l.off_ctl + 256;
    l.off_states = l.off_runs + (l.group > 1 ? sizeof(unsigned long long) * (size_t)chains * (size_t)l.tiles * width : 0);
    at = l.off_states + sizeof(unsigned) * (size_t)chains * (size_t)l.groups * width;
    l.end_ctl = at = round_up(at, 256);
  }
  if (bwd) {
    l.off_part = at;
    at = round_up(at + sizeof(float) * (size_t)l.part_rows * (size_t)s->dim, 256);
  }
  l.total = (save || handoff) ? at : 0;
  *out = l;
  return SSM_OK;
}

// The control words of a launch zeroed, and their places set.
cudaError_t gs_control(GsParams &p, const GsPlan &l, char *ws, cudaStream_t s) {
  p.tiles = l.tiles;
  p.group = (unsigned)l.group;
  p.groups = (unsigned)l.groups;
  p.sms = l.sms;
  if (!ws) return cudaSuccess;
  p.err = reinterpret_cast<unsigned *>(ws);
  if (!l.end_ctl) return cudaMemsetAsync(ws, 0, sizeof(unsigned), s);
  p.ticket = reinterpret_cast<unsigned *>(ws + l.off_ctl);
  p.runs = reinterpret_cast<unsigned long long *>(ws + l.off_runs);
  p.states = reinterpret_cast<unsigned *>(ws + l.off_states);
  if (l.ckpt_bytes == 0) return cudaMemsetAsync(ws, 0, l.end_ctl, s);
  const cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(unsigned), s);
  return e != cudaSuccess ? e : cudaMemsetAsync(ws + l.off_ctl, 0, l.end_ctl - l.off_ctl, s);
}

// Widest access every given pointer and row allows: 16 bytes, 4, or one element; and whether
// channel-major rows take 32-byte stores, token-major ones a pair of channels at once.
// Channel-major rows that are cut at aligned places need the pointers' alignment alone.
void gs_access(GsParams &p, size_t es, std::initializer_list<const void *> ptrs) {
  const size_t row = (size_t)(p.tok ? p.dim : p.L) * es;
  p.cut = p.tok ? 0 : gs_row_cut(p.L, (int)es);
  auto all = [&](size_t a) {
    if (row % a && !(p.cut && a >= 16)) return false;
    for (const void *q : ptrs)
      if (!aligned(q, a)) return false;
    return true;
  };
  p.vec = all(16) ? 2 : all(4) ? 1 : 0;
  p.v32 = p.tok ? all(2 * es) : all(32);
  p.start_vec = p.starts && p.L % 4 == 0 && aligned(p.starts, 4);
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

static size_t gs_workspace_bytes(const ssm_shape *shape, bool bwd) {
  GsPlan l;
  if (check_gscan(shape) != SSM_OK || shape->batch * shape->dim == 0 || shape->seqlen == 0) return 0;
  return gs_plan(shape, bwd, &l) == SSM_OK ? l.total : 0;
}

size_t ssm_gated_scan_fwd_workspace_bytes(const ssm_shape *shape) { return gs_workspace_bytes(shape, false); }

size_t ssm_gated_scan_bwd_workspace_bytes(const ssm_shape *shape) { return gs_workspace_bytes(shape, true); }

int32_t ssm_gated_scan_path(const ssm_shape *shape) {
  GsPlan l;
  if (check_gscan(shape) != SSM_OK || gs_plan(shape, false, &l) != SSM_OK) return SSM_PATH_AUTO;
  return l.path;
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
  GsPlan l;
  const ssm_status pst = gs_plan(shape, false, &l);
  if (pst != SSM_OK) return pst;
  if (l.total && (!workspace || ws_bytes < l.total || !aligned(workspace, 256))) return SSM_ERR_WORKSPACE;
  GsParams p;
  gs_fill(p, shape, u, f, z, f_bias, starts, initial_state);
  p.y = y; p.last = last_state;
  gs_access(p, es, {u, f, z, y});
  char *ws = l.total ? static_cast<char *>(workspace) : nullptr;
  if (shape->flags & SSM_FLAG_SAVE_STATES) p.ckpt = reinterpret_cast<float *>(ws + kHeaderBytes);
  cudaError_t e = injected_failure();
  if (e == cudaSuccess) e = gs_control(p, l, ws, s);
  if (e != cudaSuccess) return cuda_status(e);
  return cuda_status(launch_gscan_fwd(shape->io_dtype, l.path, p, s));
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
  GsPlan l;
  const ssm_status pst = gs_plan(shape, true, &l);
  if (pst != SSM_OK) return pst;
  if (!workspace || ws_bytes < l.total || !aligned(workspace, 256)) return SSM_ERR_WORKSPACE;
  char *ws = static_cast<char *>(workspace);
  GsParams p;
  gs_fill(p, shape, u, f, z, f_bias, starts, initial_state);
  gs_access(p, es, {u, f, z, dout, du, df, dz});
  cudaError_t e = injected_failure();
  if (e == cudaSuccess) e = gs_control(p, l, ws, s);
  if (e != cudaSuccess) return cuda_status(e);
  if (fwd_workspace) {
    p.ckpt = reinterpret_cast<float *>(const_cast<char *>(static_cast<const char *>(fwd_workspace)) + kHeaderBytes);
  } else {  // the forward once more, for the saved states alone (z plays no part in them)
    p.ckpt = reinterpret_cast<float *>(ws + kHeaderBytes);
    GsParams q = p;
    q.z = nullptr;
    e = launch_gscan_fwd(shape->io_dtype, l.path, q, s);
    // the control words once more; the error word keeps what the forward wrote
    if (e == cudaSuccess && l.end_ctl) e = cudaMemsetAsync(ws + l.off_ctl, 0, l.end_ctl - l.off_ctl, s);
    if (e != cudaSuccess) return cuda_status(e);
  }
  p.dout = dout; p.dlast = dlast_state; p.du = du; p.df = df; p.dz = dz;
  p.dbias = df_bias; p.dh0 = dinitial_state;
  p.part_rows = l.part_rows;
  if (df_bias) p.dbias_part = reinterpret_cast<float *>(ws + l.off_part);
  return cuda_status(launch_gscan_bwd(shape->io_dtype, l.path, p, s));
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

ssm_status ssm_gated_scan_test_wait_timeout(void *workspace, size_t ws_bytes, int64_t timeout_us,
                                            ssm_stream_t stream) {
  if (!workspace || ws_bytes < kHeaderBytes || !aligned(workspace, 256)) return SSM_ERR_WORKSPACE;
  if (timeout_us < 1 || timeout_us > 1000000) return SSM_ERR_INVALID_ARG;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char *ws = static_cast<char *>(workspace);
  const cudaError_t e = cudaMemsetAsync(ws, 0, kHeaderBytes, s);
  if (e != cudaSuccess) return cuda_status(e);
  // the words at byte 64 of the zeroed header are never set
  return cuda_status(launch_gs_wait_probe(reinterpret_cast<unsigned long long *>(ws + 64),
                                          reinterpret_cast<unsigned *>(ws), (unsigned long long)timeout_us * 1000ull, s));
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
  const int sms = device_sms();
  if (sms <= 0) return SSM_ERR_CUDA;
  return cuda_status(launch_norm(io_dtype, residual ? residual_dtype : io_dtype, p, sms,
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
