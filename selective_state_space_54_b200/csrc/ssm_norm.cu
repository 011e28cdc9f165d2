// Layer norm for sm_100a, forward (with the residual stream's addition) and
// backward.  Per row of n values:
//   s = x + residual, rounded to the residual's type; m = mean(s),
//   r = 1 / sqrt(mean((s - m)^2) + eps), q = (s - m) r, y = q w + b
//   ds = r (w dy - mean(w dy) - q mean(w dy q)) + dresidual_out
//   dw = sum over rows of dy q,  db = sum over rows of dy
#include "ssm_layer.cuh"

#include <algorithm>

namespace ssm {

namespace {

constexpr int kNormThreads = 256;

// sum over the block, the same value and order in every thread
__device__ __forceinline__ float block_sum(float v, float *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
  for (int i = 0; i < kNormThreads / 32; ++i) t += red[i];
  return t;
}

template <typename T, typename R>
__global__ void k_norm(NormParams p) {
  __shared__ float red[kNormThreads / 32];
  const int64_t base = (int64_t)blockIdx.x * p.dim;
  const T *x = static_cast<const T *>(p.x);
  const R *res = static_cast<const R *>(p.res);
  R *ro = static_cast<R *>(p.res_out);
  T *y = static_cast<T *>(p.y);
  float sum = 0.f;
  for (int64_t i = threadIdx.x; i < p.dim; i += kNormThreads) {
    float v = IO<T>::get(x, base + i);
    if (res) {
      IO<R>::store1(ro, base + i, v + IO<R>::get(res, base + i));
      v = IO<R>::get(ro, base + i);
    }
    sum += v;
  }
  auto at = [&](int64_t i) { return res ? IO<R>::get(ro, base + i) : IO<T>::get(x, base + i); };
  const float m = block_sum(sum, red) / (float)p.dim;
  float sq = 0.f;
  for (int64_t i = threadIdx.x; i < p.dim; i += kNormThreads) {
    const float c = at(i) - m;
    sq = fmaf(c, c, sq);
  }
  const float r = 1.f / sqrtf(block_sum(sq, red) / (float)p.dim + p.eps);
  for (int64_t i = threadIdx.x; i < p.dim; i += kNormThreads)
    IO<T>::store1(y, base + i, fmaf((at(i) - m) * r, p.w[i], p.b ? p.b[i] : 0.f));
}

// w dy is rounded once and the same wherever it is used (no contraction into the
// sums): a row whose terms cancel, such as one of a single column, cancels exactly.
template <typename T, typename R>
__global__ void k_norm_bwd(NormBwdParams p, float2 *stats) {
  __shared__ float red[kNormThreads / 32];
  const int64_t base = (int64_t)blockIdx.x * p.dim;
  const R *s = static_cast<const R *>(p.s), *dro = static_cast<const R *>(p.dres_out);
  const T *dy = static_cast<const T *>(p.dy);
  float a = 0.f;
  for (int64_t i = threadIdx.x; i < p.dim; i += kNormThreads) a += IO<R>::get(s, base + i);
  const float n = (float)p.dim, m = block_sum(a, red) / n;
  float sq = 0.f, c1 = 0.f, c2 = 0.f;
  for (int64_t i = threadIdx.x; i < p.dim; i += kNormThreads) {
    const float c = IO<R>::get(s, base + i) - m, wd = __fmul_rn(p.w[i], IO<T>::get(dy, base + i));
    sq = fmaf(c, c, sq);
    c1 = fmaf(wd, c, c1);
    c2 += wd;
  }
  const float r = 1.f / sqrtf(block_sum(sq, red) / n + p.eps);
  const float k1 = block_sum(c1, red) / n * r, k2 = block_sum(c2, red) / n;
  if (threadIdx.x == 0) stats[blockIdx.x] = make_float2(m, r);
  for (int64_t i = threadIdx.x; i < p.dim; i += kNormThreads) {
    const float q = (IO<R>::get(s, base + i) - m) * r, wd = __fmul_rn(p.w[i], IO<T>::get(dy, base + i));
    float v = r * (wd - k2 - q * k1);
    if (dro) v += IO<R>::get(dro, base + i);
    IO<T>::store1(static_cast<T *>(p.dx), base + i, v);
    if (p.dres) IO<R>::store1(static_cast<R *>(p.dres), base + i, v);
  }
}

template <typename T, typename R>
__global__ void k_norm_dw(NormBwdParams p, const float2 *stats) {
  const int64_t d = (int64_t)blockIdx.x * kNormThreads + threadIdx.x;
  if (d >= p.dim) return;
  float dw = 0.f, db = 0.f;
  for (int64_t row = 0; row < p.rows; ++row) {
    const float2 st = stats[row];
    const float g = IO<T>::get(static_cast<const T *>(p.dy), row * p.dim + d);
    dw = fmaf(g, (IO<R>::get(static_cast<const R *>(p.s), row * p.dim + d) - st.x) * st.y, dw);
    db += g;
  }
  p.dw[d] = dw;
  if (p.db) p.db[d] = db;
}

template <typename T, typename R>
cudaError_t norm_t(const NormParams &p, cudaStream_t s) {
  k_norm<T, R><<<(unsigned)p.rows, kNormThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T, typename R>
cudaError_t norm_bwd_t(const NormBwdParams &p, cudaStream_t s) {
  float2 *stats = reinterpret_cast<float2 *>(p.part);
  if (p.rows > 0) k_norm_bwd<T, R><<<(unsigned)p.rows, kNormThreads, 0, s>>>(p, stats);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  k_norm_dw<T, R><<<(unsigned)((p.dim + kNormThreads - 1) / kNormThreads), kNormThreads, 0, s>>>(p, stats);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm(int io_dtype, int res_dtype, const NormParams &p, cudaStream_t s) {
  if (io_dtype == SSM_F32) return norm_t<float, float>(p, s);
  return res_dtype == SSM_F32 ? norm_t<uint16_t, float>(p, s) : norm_t<uint16_t, uint16_t>(p, s);
}

size_t norm_bwd_part_floats(int64_t rows, int64_t dim, int sms) { return 2 * (size_t)rows; }

cudaError_t launch_norm_bwd(int io_dtype, int res_dtype, const NormBwdParams &p, int sms, cudaStream_t s) {
  if (io_dtype == SSM_F32) return norm_bwd_t<float, float>(p, s);
  return res_dtype == SSM_F32 ? norm_bwd_t<uint16_t, float>(p, s) : norm_bwd_t<uint16_t, uint16_t>(p, s);
}

}  // namespace ssm
