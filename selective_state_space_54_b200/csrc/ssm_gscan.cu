// Gated linear recurrence for sm_100a: forward, backward and single step.
//   g_t = sigmoid(-(f_t + bias)),  a_t = 1 - g_t
//   h_t = a_t h_{t-1} + g_t u_t   (untied: + u_t),  h_{t-1} := 0 at a start
//   y_t = h_t SiLU(z_t)
// Backward, with d_t = dout_t SiLU(z_t) and P_t = a_t G_t (0 at a start):
//   G_t = d_t + P_{t+1},  du = g G (untied: G),  dz = dout h SiLU'(z),
//   df = G (h_{t-1} - u) a g   (untied: G h_{t-1} a g),  dh0 = P_0.
#include "ssm_layer.cuh"

namespace ssm {

namespace {

constexpr int kGsThreads = 128;

// a h = h - g h in one rounding: a itself is not formed, so a gate close to 1
// (a long memory) loses nothing to the rounding of 1 - g.
__device__ __forceinline__ float gs_keep(float g, float h) { return fmaf(-g, h, h); }

// gates of one logit: g = 1 / (1 + e^f); a = e^f g with the exponent held below
// 2^120, where a is 1 to every bit (NaN passes)
__device__ __forceinline__ float min_nan(float x, float y) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void gs_gates(float f, float &a, float &g) {
  const float e = ex2(min_nan(f * kLog2e, 120.f));
  g = rcp_approx(1.f + e);
  a = e * g;
}

template <typename T>
__global__ void k_gs_fwd(GsParams p) {
  const int64_t i = (int64_t)blockIdx.x * kGsThreads + threadIdx.x;
  if (i >= p.batch * p.dim) return;
  const int64_t b = i / p.dim, d = i - b * p.dim;
  const int64_t base = p.tok ? b * p.L * p.dim + d : i * p.L, st = p.tok ? p.dim : 1;
  const T *u = static_cast<const T *>(p.u), *f = static_cast<const T *>(p.f), *z = static_cast<const T *>(p.z);
  const float bias = p.bias ? p.bias[d] : 0.f;
  float h = p.h0 ? p.h0[i] : 0.f;
  for (int64_t t = 0; t < p.L; ++t) {
    if (p.ckpt && t % kGsCkpt == 0) p.ckpt[(b * gs_chunks(p.L) + t / kGsCkpt) * p.dim + d] = h;
    const int64_t j = base + t * st;
    float a, g;
    gs_gates(IO<T>::get(f, j) + bias, a, g);
    if (p.starts && p.starts[b * p.L + t]) h = 0.f;
    const float uv = IO<T>::get(u, j);
    h = p.untied ? gs_keep(g, h) + uv : fmaf(g, uv - h, h);
    if (p.y) IO<T>::store1(static_cast<T *>(p.y), j, z ? h * silu_fast(IO<T>::get(z, j)) : h);
  }
  if (p.last) p.last[i] = h;
}

template <typename T>
__global__ void k_gs_bwd(GsParams p) {
  const int64_t i = (int64_t)blockIdx.x * kGsThreads + threadIdx.x;
  if (i >= p.batch * p.dim) return;
  const int64_t b = i / p.dim, d = i - b * p.dim;
  const int64_t base = p.tok ? b * p.L * p.dim + d : i * p.L, st = p.tok ? p.dim : 1;
  const T *u = static_cast<const T *>(p.u), *f = static_cast<const T *>(p.f), *z = static_cast<const T *>(p.z);
  const T *dout = static_cast<const T *>(p.dout);
  T *du = static_cast<T *>(p.du), *df = static_cast<T *>(p.df), *dz = static_cast<T *>(p.dz);
  const float bias = p.bias ? p.bias[d] : 0.f;
  float P = p.dlast ? p.dlast[i] : 0.f, db = 0.f;
  float hs[kGsCkpt + 1];
  for (int64_t c = gs_chunks(p.L) - 1; c >= 0; --c) {
    const int64_t t0 = c * kGsCkpt;
    const int n = (int)(p.L - t0 < kGsCkpt ? p.L - t0 : kGsCkpt);
    float h = p.ckpt[(b * gs_chunks(p.L) + c) * p.dim + d];
    for (int k = 0; k < n; ++k) {
      const int64_t j = base + (t0 + k) * st;
      float a, g;
      gs_gates(IO<T>::get(f, j) + bias, a, g);
      if (p.starts && p.starts[b * p.L + t0 + k]) h = 0.f;
      hs[k] = h;
      const float uv = IO<T>::get(u, j);
      h = p.untied ? gs_keep(g, h) + uv : fmaf(g, uv - h, h);
    }
    hs[n] = h;
    for (int k = n - 1; k >= 0; --k) {
      const int64_t j = base + (t0 + k) * st;
      float a, g;
      gs_gates(IO<T>::get(f, j) + bias, a, g);
      const float uv = IO<T>::get(u, j), dy = IO<T>::get(dout, j);
      const float hp = hs[k], hn = p.untied ? gs_keep(g, hp) + uv : fmaf(g, uv - hp, hp);
      float dh = dy;
      if (z) {
        const float zv = IO<T>::get(z, j), s = sigmoid_f(zv);
        dh = dy * zv * s;
        IO<T>::store1(dz, j, dy * hn * s * fmaf(zv, 1.f - s, 1.f));
      }
      const float G = dh + P;
      const float dfv = G * (p.untied ? hp : hp - uv) * (a * g);
      db += dfv;
      IO<T>::store1(df, j, dfv);
      IO<T>::store1(du, j, p.untied ? G : G * g);
      P = p.starts && p.starts[b * p.L + t0 + k] ? 0.f : gs_keep(g, G);
    }
  }
  if (p.dh0) p.dh0[i] = P;
  if (p.dbias_part) p.dbias_part[i] = db;
}

__global__ void k_gs_dbias(const float *part, float *out, int64_t batch, int64_t dim) {
  const int64_t d = (int64_t)blockIdx.x * kGsThreads + threadIdx.x;
  if (d >= dim) return;
  float v = 0.f;
  for (int64_t b = 0; b < batch; ++b) v += part[b * dim + d];
  out[d] = v;
}

template <typename T>
__global__ void k_gs_step(GsStepParams p) {
  const int64_t i = (int64_t)blockIdx.x * kGsThreads + threadIdx.x;
  if (i >= p.batch * p.dim) return;
  const T *u = static_cast<const T *>(p.u), *f = static_cast<const T *>(p.f), *z = static_cast<const T *>(p.z);
  float a, g;
  gs_gates(IO<T>::get(f, i) + (p.bias ? p.bias[i % p.dim] : 0.f), a, g);
  const float uv = IO<T>::get(u, i);
  float h = p.state[i];
  h = p.untied ? gs_keep(g, h) + uv : fmaf(g, uv - h, h);
  p.state[i] = h;
  IO<T>::store1(static_cast<T *>(p.y), i, z ? h * silu_fast(IO<T>::get(z, i)) : h);
}

unsigned blocks_of(int64_t n) { return (unsigned)((n + kGsThreads - 1) / kGsThreads); }

}  // namespace

cudaError_t launch_gscan_fwd(int io_dtype, const GsParams &p, cudaStream_t s) {
  const unsigned g = blocks_of(p.batch * p.dim);
  if (io_dtype == SSM_BF16) k_gs_fwd<uint16_t><<<g, kGsThreads, 0, s>>>(p);
  else k_gs_fwd<float><<<g, kGsThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_gscan_bwd(int io_dtype, const GsParams &p, cudaStream_t s) {
  const unsigned g = blocks_of(p.batch * p.dim);
  if (io_dtype == SSM_BF16) k_gs_bwd<uint16_t><<<g, kGsThreads, 0, s>>>(p);
  else k_gs_bwd<float><<<g, kGsThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.dbias) return e;
  k_gs_dbias<<<blocks_of(p.dim), kGsThreads, 0, s>>>(p.dbias_part, p.dbias, p.batch, p.dim);
  return cudaGetLastError();
}

cudaError_t launch_gscan_step(int io_dtype, const GsStepParams &p, cudaStream_t s) {
  const unsigned g = blocks_of(p.batch * p.dim);
  if (io_dtype == SSM_BF16) k_gs_step<uint16_t><<<g, kGsThreads, 0, s>>>(p);
  else k_gs_step<float><<<g, kGsThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace ssm
