// Gated recurrence: the single step, the sum of the bias gradient's partials, and the
// choice between the layouts' kernels.
#include "ssm_gscan.cuh"

namespace ssm {

namespace {

constexpr int kStepThreads = 128;

// One token: 2 bytes each of u, f, z, y and 8 of state per channel in bf16, so HBM (or
// L2, for one batch) bounds it, and below some 1e5 channels the launch does.  VEC: a
// thread takes 8 neighbouring channels of one batch element with 16-byte accesses.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kStepThreads) k_gs_step(GsStepParams p) {
  constexpr int N = VEC ? 8 : 1;
  const int64_t i = ((int64_t)blockIdx.x * kStepThreads + threadIdx.x) * N;
  if (i >= p.batch * p.dim) return;
  const T *u = static_cast<const T *>(p.u), *f = static_cast<const T *>(p.f), *z = static_cast<const T *>(p.z);
  T *y = static_cast<T *>(p.y);
  const int64_t d = i % p.dim;
  float uv[8], fv[8], zv[8], hv[8], bv[8];
  if constexpr (VEC) {
    IO<T>::load8(f, i, i + 8, true, fv);
    IO<T>::load8(u, i, i + 8, true, uv);
    if (z) IO<T>::load8(z, i, i + 8, true, zv);
    // the state is read and overwritten: no read-only path
    const float4 a = *reinterpret_cast<const float4 *>(p.state + i), b = *reinterpret_cast<const float4 *>(p.state + i + 4);
    hv[0] = a.x; hv[1] = a.y; hv[2] = a.z; hv[3] = a.w; hv[4] = b.x; hv[5] = b.y; hv[6] = b.z; hv[7] = b.w;
    if (p.bias) IO<float>::load8(p.bias, d, d + 8, true, bv);
  } else {
    fv[0] = IO<T>::get(f, i);
    uv[0] = IO<T>::get(u, i);
    if (z) zv[0] = IO<T>::get(z, i);
    hv[0] = p.state[i];
    if (p.bias) bv[0] = p.bias[d];
  }
  float o[8];
  // channels in pairs; a single one goes with itself
#pragma unroll
  for (int k = 0; k < N; k += 2) {
    constexpr int J = VEC ? 1 : 0;
    const f2 b2 = p.bias ? mul2(pack2(bv[k], bv[k + J]), splat2(kLog2e)) : splat2(0.f);
    const f2 c = signed_gate2(pack2(fv[k], fv[k + J]), b2), h = pack2(hv[k], hv[k + J]), u = pack2(uv[k], uv[k + J]);
    float lo, hi;
    unpack2(p.untied ? state_step<false, true>(h, c, u) : state_step<true, true>(h, c, u), lo, hi);
    hv[k] = lo;
    hv[k + J] = hi;
    o[k] = z ? hv[k] * silu_fast(zv[k]) : hv[k];
    o[k + J] = z ? hv[k + J] * silu_fast(zv[k + J]) : hv[k + J];
  }
  if constexpr (VEC) {
    IO<float>::store8(p.state, i, i + 8, true, hv);
    IO<T>::store8(y, i, i + 8, true, o);
  } else {
    p.state[i] = hv[0];
    IO<T>::store1(y, i, o[0]);
  }
}

// Sum over the rows of part [n][dim]: 32 channels a block, 32 threads a channel, each
// adding every 32nd row, joined in a fixed order.
__global__ void __launch_bounds__(1024) k_gs_dbias(const float *part, float *out, int64_t n, int64_t dim) {
  __shared__ float s[32][33];
  const int64_t d = (int64_t)blockIdx.x * 32 + threadIdx.x;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (d < dim) {
    int64_t r = threadIdx.y;
    for (; r + 96 < n; r += 128) {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] += part[(r + 32 * k) * dim + d];
    }
    for (; r < n; r += 32) v[0] += part[r * dim + d];
  }
  s[threadIdx.y][threadIdx.x] = (v[0] + v[1]) + (v[2] + v[3]);
  __syncthreads();
  float t = s[threadIdx.x][threadIdx.y];  // channel threadIdx.y, over the warp
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  const int64_t dd = (int64_t)blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && dd < dim) out[dd] = t;
}

// The tiles' wait on its own (a test hook): two warps, each thread at one of 8 words
// that nothing sets.
__global__ void __launch_bounds__(64) k_gs_wait_probe(const unsigned long long *words, unsigned *err,
                                                      unsigned long long limit_ns) {
  unsigned long long started = 0;
  unsigned n = 0;
  while (look64(words + (threadIdx.x & 7)) == 0ull)
    if (!spun(started, n, err, limit_ns)) break;
}

template <typename T>
cudaError_t launch_step_t(const GsStepParams &p, bool vec, cudaStream_t s) {
  const int64_t n = p.batch * p.dim, per = (int64_t)kStepThreads * (vec ? 8 : 1), blocks = (n + per - 1) / per;
  if (vec) k_gs_step<T, true><<<(unsigned)blocks, kStepThreads, 0, s>>>(p);
  else k_gs_step<T, false><<<(unsigned)blocks, kStepThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gscan_fwd(int io_dtype, int path, const GsParams &p, cudaStream_t s) {
  return p.tok ? launch_gs_tok_fwd(io_dtype, p, s) : launch_gs_rows_fwd(io_dtype, path, p, s);
}

cudaError_t launch_gscan_bwd(int io_dtype, int path, const GsParams &p, cudaStream_t s) {
  const cudaError_t e = p.tok ? launch_gs_tok_bwd(io_dtype, p, s) : launch_gs_rows_bwd(io_dtype, path, p, s);
  if (e != cudaSuccess || !p.dbias) return e;
  k_gs_dbias<<<(unsigned)((p.dim + 31) / 32), dim3(32, 32), 0, s>>>(p.dbias_part, p.dbias, p.part_rows, p.dim);
  return cudaGetLastError();
}

cudaError_t launch_gscan_step(int io_dtype, const GsStepParams &p, cudaStream_t s) {
  auto a16 = [](const void *q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; };
  const bool vec = p.dim % 8 == 0 && a16(p.u) && a16(p.f) && a16(p.z) && a16(p.y) && a16(p.state) && a16(p.bias);
  return io_dtype == SSM_BF16 ? launch_step_t<uint16_t>(p, vec, s) : launch_step_t<float>(p, vec, s);
}

cudaError_t launch_gs_wait_probe(const unsigned long long *words, unsigned *err, unsigned long long limit_ns,
                                 cudaStream_t s) {
  k_gs_wait_probe<<<1, 64, 0, s>>>(words, err, limit_ns);
  return cudaGetLastError();
}

}  // namespace ssm
