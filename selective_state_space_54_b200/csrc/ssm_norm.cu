// Layer norm for sm_100a, forward (with the residual stream's addition) and
// backward.  Per row of n values:
//   s = x + residual, rounded to the residual's type; m = mean(s),
//   r = 1 / sqrt(mean((s - m)^2) + eps), q = (s - m) r, y = q w + b
//   ds = r (w dy - mean(w dy) - q mean(w dy q)) + dresidual_out
//   dw = sum over rows of dy q,  db = sum over rows of dy
//
// Memory bound: every value is read once and written once.  A row sits in the
// registers of the 1 to 32 warps that share it, so the mean and then the centred
// squares are formed from registers (two short reductions, no second read and no
// difference of large sums).  w and b are read per row, from L1.  Rows wider than the
// registers hold take loops over memory instead.
#include "ssm_layer.cuh"

#include <algorithm>

namespace ssm {

namespace {

// VEC values at i: 16-byte accesses for 8, element accesses for 1
template <typename T, int VEC>
__device__ __forceinline__ void load_v(const T *p, int64_t i, float (&o)[VEC]) {
  if constexpr (VEC == 1) {
    o[0] = IO<T>::get(p, i);
  } else if constexpr (sizeof(T) == 2) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p + i));
    o[0] = bf16_lo(v.x); o[1] = bf16_hi(v.x); o[2] = bf16_lo(v.y); o[3] = bf16_hi(v.y);
    o[4] = bf16_lo(v.z); o[5] = bf16_hi(v.z); o[6] = bf16_lo(v.w); o[7] = bf16_hi(v.w);
  } else {
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p + i)), b = __ldcs(reinterpret_cast<const float4 *>(p + i) + 1);
    o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w; o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
  }
}
// w and b: read by every row, kept in L1
template <int VEC>
__device__ __forceinline__ void load_w(const float *p, int64_t i, float (&o)[VEC]) {
  if constexpr (VEC == 1) o[0] = __ldg(p + i);
  else IO<float>::load8(p, i, i + 8, true, o);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_v(T *p, int64_t i, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    IO<T>::store1(p, i, v[0]);
  } else if constexpr (sizeof(T) == 2) {
    __stcs(reinterpret_cast<uint4 *>(p + i), make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                        pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
  } else {
    __stcs(reinterpret_cast<float4 *>(p + i), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4 *>(p + i) + 1, make_float4(v[4], v[5], v[6], v[7]));
  }
}
// the same without the streaming hint, for what is read again (and may have been written
// by this thread: no read-only path)
template <typename T, int VEC>
__device__ __forceinline__ void load_again(const T *p, int64_t i, float (&o)[VEC]) {
  if constexpr (VEC == 1) {
    o[0] = IO<T>::get(p, i);
  } else if constexpr (sizeof(T) == 2) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p + i);
    o[0] = bf16_lo(v.x); o[1] = bf16_hi(v.x); o[2] = bf16_lo(v.y); o[3] = bf16_hi(v.y);
    o[4] = bf16_lo(v.z); o[5] = bf16_hi(v.z); o[6] = bf16_lo(v.w); o[7] = bf16_hi(v.w);
  } else {
    const float4 a = *reinterpret_cast<const float4 *>(p + i), b = *(reinterpret_cast<const float4 *>(p + i) + 1);
    o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w; o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_again(T *p, int64_t i, const float (&v)[VEC]) {
  if constexpr (VEC == 1) IO<T>::store1(p, i, v[0]);
  else IO<T>::store8(p, i, i + 8, true, v);
}
// the value as its type stores it
template <typename R>
__device__ __forceinline__ float stored(float v) {
  if constexpr (sizeof(R) == 2) return __bfloat162float(__float2bfloat16_rn(v));
  return v;
}

// Sums of K values over the wpr warps of a row, the same in every thread of the row and
// in a fixed order.  `red` alternates between calls, so one barrier each is enough.
template <int K>
__device__ __forceinline__ void row_sums(float (&v)[K], int wpr, float *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  }
  if (wpr == 1) return;
  const int w = threadIdx.x >> 5, first = w & ~(wpr - 1);
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) red[32 * k + w] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = 0.f;
  for (int i = 0; i < wpr; ++i) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += red[32 * k + first + i];
  }
}

// ---- forward ------------------------------------------------------------------------
// NV pieces of VEC values per thread; a block holds blockDim / (32 wpr) rows.
template <typename T, typename R, int VEC, int NV>
__global__ void k_norm(NormParams p, int wpr) {
  __shared__ float red[2][32];
  const int tpr = 32 * wpr, rpb = blockDim.x / tpr, tid = threadIdx.x & (tpr - 1);
  const int64_t row = (int64_t)blockIdx.x * rpb + threadIdx.x / tpr;
  const bool live = row < p.rows;  // the last block's spare threads only keep the barriers company
  const int64_t base = row * p.dim;
  const int dim = (int)p.dim;
  const T *x = static_cast<const T *>(p.x) + base;
  float v[NV][VEC];
  float sum[1] = {0.f};
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = (k * tpr + tid) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[k][e] = 0.f;
    if (live && i < dim) load_v<T, VEC>(x, i, v[k]);
  }
  if (p.res) {
    const R *res = static_cast<const R *>(p.res) + base;
    R *ro = static_cast<R *>(p.res_out) + base;
    float a[NV][VEC];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = (k * tpr + tid) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) a[k][e] = 0.f;
      if (live && i < dim) load_v<R, VEC>(res, i, a[k]);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = (k * tpr + tid) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[k][e] = stored<R>(v[k][e] + a[k][e]);
      if (live && i < dim) store_v<R, VEC>(ro, i, v[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < NV; ++k) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum[0] += v[k][e];
  }
  row_sums<1>(sum, wpr, red[0]);
  const float m = sum[0] / (float)dim;
  float sq[1] = {0.f};
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const bool in = (k * tpr + tid) * VEC < dim;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      v[k][e] -= m;
      if (in) sq[0] = fmaf(v[k][e], v[k][e], sq[0]);
    }
  }
  row_sums<1>(sq, wpr, red[1]);
  if (!live) return;
  const float r = 1.f / sqrtf(sq[0] / (float)dim + p.eps);
  T *y = static_cast<T *>(p.y) + base;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = (k * tpr + tid) * VEC;
    if (i >= dim) continue;
    float w[VEC], b[VEC];
    load_w<VEC>(p.w, i, w);
    if (p.b) load_w<VEC>(p.b, i, b);
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[e] = p.b ? fmaf(v[k][e] * r, w[e], b[e]) : v[k][e] * r * w[e];
    store_v<T, VEC>(y, i, w);
  }
}

constexpr int kWideThreads = 512;

// rows wider than the registers: three walks over the row, the later ones from L2
template <typename T, typename R, int VEC>
__global__ void __launch_bounds__(kWideThreads) k_norm_wide(NormParams p) {
  __shared__ float red[2][32];
  const int64_t base = (int64_t)blockIdx.x * p.dim;
  const T *x = static_cast<const T *>(p.x) + base;
  const R *res = static_cast<const R *>(p.res);
  R *ro = static_cast<R *>(p.res_out) + base;
  T *y = static_cast<T *>(p.y) + base;
  const int64_t i0 = (int64_t)threadIdx.x * VEC, step = (int64_t)kWideThreads * VEC;
  float sum[1] = {0.f}, sq[1] = {0.f}, v[VEC], a[VEC], w[VEC];
  for (int64_t i = i0; i < p.dim; i += step) {
    load_again<T, VEC>(x, i, v);
    if (res) {
      load_again<R, VEC>(res + base, i, a);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = stored<R>(v[e] + a[e]);
      store_again<R, VEC>(ro, i, v);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum[0] += v[e];
  }
  // a thread reads back only what it wrote itself
  auto at = [&](int64_t i) {
    if (res) load_again<R, VEC>(ro, i, v);
    else load_again<T, VEC>(x, i, v);
  };
  row_sums<1>(sum, kWideThreads / 32, red[0]);
  const float m = sum[0] / (float)p.dim;
  for (int64_t i = i0; i < p.dim; i += step) {
    at(i);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float c = v[e] - m;
      sq[0] = fmaf(c, c, sq[0]);
    }
  }
  row_sums<1>(sq, kWideThreads / 32, red[1]);
  const float r = 1.f / sqrtf(sq[0] / (float)p.dim + p.eps);
  for (int64_t i = i0; i < p.dim; i += step) {
    at(i);
    load_w<VEC>(p.w, i, w);
    if (p.b) load_w<VEC>(p.b, i, a);
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[e] = p.b ? fmaf((v[e] - m) * r, w[e], a[e]) : (v[e] - m) * r * w[e];
    store_v<T, VEC>(y, i, w);
  }
}

// ---- backward -----------------------------------------------------------------------
// Blocks walk the rows, wpr warps a row, each thread on the same
// columns of every row, whose dw and db it sums in registers; the block's sums go to the
// workspace and k_norm_sum adds them in a fixed order.  w dy is rounded once and the same
// wherever it is used (no contraction into the sums): a row whose terms cancel, such as
// one of a single column, cancels exactly.
// WARPS per block: 8, or 16 for rows that 8 do not hold.
template <typename T, typename R, int VEC, int NV, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, WARPS > 8 ? 1 : VEC * NV <= (VEC == 8 ? 8 : 4) ? 3 : 2)
    k_norm_bwd(NormBwdParams p, int wpr) {
  constexpr int kBwdThreads = 32 * WARPS;
  __shared__ float red[2][96];
  __shared__ float acc[kBwdThreads][9];
  const int tpr = 32 * wpr, rpb = kBwdThreads / tpr, tid = threadIdx.x & (tpr - 1);
  const int dim = (int)p.dim;
  const float n = (float)dim;
  float dw[NV][VEC], db[NV][VEC], w[NV][VEC];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = (k * tpr + tid) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[k][e] = db[k][e] = w[k][e] = 0.f;
    if (i < dim) load_w<VEC>(p.w, i, w[k]);
  }
  for (int64_t r0 = (int64_t)blockIdx.x * rpb; r0 < p.rows; r0 += (int64_t)gridDim.x * rpb) {
    const int64_t row = r0 + threadIdx.x / tpr, base = row * p.dim;
    const bool live = row < p.rows;
    float c[NV][VEC], g[NV][VEC], o[NV][VEC];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = (k * tpr + tid) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) c[k][e] = g[k][e] = o[k][e] = 0.f;
      if (live && i < dim) {
        load_v<R, VEC>(static_cast<const R *>(p.s) + base, i, c[k]);
        load_v<T, VEC>(static_cast<const T *>(p.dy) + base, i, g[k]);
      }
    }
    if (p.dres_out) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int i = (k * tpr + tid) * VEC;
        if (live && i < dim) load_v<R, VEC>(static_cast<const R *>(p.dres_out) + base, i, o[k]);
      }
    }
    float sum[1] = {0.f}, s3[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) sum[0] += c[k][e];
    }
    row_sums<1>(sum, wpr, red[0]);
    const float m = sum[0] / n;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if ((k * tpr + tid) * VEC < dim) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          c[k][e] -= m;
          const float wd = __fmul_rn(w[k][e], g[k][e]);
          s3[0] = fmaf(c[k][e], c[k][e], s3[0]);
          s3[1] = fmaf(wd, c[k][e], s3[1]);
          s3[2] += wd;
        }
      }
    }
    row_sums<3>(s3, wpr, red[1]);
    const float r = 1.f / sqrtf(s3[0] / n + p.eps), k1 = s3[1] / n * r, k2 = s3[2] / n;
    if (!live) continue;  // only in the last round: the barriers are behind
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = (k * tpr + tid) * VEC;
      if (i >= dim) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float q = c[k][e] * r, wd = __fmul_rn(w[k][e], g[k][e]);
        dw[k][e] = fmaf(g[k][e], q, dw[k][e]);
        db[k][e] += g[k][e];
        o[k][e] = fmaf(r, (wd - k2) - q * k1, o[k][e]);
      }
      store_v<T, VEC>(static_cast<T *>(p.dx) + base, i, o[k]);
      if (p.dres) store_v<R, VEC>(static_cast<R *>(p.dres) + base, i, o[k]);
    }
  }
  // the block's rows' sums together, then out: [block][2][dim]
  float *part = p.part + (int64_t)blockIdx.x * 2 * p.dim;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = (k * tpr + tid) * VEC;
      if (rpb > 1) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[threadIdx.x][e] = h ? db[k][e] : dw[k][e];
        __syncthreads();
        if (threadIdx.x < tpr && i < dim) {
          float t[VEC];
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            t[e] = 0.f;
            for (int j = 0; j < rpb; ++j) t[e] += acc[j * tpr + tid][e];
          }
#pragma unroll
          for (int e = 0; e < VEC; ++e) part[h * p.dim + i + e] = t[e];
        }
      } else if (i < dim) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) part[h * p.dim + i + e] = h ? db[k][e] : dw[k][e];
      }
    }
  }
}

// wide rows: ds by walks over the row (one block each), mean and r kept for the columns
template <typename T, typename R, int VEC>
__global__ void __launch_bounds__(kWideThreads) k_norm_bwd_wide(NormBwdParams p, float2 *stats) {
  __shared__ float red[2][96];
  const int64_t base = (int64_t)blockIdx.x * p.dim;
  const R *s = static_cast<const R *>(p.s) + base;
  const T *dy = static_cast<const T *>(p.dy) + base;
  const int64_t i0 = (int64_t)threadIdx.x * VEC, step = (int64_t)kWideThreads * VEC;
  const float n = (float)p.dim;
  float sum[1] = {0.f}, s3[3] = {0.f, 0.f, 0.f}, c[VEC], g[VEC], w[VEC], o[VEC];
  for (int64_t i = i0; i < p.dim; i += step) {
    load_again<R, VEC>(s, i, c);
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum[0] += c[e];
  }
  row_sums<1>(sum, kWideThreads / 32, red[0]);
  const float m = sum[0] / n;
  for (int64_t i = i0; i < p.dim; i += step) {
    load_again<R, VEC>(s, i, c);
    load_again<T, VEC>(dy, i, g);
    load_w<VEC>(p.w, i, w);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float d = c[e] - m, wd = __fmul_rn(w[e], g[e]);
      s3[0] = fmaf(d, d, s3[0]);
      s3[1] = fmaf(wd, d, s3[1]);
      s3[2] += wd;
    }
  }
  row_sums<3>(s3, kWideThreads / 32, red[1]);
  const float r = 1.f / sqrtf(s3[0] / n + p.eps), k1 = s3[1] / n * r, k2 = s3[2] / n;
  if (threadIdx.x == 0) stats[blockIdx.x] = make_float2(m, r);
  for (int64_t i = i0; i < p.dim; i += step) {
    load_again<R, VEC>(s, i, c);
    load_again<T, VEC>(dy, i, g);
    load_w<VEC>(p.w, i, w);
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[e] = 0.f;
    if (p.dres_out) load_again<R, VEC>(static_cast<const R *>(p.dres_out) + base, i, o);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float q = (c[e] - m) * r, wd = __fmul_rn(w[e], g[e]);
      o[e] = fmaf(r, (wd - k2) - q * k1, o[e]);
    }
    store_v<T, VEC>(static_cast<T *>(p.dx) + base, i, o);
    if (p.dres) store_v<R, VEC>(static_cast<R *>(p.dres) + base, i, o);
  }
}

// wide rows: dw and db of 256 columns over every gridDim.y-th row
template <typename T, typename R>
__global__ void __launch_bounds__(256) k_norm_cols(NormBwdParams p, const float2 *stats) {
  const int64_t d = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (d >= p.dim) return;
  float dw[4] = {0.f, 0.f, 0.f, 0.f}, db[4] = {0.f, 0.f, 0.f, 0.f};
  const int64_t step = gridDim.y;
  int64_t row = blockIdx.y;
  auto add = [&](int64_t r, int k) {
    const float2 st = stats[r];
    const float g = IO<T>::get(static_cast<const T *>(p.dy), r * p.dim + d);
    dw[k] = fmaf(g, (IO<R>::get(static_cast<const R *>(p.s), r * p.dim + d) - st.x) * st.y, dw[k]);
    db[k] += g;
  };
  for (; row + 3 * step < p.rows; row += 4 * step) {
#pragma unroll
    for (int k = 0; k < 4; ++k) add(row + k * step, k);
  }
  for (; row < p.rows; row += step) add(row, 0);
  float *part = p.part + (int64_t)blockIdx.y * 2 * p.dim;
  part[d] = (dw[0] + dw[1]) + (dw[2] + dw[3]);
  part[p.dim + d] = (db[0] + db[1]) + (db[2] + db[3]);
}

// dw and db: sums over the blocks' parts [n][2 dim], 32 columns a block, 32 threads a column
__global__ void __launch_bounds__(1024) k_norm_sum(const float *part, float *dw, float *db, int64_t n, int64_t dim) {
  __shared__ float s[32][33];
  const int64_t cols = db ? 2 * dim : dim, d = (int64_t)blockIdx.x * 32 + threadIdx.x;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (d < cols) {
    int64_t r = threadIdx.y;
    for (; r + 96 < n; r += 128) {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] += part[(r + 32 * k) * 2 * dim + d];
    }
    for (; r < n; r += 32) v[0] += part[r * 2 * dim + d];
  }
  s[threadIdx.y][threadIdx.x] = (v[0] + v[1]) + (v[2] + v[3]);
  __syncthreads();
  float t = s[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && c < cols) (c < dim ? dw[c] : db[c - dim]) = t;
}

// ---- launches -----------------------------------------------------------------------
bool a16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int kFwdValues = 32;  // values of a row a thread holds at most, forward
constexpr int kBwdValues = 16;  // backward (beside as many dw, db and w)
constexpr int kBwdWidest = 16 * 32 * kBwdValues;

template <typename T, typename R, int VEC, int NV>
cudaError_t norm_nv(const NormParams &p, int wpr, cudaStream_t s) {
  const int threads = std::max(128, 32 * wpr), rpb = threads / (32 * wpr);
  k_norm<T, R, VEC, NV><<<(unsigned)((p.rows + rpb - 1) / rpb), threads, 0, s>>>(p, wpr);
  return cudaGetLastError();
}

template <typename T, typename R>
cudaError_t norm_t(const NormParams &p, int sms, cudaStream_t s) {
  const bool vec = p.dim % 8 == 0 && a16(p.x) && a16(p.res) && a16(p.y) && a16(p.res_out) && a16(p.w) && a16(p.b);
  const int per = vec ? 8 : 1;
  if (p.dim > 512 * kFwdValues) {
    if (vec) k_norm_wide<T, R, 8><<<(unsigned)p.rows, kWideThreads, 0, s>>>(p);
    else k_norm_wide<T, R, 1><<<(unsigned)p.rows, kWideThreads, 0, s>>>(p);
    return cudaGetLastError();
  }
  // the fewest warps a row that hold it; more while the rows leave the machine empty
  int wpr = 1;
  while (wpr * 32 * kFwdValues < p.dim) wpr *= 2;
  while (wpr < 16 && p.rows * wpr < 16 * sms && wpr * 32 * per < p.dim) wpr *= 2;
  const int nv = (int)((p.dim + 32 * wpr * per - 1) / (32 * wpr * per));
  if (vec) {
    if (nv <= 1) return norm_nv<T, R, 8, 1>(p, wpr, s);
    if (nv <= 2) return norm_nv<T, R, 8, 2>(p, wpr, s);
    if (nv <= 3) return norm_nv<T, R, 8, 3>(p, wpr, s);
    return norm_nv<T, R, 8, 4>(p, wpr, s);
  }
  if (nv <= 4) return norm_nv<T, R, 1, 4>(p, wpr, s);
  if (nv <= 8) return norm_nv<T, R, 1, 8>(p, wpr, s);
  if (nv <= 16) return norm_nv<T, R, 1, 16>(p, wpr, s);
  return norm_nv<T, R, 1, 32>(p, wpr, s);
}

// blocks of the backward: enough to fill the machine, no more than there are rows
int64_t bwd_blocks_for(int64_t rows, int sms) { return std::max<int64_t>(1, std::min<int64_t>(rows, 3 * (int64_t)sms)); }

template <typename T, typename R, int VEC, int NV, int WARPS>
cudaError_t norm_bwd_nv(const NormBwdParams &p, int wpr, int sms, cudaStream_t s) {
  auto kern = k_norm_bwd<T, R, VEC, NV, WARPS>;
  int occ = 0;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, 32 * WARPS, 0);
  if (e != cudaSuccess) return e;
  const int rpb = WARPS / wpr;
  const int64_t fit = (int64_t)std::max(occ, 1) * sms, need = (p.rows + rpb - 1) / rpb;
  const int64_t blocks = std::min(std::min(need, fit), bwd_blocks_for(p.rows, sms));
  kern<<<(unsigned)blocks, 32 * WARPS, 0, s>>>(p, wpr);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  k_norm_sum<<<(unsigned)(((p.db ? 2 : 1) * p.dim + 31) / 32), dim3(32, 32), 0, s>>>(p.part, p.dw, p.db, blocks, p.dim);
  return cudaGetLastError();
}

template <typename T, typename R>
cudaError_t norm_bwd_t(const NormBwdParams &p, int sms, cudaStream_t s) {
  const bool vec = p.dim % 8 == 0 && a16(p.s) && a16(p.dy) && a16(p.dres_out) && a16(p.dx) && a16(p.dres) && a16(p.w);
  if (p.dim > kBwdWidest) {
    const int64_t splits = bwd_blocks_for((p.rows + 31) / 32, sms);
    float2 *stats = reinterpret_cast<float2 *>(p.part + splits * 2 * p.dim);
    if (vec) k_norm_bwd_wide<T, R, 8><<<(unsigned)p.rows, kWideThreads, 0, s>>>(p, stats);
    else k_norm_bwd_wide<T, R, 1><<<(unsigned)p.rows, kWideThreads, 0, s>>>(p, stats);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    k_norm_cols<T, R><<<dim3((unsigned)((p.dim + 255) / 256), (unsigned)splits), 256, 0, s>>>(p, stats);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    k_norm_sum<<<(unsigned)(((p.db ? 2 : 1) * p.dim + 31) / 32), dim3(32, 32), 0, s>>>(p.part, p.dw, p.db, splits, p.dim);
    return cudaGetLastError();
  }
  // 8 values a thread while 8 warps hold the row, then 16, then 16 warps
  int wpr = 1;
  while (wpr < 8 && wpr * 256 < p.dim) wpr *= 2;
  if (p.dim > 8 * 32 * kBwdValues)
    return vec ? norm_bwd_nv<T, R, 8, 2, 16>(p, 16, sms, s) : norm_bwd_nv<T, R, 1, 16, 16>(p, 16, sms, s);
  const bool two = wpr * 256 < p.dim;
  if (vec) return two ? norm_bwd_nv<T, R, 8, 2, 8>(p, wpr, sms, s) : norm_bwd_nv<T, R, 8, 1, 8>(p, wpr, sms, s);
  if (wpr * 128 >= p.dim) return norm_bwd_nv<T, R, 1, 4, 8>(p, wpr, sms, s);
  return two ? norm_bwd_nv<T, R, 1, 16, 8>(p, wpr, sms, s) : norm_bwd_nv<T, R, 1, 8, 8>(p, wpr, sms, s);
}

}  // namespace

cudaError_t launch_norm(int io_dtype, int res_dtype, const NormParams &p, int sms, cudaStream_t s) {
  if (io_dtype == SSM_F32) return norm_t<float, float>(p, sms, s);
  return res_dtype == SSM_F32 ? norm_t<uint16_t, float>(p, sms, s) : norm_t<uint16_t, uint16_t>(p, sms, s);
}

size_t norm_bwd_part_floats(int64_t rows, int64_t dim, int sms) {
  return (size_t)bwd_blocks_for(rows, sms) * 2 * (size_t)dim + (dim > kBwdWidest ? 2 * (size_t)rows : 0);
}

cudaError_t launch_norm_bwd(int io_dtype, int res_dtype, const NormBwdParams &p, int sms, cudaStream_t s) {
  if (io_dtype == SSM_F32) return norm_bwd_t<float, float>(p, sms, s);
  return res_dtype == SSM_F32 ? norm_bwd_t<uint16_t, float>(p, sms, s) : norm_bwd_t<uint16_t, uint16_t>(p, sms, s);
}

}  // namespace ssm
