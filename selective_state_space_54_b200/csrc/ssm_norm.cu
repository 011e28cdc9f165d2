// Layer norm for sm_100a, forward (with the residual stream's addition) and
// backward.  Per row of n values:
//   s = x + residual, rounded to the residual's type; m = mean(s),
//   r = 1 / sqrt(mean((s - m)^2) + eps), q = (s - m) r, y = q w + b
//   ds = r (w dy - mean(w dy) - q mean(w dy q)) + dresidual_out
//   dw = sum over rows of dy q,  db = sum over rows of dy
//
// Memory bound: every value is read once and written once.  1 to 16 warps share a row;
// blocks walk the rows, each thread always on the same columns.  Where rows allow 16-byte
// (fp32: 32-byte) accesses a thread loads its columns of the next rows into registers while
// it works on the current ones; the mean and then the centred squares are formed from
// registers (two short reductions, no second read and no difference of large sums), on f32x2
// pairs.  What bounds such a kernel next to HBM is the work per row that does not shrink with
// the row's share of a thread: reductions, barriers, addresses, w and b.  So the forward takes
// two rows at a time where the registers allow.  Measured and dropped: rows copied ahead by
// cp.async (16-byte copies of fp32 rows read every sector twice: 170 against 136 us at
// 16384 x 4096 on an fp32 residual), w and b read from L1 for every single row.
// Rows wider than 16384 (backward 8192) take walks over memory.  Forward and backward of the
// measured copy rate (6.46 TB/s): 32768 x 4096 bf16 110 us, 76 %; 16384 x 4096 bf16 on an
// fp32 residual 343 us, 85 % of the 291 us that the two calls' own accesses take.
#include "ssm_layer.cuh"

#include <algorithm>
#include <initializer_list>
#include <utility>

namespace ssm {

namespace {

// VEC values at i, 16-byte accesses for 8 and element accesses for 1: w and b, which every
// row reads
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

// Sums of K values over the wpr warps of a row, the same in every thread of the row and in
// a fixed order.  Each row of the block has 16 slots a value, 0 where there is no warp; the
// array alternates between calls, so one barrier each is enough.  Q: quarters of the 16 in use.
struct alignas(16) RowSums {
  float v[3][8 * 16];
};
__device__ __forceinline__ void clear(RowSums &r) {
  for (int i = threadIdx.x; i < 3 * 8 * 16; i += blockDim.x) (&r.v[0][0])[i] = 0.f;
}
template <int K, int Q = 4>
__device__ __forceinline__ void row_sums(float (&v)[K], int wpr, int group, RowSums &red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  }
  if (wpr == 1) return;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) red.v[k][group * 16 + (threadIdx.x >> 5) - group * wpr] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    v[k] = 0.f;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const float4 q = *reinterpret_cast<const float4 *>(&red.v[k][group * 16 + 4 * i]);
      v[k] += (q.x + q.y) + (q.z + q.w);
    }
  }
}

// ---- 8 neighbouring values of a row ---------------------------------------------------
template <typename T>
struct Raw8 {
  uint32_t w[8 * sizeof(T) / 4];
};
template <typename T>
__device__ __forceinline__ void load8(Raw8<T> &r, const T *p) {
  if constexpr (sizeof(T) == 2) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
    r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
  } else {
    asm volatile("ld.global.cs.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]),
                   "=r"(r.w[7])
                 : "l"(p));
  }
}
template <typename T>
__device__ __forceinline__ f2 pair_of(const Raw8<T> &r, int e) {
  if constexpr (sizeof(T) == 2) return pack2(bf16_lo(r.w[e]), bf16_hi(r.w[e]));
  else return pack2(__uint_as_float(r.w[2 * e]), __uint_as_float(r.w[2 * e + 1]));
}
template <typename T>
__device__ __forceinline__ void put8(T *p, const f2 (&o)[4]) {
  float v[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) unpack2(o[k], v[2 * k], v[2 * k + 1]);
  if constexpr (sizeof(T) == 2) {
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                    pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
  } else {
    asm volatile("st.global.cs.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
  }
}
// ---- rows whose start is not aligned ----------------------------------------------------
// A row begins `pad` values (0..7) after an aligned place.  Its pieces are the aligned ones,
// so that its first and last may reach into the neighbouring rows: they are loaded whole (one by
// one only at the tensor's own ends), what is not the row's counts as 0, and only the row's
// own values are stored.  Rows a `period`
// (8 over the greatest common divisor of 8 and dim) apart have the same pad: a block takes
// rows of one pad only, and every thread keeps its columns.
struct Pieces {
  int period, cls, pad;  // the block's class of rows: row = cls (mod period)
};
template <bool SHIFT>
__device__ __forceinline__ Pieces pieces_of(int period, int base, int64_t dim) {
  if constexpr (!SHIFT) return {1, 0, 0};
  const int cls = blockIdx.x % period;
  return {period, cls, (int)((base + cls * (dim & 7)) & 7)};
}
__device__ __forceinline__ bool whole(int i, int dim) { return i >= 0 && i + 8 <= dim; }
// the piece at column i of row r (the tensor's first value at p)
template <typename T, bool SHIFT>
__device__ __forceinline__ void load_piece(Raw8<T> &q, const void *p, int64_t r, int64_t rows, int i, int dim) {
  const int64_t at = r * dim + i;
  const T *src = static_cast<const T *>(p) + at;
  if (!SHIFT || (at >= 0 && at + 8 <= rows * dim)) {
    load8<T>(q, src);
  } else {
#pragma unroll
    for (int w = 0; w < (int)(8 * sizeof(T) / 4); ++w) q.w[w] = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (i + e >= 0 && i + e < dim) {
        if constexpr (sizeof(T) == 2) q.w[e >> 1] |= (uint32_t)src[e] << (16 * (e & 1));
        else q.w[e] = __float_as_uint(src[e]);
      }
  }
}
template <typename T, bool SHIFT>
__device__ __forceinline__ void put_piece(T *p, const f2 (&o)[4], int i, int dim) {
  if (!SHIFT || whole(i, dim)) {
    put8<T>(p, o);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float a, b;
      unpack2(o[e >> 1], a, b);
      if (i + e >= 0 && i + e < dim) IO<T>::store1(p, e, (e & 1) ? b : a);
    }
  }
}
// the values of a piece that are not the row's, set to 0
template <bool SHIFT>
__device__ __forceinline__ void keep_own(f2 (&v)[4], int i, int dim) {
  if (SHIFT && !whole(i, dim)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a, b;
      unpack2(v[e], a, b);
      const int k = i + 2 * e;
      v[e] = pack2(k >= 0 && k < dim ? a : 0.f, k + 1 >= 0 && k + 1 < dim ? b : 0.f);
    }
  }
}
template <typename T>
__device__ __forceinline__ void drop_others(Raw8<T> &r, int i, int dim) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (i + e < 0 || i + e >= dim) {
      if constexpr (sizeof(T) == 2) r.w[e >> 1] &= (e & 1) ? 0x0000ffffu : 0xffff0000u;
      else r.w[e] = 0u;
    }
}
// w (and b) moved by pad into shared memory, 0 outside the row, n columns in all
__device__ __forceinline__ void shift_w(float *to, const float *w, int pad, int dim, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) to[i] = w && i >= pad && i - pad < dim ? w[i - pad] : 0.f;
}
__device__ __forceinline__ void get_w_shared(const float *p, f2 (&o)[4]) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(p), b = *(reinterpret_cast<const ulonglong2 *>(p) + 1);
  o[0] = a.x; o[1] = a.y; o[2] = b.x; o[3] = b.y;
}

// 8 fp32 parameters as pairs
__device__ __forceinline__ void get_w(const float *p, f2 (&o)[4]) {
  const ulonglong2 a = __ldg(reinterpret_cast<const ulonglong2 *>(p)), b = __ldg(reinterpret_cast<const ulonglong2 *>(p) + 1);
  o[0] = a.x; o[1] = a.y; o[2] = b.x; o[3] = b.y;
}
__device__ __forceinline__ f2 stored_bf16(f2 v) {
  float a, b;
  unpack2(v, a, b);
  const uint32_t w = pack_bf16x2(a, b);
  return pack2(bf16_lo(w), bf16_hi(w));
}
__device__ __forceinline__ float both(f2 v) {
  float a, b;
  unpack2(v, a, b);
  return a + b;
}

// ---- forward ------------------------------------------------------------------------
// NV pieces of 8 values per thread and row, RB rows at a time, wpr warps a row; a block
// holds blockDim / (32 wpr) such groups.  Q as in row_sums; MAXT threads, MINB blocks an SM.
template <typename T, typename R, bool RES, int NV, int RB, int Q, int MAXT, int MINB, bool SHIFT>
__global__ void __launch_bounds__(MAXT, MINB) k_norm_rows(NormParams p, int wpr, int period, int pad0) {
  extern __shared__ __align__(16) float shifted[];  // SHIFT: w, then b
  __shared__ RowSums red[2];
  const int tpr = 32 * wpr, groups = blockDim.x / tpr, group = threadIdx.x / tpr, tid = threadIdx.x - group * tpr;
  const int dim = (int)p.dim;
  const float inv = 1.f / (float)dim;
  const Pieces pc = pieces_of<SHIFT>(period, pad0, p.dim);
  const int per = pc.period, pad = pc.pad, cols = 8 * NV * tpr;
  // rows cls, cls + per, ..: RB of them at a time from `row`
  const int64_t step = (int64_t)(gridDim.x / per) * groups * RB * per;
  int64_t row = ((int64_t)(blockIdx.x / per) * groups + group) * RB * per + pc.cls;
  if constexpr (SHIFT) {
    shift_w(shifted, p.w, pad, dim, cols);
    shift_w(shifted + cols, p.b, pad, dim, cols);
  }
  Raw8<T> x[RB][NV];
  Raw8<R> a[RES ? RB : 1][NV];
  auto load = [&](int64_t r) {
#pragma unroll
    for (int j = 0; j < RB; ++j) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int i = (k * tpr + tid) * 8 - pad;
        if (r + j * per < p.rows && i < dim) {
          load_piece<T, SHIFT>(x[j][k], p.x, r + j * per, p.rows, i, dim);
          if constexpr (RES) load_piece<R, SHIFT>(a[j][k], p.res, r + j * per, p.rows, i, dim);
        }
      }
    }
  };
  load(row);
  clear(red[0]);
  clear(red[1]);
  __syncthreads();
  // every group of the block takes the same rounds (barriers in row_sums)
  for (int64_t r0 = (int64_t)(blockIdx.x / per) * groups * RB * per + pc.cls; r0 < p.rows; r0 += step, row += step) {
    f2 v[RB][NV][4];
    float sum[RB], sq[RB];
#pragma unroll
    for (int j = 0; j < RB; ++j) {
      f2 t = splat2(0.f);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int i = (k * tpr + tid) * 8 - pad;
        if (row + j * per >= p.rows || i >= dim) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[j][k][e] = pair_of<T>(x[j][k], e);
        if constexpr (RES) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[j][k][e] = add2(v[j][k][e], pair_of<R>(a[j][k], e));
            if constexpr (sizeof(R) == 2) v[j][k][e] = stored_bf16(v[j][k][e]);
          }
          put_piece<R, SHIFT>(static_cast<R *>(p.res_out) + (row + j * per) * p.dim + i, v[j][k], i, dim);
        }
        keep_own<SHIFT>(v[j][k], i, dim);
        t = add2(t, add2(add2(v[j][k][0], v[j][k][1]), add2(v[j][k][2], v[j][k][3])));
      }
      sum[j] = both(t);
    }
    load(row + step);
    row_sums<RB, Q>(sum, wpr, group, red[0]);
#pragma unroll
    for (int j = 0; j < RB; ++j) {
      const f2 m = splat2(-sum[j] * inv);
      f2 t = splat2(0.f);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (row + j * per >= p.rows || (k * tpr + tid) * 8 - pad >= dim) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[j][k][e] = add2(v[j][k][e], m);
        keep_own<SHIFT>(v[j][k], (k * tpr + tid) * 8 - pad, dim);
#pragma unroll
        for (int e = 0; e < 4; ++e) t = fma2(v[j][k][e], v[j][k][e], t);
      }
      sq[j] = both(t);
    }
    row_sums<RB, Q>(sq, wpr, group, red[1]);
#pragma unroll
    for (int j = 0; j < RB; ++j) sq[j] = rsqrtf(fmaf(sq[j], inv, p.eps));
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = (k * tpr + tid) * 8 - pad;
      if (i >= dim) continue;
      f2 w[4], b[4];
      if constexpr (SHIFT) {
        get_w_shared(shifted + i + pad, w);
        get_w_shared(shifted + cols + i + pad, b);
      } else {
        get_w(p.w + i, w);
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = splat2(0.f);
        if (p.b) get_w(p.b + i, b);
      }
#pragma unroll
      for (int j = 0; j < RB; ++j) {
        if (row + j * per >= p.rows) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[j][k][e] = fma2(mul2(v[j][k][e], splat2(sq[j])), w[e], b[e]);
        put_piece<T, SHIFT>(static_cast<T *>(p.y) + (row + j * per) * p.dim + i, v[j][k], i, dim);
      }
    }
  }
}

// Rows without such accesses: NV single columns per thread, a warp's 32 lanes side by side;
// otherwise as above, one row at a time.
template <typename T, typename R, bool RES, int NV, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) k_norm_elems(NormParams p, int wpr) {
  __shared__ RowSums red[2];
  const int tpr = 32 * wpr, groups = blockDim.x / tpr, group = threadIdx.x / tpr, tid = threadIdx.x - group * tpr;
  const int dim = (int)p.dim;
  const float inv = 1.f / (float)dim;
  const int64_t step = (int64_t)gridDim.x * groups;
  int64_t row = (int64_t)blockIdx.x * groups + group;
  T x[NV];
  R a[RES ? NV : 1];
  auto load = [&](int64_t r) {
    const int64_t base = r * p.dim + tid;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      x[k] = T(0);
      if constexpr (RES) a[k] = R(0);
      if (r < p.rows && k * tpr + tid < dim) {
        x[k] = static_cast<const T *>(p.x)[base + k * tpr];
        if constexpr (RES) a[k] = static_cast<const R *>(p.res)[base + k * tpr];
      }
    }
  };
  load(row);
  clear(red[0]);
  clear(red[1]);
  __syncthreads();
  for (int64_t r0 = (int64_t)blockIdx.x * groups; r0 < p.rows; r0 += step, row += step) {
    const bool live = row < p.rows;
    const int64_t base = row * p.dim + tid;
    float v[NV], sum[1] = {0.f}, sq[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      v[k] = IO<T>::get(&x[k], 0);
      if constexpr (RES) {
        v[k] = stored<R>(v[k] + IO<R>::get(&a[k], 0));
        if (live && k * tpr + tid < dim) IO<R>::store1(static_cast<R *>(p.res_out), base + k * tpr, v[k]);
      }
      sum[0] += v[k];
    }
    load(row + step);
    row_sums<1>(sum, wpr, group, red[0]);
    const float m = sum[0] * inv;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      v[k] -= m;
      if (k * tpr + tid < dim) sq[0] = fmaf(v[k], v[k], sq[0]);
    }
    row_sums<1>(sq, wpr, group, red[1]);
    const float r = rsqrtf(fmaf(sq[0], inv, p.eps));
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = k * tpr + tid;
      if (live && i < dim)
        IO<T>::store1(static_cast<T *>(p.y), base + k * tpr, fmaf(v[k] * r, __ldg(p.w + i), p.b ? __ldg(p.b + i) : 0.f));
    }
  }
}

constexpr int kWideThreads = 512;

// rows wider than the registers: three walks over the row, the later ones from L2
template <typename T, typename R, int VEC>
__global__ void __launch_bounds__(kWideThreads) k_norm_wide(NormParams p) {
  __shared__ RowSums red[2];
  const int64_t base = (int64_t)blockIdx.x * p.dim;
  const T *x = static_cast<const T *>(p.x) + base;
  const R *res = static_cast<const R *>(p.res);
  R *ro = static_cast<R *>(p.res_out) + base;
  T *y = static_cast<T *>(p.y) + base;
  const int64_t i0 = (int64_t)threadIdx.x * VEC, step = (int64_t)kWideThreads * VEC;
  clear(red[0]);
  clear(red[1]);
  __syncthreads();
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
  row_sums<1>(sum, kWideThreads / 32, 0, red[0]);
  const float m = sum[0] / (float)p.dim;
  for (int64_t i = i0; i < p.dim; i += step) {
    at(i);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float c = v[e] - m;
      sq[0] = fmaf(c, c, sq[0]);
    }
  }
  row_sums<1>(sq, kWideThreads / 32, 0, red[1]);
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
// Blocks walk the rows, wpr warps a row, each thread on the same columns of every row,
// whose dw and db it sums in registers.  The block's sums go to the workspace and k_norm_sum
// adds them in a fixed order.  Rows column by column (all those of fewer than 8 columns):
// w dy is rounded once and the same wherever it is used (no contraction into the sums), so
// that a row whose terms cancel, such as one of a single column, cancels exactly.
__device__ __forceinline__ void grad_terms(float c, float g, float w, float (&s3)[3]) {
  const float wd = __fmul_rn(w, g);
  s3[0] = fmaf(c, c, s3[0]);
  s3[1] = fmaf(wd, c, s3[1]);
  s3[2] += wd;
}

// the sums of a block's rows (rpb of them at a time) of one column each, to `out` by the
// first row's threads
__device__ __forceinline__ void block_part(float *acc, float v, int tpr, int rpb, float *out, bool in) {
  if (rpb > 1) {
    __syncthreads();
    acc[threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.x >= tpr) return;
    v = 0.f;
    for (int j = 0; j < rpb; ++j) v += acc[j * tpr + threadIdx.x];
  }
  if (in) *out = v;
}

template <typename T, typename R, bool DRO, int NV, int Q, int MAXT, int MINB, bool SHIFT>
__global__ void __launch_bounds__(MAXT, MINB) k_norm_bwd_rows(NormBwdParams p, int wpr, int period, int pad0) {
  extern __shared__ __align__(16) float shifted[];  // SHIFT: w
  __shared__ RowSums red[2];
  __shared__ float acc[MAXT];
  const int tpr = 32 * wpr, groups = blockDim.x / tpr, group = threadIdx.x / tpr, tid = threadIdx.x - group * tpr;
  const int dim = (int)p.dim;
  const float inv = 1.f / (float)dim;
  const Pieces pc = pieces_of<SHIFT>(period, pad0, p.dim);
  const int per = pc.period, pad = pc.pad;
  const int64_t step = (int64_t)(gridDim.x / per) * groups * per;
  int64_t row = ((int64_t)(blockIdx.x / per) * groups + group) * per + pc.cls;
  if constexpr (SHIFT) shift_w(shifted, p.w, pad, dim, 8 * NV * tpr);
  Raw8<R> s[NV], dro[DRO ? NV : 1];
  Raw8<T> d[NV];
  auto load = [&](int64_t r) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = (k * tpr + tid) * 8 - pad;
      if (r < p.rows && i < dim) {
        load_piece<R, SHIFT>(s[k], p.s, r, p.rows, i, dim);
        load_piece<T, SHIFT>(d[k], p.dy, r, p.rows, i, dim);
        if constexpr (DRO) load_piece<R, SHIFT>(dro[k], p.dres_out, r, p.rows, i, dim);
      }
    }
  };
  load(row);
  f2 dw[NV][4], db[NV][4];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
#pragma unroll
    for (int e = 0; e < 4; ++e) dw[k][e] = db[k][e] = splat2(0.f);
  }
  clear(red[0]);
  clear(red[1]);
  __syncthreads();
  for (int64_t r0 = (int64_t)(blockIdx.x / per) * groups * per + pc.cls; r0 < p.rows; r0 += step, row += step) {
    const bool live = row < p.rows;
    f2 c[NV][4], t = splat2(0.f);
    Raw8<T> g[NV];
    Raw8<R> o[DRO ? NV : 1];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = (k * tpr + tid) * 8 - pad;
      if (!live || i >= dim) continue;
      if constexpr (DRO) o[k] = dro[k];
      g[k] = d[k];
#pragma unroll
      for (int e = 0; e < 4; ++e) c[k][e] = pair_of<R>(s[k], e);
      keep_own<SHIFT>(c[k], i, dim);
      if (SHIFT && !whole(i, dim)) drop_others<T>(g[k], i, dim);
      t = add2(t, add2(add2(c[k][0], c[k][1]), add2(c[k][2], c[k][3])));
    }
    load(row + step);
    float sum[1] = {both(t)};
    row_sums<1, Q>(sum, wpr, group, red[0]);
    const f2 m = splat2(-sum[0] * inv);
    f2 a0 = splat2(0.f), a1 = splat2(0.f), a2 = splat2(0.f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = (k * tpr + tid) * 8 - pad;
      if (!live || i >= dim) continue;
      f2 w[4];
      if constexpr (SHIFT) get_w_shared(shifted + i + pad, w);
      else get_w(p.w + i, w);
#pragma unroll
      for (int e = 0; e < 4; ++e) c[k][e] = add2(c[k][e], m);
      keep_own<SHIFT>(c[k], i, dim);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f2 wd = mul2(w[e], pair_of<T>(g[k], e));
        a0 = fma2(c[k][e], c[k][e], a0);
        a1 = fma2(wd, c[k][e], a1);
        a2 = add2(a2, wd);
      }
    }
    float s3[3] = {both(a0), both(a1), both(a2)};
    row_sums<3, Q>(s3, wpr, group, red[1]);
    const float r = rsqrtf(fmaf(s3[0], inv, p.eps));
    const f2 r2 = splat2(r), k1 = splat2(-(s3[1] * inv * r)), k2 = splat2(-(s3[2] * inv));
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = (k * tpr + tid) * 8 - pad;
      if (!live || i >= dim) continue;
      f2 w[4], v[4];
      if constexpr (SHIFT) get_w_shared(shifted + i + pad, w);
      else get_w(p.w + i, w);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f2 q = mul2(c[k][e], r2), gd = pair_of<T>(g[k], e);
        dw[k][e] = fma2(gd, q, dw[k][e]);
        db[k][e] = add2(db[k][e], gd);
        const f2 ds = fma2(q, k1, add2(mul2(w[e], gd), k2));
        if constexpr (DRO) v[e] = fma2(r2, ds, pair_of<R>(o[k], e));
        else v[e] = mul2(r2, ds);
      }
      put_piece<T, SHIFT>(static_cast<T *>(p.dx) + row * p.dim + i, v, i, dim);
      if constexpr (sizeof(R) != sizeof(T)) put_piece<R, SHIFT>(static_cast<R *>(p.dres) + row * p.dim + i, v, i, dim);
    }
  }
  float *part = p.part + (int64_t)blockIdx.x * 2 * p.dim;  // [block][2][dim]
#pragma unroll
  for (int k = 0; k < NV; ++k) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = (k * tpr + tid) * 8 - pad + 2 * e;
      float v[4];
      unpack2(dw[k][e], v[0], v[1]);
      unpack2(db[k][e], v[2], v[3]);
#pragma unroll
      for (int h = 0; h < 4; ++h)
        block_part(acc, v[h], tpr, groups, part + (h >> 1) * p.dim + i + (h & 1),
                        i + (h & 1) >= 0 && i + (h & 1) < dim);
    }
  }
}

// rows without 16-byte accesses: NV single columns per thread
template <typename T, typename R, bool DRO, int NV, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) k_norm_bwd_elems(NormBwdParams p, int wpr) {
  __shared__ RowSums red[2];
  __shared__ float acc[MAXT];
  const int tpr = 32 * wpr, groups = blockDim.x / tpr, group = threadIdx.x / tpr, tid = threadIdx.x - group * tpr;
  const int dim = (int)p.dim;
  const float inv = 1.f / (float)dim;
  const int64_t step = (int64_t)gridDim.x * groups;
  int64_t row = (int64_t)blockIdx.x * groups + group;
  R s[NV];
  T d[NV];
  auto load = [&](int64_t r) {
    const int64_t base = r * p.dim + tid;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      s[k] = R(0);
      d[k] = T(0);
      if (r < p.rows && k * tpr + tid < dim) {
        s[k] = static_cast<const R *>(p.s)[base + k * tpr];
        d[k] = static_cast<const T *>(p.dy)[base + k * tpr];
      }
    }
  };
  load(row);
  float dw[NV], db[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) dw[k] = db[k] = 0.f;
  clear(red[0]);
  clear(red[1]);
  __syncthreads();
  for (int64_t r0 = (int64_t)blockIdx.x * groups; r0 < p.rows; r0 += step, row += step) {
    const bool live = row < p.rows;
    const int64_t base = row * p.dim + tid;
    float c[NV], g[NV], sum[1] = {0.f}, s3[3] = {0.f, 0.f, 0.f};
    R o[DRO ? NV : 1];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if constexpr (DRO) {
        o[k] = R(0);
        if (live && k * tpr + tid < dim) o[k] = static_cast<const R *>(p.dres_out)[base + k * tpr];
      }
      c[k] = IO<R>::get(&s[k], 0);
      g[k] = IO<T>::get(&d[k], 0);
      sum[0] += c[k];
    }
    load(row + step);
    row_sums<1>(sum, wpr, group, red[0]);
    const float m = sum[0] * inv;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = k * tpr + tid;
      c[k] -= m;
      if (i < dim) grad_terms(c[k], g[k], __ldg(p.w + i), s3);
    }
    row_sums<3>(s3, wpr, group, red[1]);
    const float r = rsqrtf(fmaf(s3[0], inv, p.eps)), k1 = s3[1] * inv * r, k2 = s3[2] * inv;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = k * tpr + tid;
      if (!live || i >= dim) continue;
      const float q = c[k] * r, wd = __fmul_rn(__ldg(p.w + i), g[k]);
      dw[k] = fmaf(g[k], q, dw[k]);
      db[k] += g[k];
      float v = DRO ? IO<R>::get(&o[k], 0) : 0.f;
      v = fmaf(r, fmaf(q, -k1, wd - k2), v);
      IO<T>::store1(static_cast<T *>(p.dx), base + k * tpr, v);
      if constexpr (sizeof(R) != sizeof(T)) IO<R>::store1(static_cast<R *>(p.dres), base + k * tpr, v);
    }
  }
  float *part = p.part + (int64_t)blockIdx.x * 2 * p.dim;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = k * tpr + tid;
    block_part(acc, dw[k], tpr, groups, part + i, i < dim);
    block_part(acc, db[k], tpr, groups, part + p.dim + i, i < dim);
  }
}

// wide rows: ds by walks over the row (one block each), mean and r kept for the columns
template <typename T, typename R, int VEC>
__global__ void __launch_bounds__(kWideThreads) k_norm_bwd_wide(NormBwdParams p, float2 *stats) {
  __shared__ RowSums red[2];
  const int64_t base = (int64_t)blockIdx.x * p.dim;
  const R *s = static_cast<const R *>(p.s) + base;
  const T *dy = static_cast<const T *>(p.dy) + base;
  const int64_t i0 = (int64_t)threadIdx.x * VEC, step = (int64_t)kWideThreads * VEC;
  clear(red[0]);
  clear(red[1]);
  __syncthreads();
  const float n = (float)p.dim;
  float sum[1] = {0.f}, s3[3] = {0.f, 0.f, 0.f}, c[VEC], g[VEC], w[VEC], o[VEC];
  for (int64_t i = i0; i < p.dim; i += step) {
    load_again<R, VEC>(s, i, c);
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum[0] += c[e];
  }
  row_sums<1>(sum, kWideThreads / 32, 0, red[0]);
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
  row_sums<3>(s3, kWideThreads / 32, 0, red[1]);
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

constexpr int kWidest = 16384;     // columns that 16 warps hold at 32 values a thread
constexpr int kWidestBwd = 8192;   // backward, 16 values a thread beside their sums

// How rows are cut into pieces of 8 values: aligned (period 0), or moved.  The tensors of a
// call have to be off by the same number of values.
struct Cut {
  bool ok;
  int period, pad;
};
Cut cut_of(int64_t dim, std::initializer_list<std::pair<const void *, size_t>> tensors) {
  int pad = -1;
  for (const auto &t : tensors) {
    if (!t.first) continue;
    const int q = (int)(reinterpret_cast<uintptr_t>(t.first) / t.second % 8);
    if (pad >= 0 && q != pad) return {false, 0, 0};
    pad = q;
  }
  if (pad == 0 && dim % 8 == 0) return {true, 0, 0};
  if (dim < 8) return {false, 0, 0};  // not one piece: columns one by one
  return {true, dim % 8 == 0 ? 1 : dim % 4 == 0 ? 2 : dim % 2 == 0 ? 4 : 8, pad};
}

// Warps a row and pieces of 8 values a thread: up to 2048 columns 1, 2 or 4 warps (blocks
// of 8 warps hold several rows), above that a block a row, as many warps as 16 values a
// thread need (32 above 8192 columns).
struct RowShape {
  int wpr, nv, threads;
};
RowShape row_shape(int64_t dim, int64_t rows, int sms) {
  RowShape r;
  if (dim <= 2048) {
    r.wpr = dim <= 512 ? 1 : dim <= 1024 ? 2 : 4;
    // few rows: twice the warps, 8 values a thread
    if (dim > 256 && rows * r.wpr < 8 * (int64_t)sms) r.wpr *= 2;
    r.nv = dim > 256 * r.wpr ? 2 : 1;
    r.threads = 256;
  } else {
    r.nv = dim <= 4096 && rows < sms ? 1 : dim <= 8192 ? 2 : 4;
    r.wpr = (int)((dim + 256 * r.nv - 1) / (256 * r.nv));
    r.threads = 32 * r.wpr;
  }
  return r;
}

// a grid of at most `most` blocks for `need`, in whole periods
unsigned grid_of(int64_t need, int64_t most, int period) {
  const int64_t n = std::max<int64_t>(1, std::min(need, most));
  return (unsigned)(period <= 1 ? n : std::max<int64_t>(period, n / period * period));
}

template <typename K>
cudaError_t with_smem(K kern, int smem) {
  return smem > 40 * 1024 ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) : cudaSuccess;
}

// Forward rows that are not aligned go in moved pieces where every tensor is bf16 (5000 x
// 1001 with a residual: 16.6 us, column by column 20.7) and column by column, whose 4-byte
// accesses are full-width already, where one is fp32 (5000 x 4001: 58 us, moved 73).  The
// backward, with more tensors to a column, always goes in moved pieces (85 us against 94).
template <typename T, typename R, bool RES>
constexpr bool kMoved = sizeof(T) == 2 && (!RES || sizeof(R) == 2);

template <typename T, typename R, bool RES, int NV, int RB, int Q, int MAXT, int MINB>
cudaError_t norm_rows(const NormParams &p, const Cut &c, const RowShape &sh, int sms, cudaStream_t s) {
  const int rows = RB * (sh.threads / (32 * sh.wpr));  // a block's at a time
  const int64_t need = (p.rows + rows - 1) / rows, fit = (int64_t)sms * std::max(MINB, MAXT * MINB / sh.threads);
  const unsigned grid = grid_of(need, fit, c.period);
  if (c.period == 0) {
    k_norm_rows<T, R, RES, NV, RB, Q, MAXT, MINB, false><<<grid, sh.threads, 0, s>>>(p, sh.wpr, 0, 0);
  } else if constexpr (kMoved<T, R, RES>) {
    const int smem = 2 * 4 * 256 * NV * sh.wpr;
    auto kern = k_norm_rows<T, R, RES, NV, RB, Q, MAXT, MINB, true>;
    const cudaError_t e = with_smem(kern, smem);
    if (e != cudaSuccess) return e;
    kern<<<grid, sh.threads, smem, s>>>(p, sh.wpr, c.period, c.pad);
  }
  return cudaGetLastError();
}

template <typename T, typename R, bool RES>
cudaError_t norm_vec(const NormParams &p, const Cut &c, int sms, cudaStream_t s) {
  const int64_t dim = p.dim + (c.period ? 7 : 0);  // columns the pieces reach over
  RowShape sh = row_shape(dim, p.rows, sms);
  constexpr int BYTES = (int)sizeof(T) + (RES ? (int)sizeof(R) : 0);
  if constexpr (BYTES <= 2) {
    // bf16 alone is bound by instructions as much as by memory: 32 values a thread, of one
    // row or of several, in blocks of 4 warps (16384 columns: 16).  Measured at 32768 x 4096:
    // 105 us; 109 us with 2 rows of 16 values in blocks of 8 warps, 118 us with one.
    if (p.rows * ((dim + 1023) / 1024) >= 8 * (int64_t)sms) {
      sh.nv = dim <= 256 ? 1 : dim <= 512 ? 2 : 4;
      sh.wpr = (int)((dim + 256 * sh.nv - 1) / (256 * sh.nv));
      sh.threads = sh.wpr == 1 || sh.wpr == 2 ? 128 : 32 * sh.wpr;
      if (sh.nv == 1) return norm_rows<T, R, RES, 1, 4, 1, 128, 4>(p, c, sh, sms, s);
      if (sh.nv == 2) return norm_rows<T, R, RES, 2, 2, 1, 128, 4>(p, c, sh, sms, s);
      if (sh.threads <= 128) return norm_rows<T, R, RES, 4, 1, 1, 128, 4>(p, c, sh, sms, s);
      if (sh.threads <= 256) return norm_rows<T, R, RES, 4, 1, 2, 256, 2>(p, c, sh, sms, s);
      return norm_rows<T, R, RES, 4, 1, 4, 512, 1>(p, c, sh, sms, s);
    }
  }
  // two rows at a time while the next rows' registers (4 a piece in bf16, 8 in fp32) allow
  constexpr int RB = BYTES <= 6 ? 2 : 1;
  if (sh.nv == 1) {
    if (sh.threads <= 256) return norm_rows<T, R, RES, 1, RB, 2, 256, RB == 2 ? 3 : 4>(p, c, sh, sms, s);
    return norm_rows<T, R, RES, 1, 1, 4, 512, 2>(p, c, sh, sms, s);
  }
  if (sh.nv == 2) {
    if (sh.threads <= 256) return norm_rows<T, R, RES, 2, RB, 2, 256, 2>(p, c, sh, sms, s);
    return norm_rows<T, R, RES, 2, 1, 4, 512, 1>(p, c, sh, sms, s);
  }
  return norm_rows<T, R, RES, 4, 1, 4, 512, 1>(p, c, sh, sms, s);
}

// Columns one by one: 8 a thread up to 4096 columns, 16 and 32 beyond.
RowShape elem_shape(int64_t dim) {
  RowShape r;
  r.nv = dim <= 4096 ? 8 : dim <= 8192 ? 16 : 32;
  r.wpr = (int)((dim + 32 * r.nv - 1) / (32 * r.nv));
  if (r.wpr <= 4) {  // several rows a block: a power of two of warps each
    while (r.wpr & (r.wpr - 1)) ++r.wpr;
    r.threads = 256;
  } else {
    r.threads = 32 * r.wpr;
  }
  return r;
}

template <typename T, typename R, bool RES, int NV, int MAXT, int MINB>
cudaError_t norm_elems(const NormParams &p, const RowShape &sh, int sms, cudaStream_t s) {
  const int rows = sh.threads / (32 * sh.wpr);
  const int64_t need = (p.rows + rows - 1) / rows, fit = (int64_t)sms * std::max(MINB, MAXT * MINB / sh.threads);
  k_norm_elems<T, R, RES, NV, MAXT, MINB><<<(unsigned)std::min(need, fit), sh.threads, 0, s>>>(p, sh.wpr);
  return cudaGetLastError();
}

template <typename T, typename R, bool RES>
cudaError_t norm_scalar(const NormParams &p, int sms, cudaStream_t s) {
  const RowShape sh = elem_shape(p.dim);
  if (sh.nv == 8)
    return sh.threads <= 256 ? norm_elems<T, R, RES, 8, 256, 5>(p, sh, sms, s) : norm_elems<T, R, RES, 8, 512, 2>(p, sh, sms, s);
  return sh.nv == 16 ? norm_elems<T, R, RES, 16, 512, 1>(p, sh, sms, s) : norm_elems<T, R, RES, 32, 512, 1>(p, sh, sms, s);
}

template <typename T, typename R>
cudaError_t norm_t(const NormParams &p, int sms, cudaStream_t s) {
  const Cut c = cut_of(p.dim, {{p.x, sizeof(T)}, {p.res, sizeof(R)}, {p.y, sizeof(T)}, {p.res_out, sizeof(R)}});
  const bool vec = c.ok && c.period == 0 && a16(p.w) && a16(p.b);
  if (p.dim > kWidest) {
    if (vec) k_norm_wide<T, R, 8><<<(unsigned)p.rows, kWideThreads, 0, s>>>(p);
    else k_norm_wide<T, R, 1><<<(unsigned)p.rows, kWideThreads, 0, s>>>(p);
    return cudaGetLastError();
  }
  const bool moved = c.ok && c.period && p.dim + 7 <= kWidest;
  if (p.res ? vec || (moved && kMoved<T, R, true>) : vec || (moved && kMoved<T, R, false>))
    return p.res ? norm_vec<T, R, true>(p, c, sms, s) : norm_vec<T, R, false>(p, c, sms, s);
  return p.res ? norm_scalar<T, R, true>(p, sms, s) : norm_scalar<T, R, false>(p, sms, s);
}

// blocks of the backward: enough to fill the machine, no more than there are rows
int64_t bwd_blocks_for(int64_t rows, int sms) { return std::max<int64_t>(8, std::min<int64_t>(rows, 3 * (int64_t)sms)); }

cudaError_t norm_parts(const NormBwdParams &p, int64_t blocks, cudaStream_t s) {
  k_norm_sum<<<(unsigned)(((p.db ? 2 : 1) * p.dim + 31) / 32), dim3(32, 32), 0, s>>>(p.part, p.dw, p.db, blocks, p.dim);
  return cudaGetLastError();
}

template <typename T, typename R, bool DRO, int NV, int Q, int MAXT, int MINB>
cudaError_t bwd_rows(const NormBwdParams &p, const Cut &c, const RowShape &sh, int sms, cudaStream_t s) {
  const int groups = sh.threads / (32 * sh.wpr);
  const int64_t fit = std::min<int64_t>((int64_t)sms * std::max(MINB, MAXT * MINB / sh.threads), bwd_blocks_for(p.rows, sms));
  const unsigned grid = grid_of((p.rows + groups - 1) / groups, fit, c.period);
  cudaError_t e;
  if (c.period == 0) {
    k_norm_bwd_rows<T, R, DRO, NV, Q, MAXT, MINB, false><<<grid, sh.threads, 0, s>>>(p, sh.wpr, 0, 0);
  } else {
    const int smem = 4 * 256 * NV * sh.wpr;
    auto kern = k_norm_bwd_rows<T, R, DRO, NV, Q, MAXT, MINB, true>;
    if ((e = with_smem(kern, smem)) != cudaSuccess) return e;
    kern<<<grid, sh.threads, smem, s>>>(p, sh.wpr, c.period, c.pad);
  }
  e = cudaGetLastError();
  return e != cudaSuccess ? e : norm_parts(p, grid, s);
}

template <typename T, typename R, bool DRO>
cudaError_t bwd_vec(const NormBwdParams &p, const Cut &c, int sms, cudaStream_t s) {
  const int64_t dim = p.dim + (c.period ? 7 : 0);
  RowShape sh = row_shape(dim, p.rows, sms);
  // with the residual's gradient on an fp32 stream a third tensor waits in registers: 8
  // values a thread up to 4096 columns (16384 x 4096: 192 us, 261 us with 16)
  constexpr bool WIDE = DRO && sizeof(R) == 4;
  if (WIDE && dim <= 4096) {
    sh.nv = 1;
    sh.wpr = (int)((dim + 255) / 256);
    if (sh.wpr <= 4) {
      while (sh.wpr & (sh.wpr - 1)) ++sh.wpr;
      sh.threads = 256;
    } else {
      sh.threads = 32 * sh.wpr;
    }
  }
  if (sh.nv == 1) {
    if (sh.threads <= 256) return bwd_rows<T, R, DRO, 1, 2, 256, WIDE ? 2 : 3>(p, c, sh, sms, s);
    return bwd_rows<T, R, DRO, 1, 4, 512, 1>(p, c, sh, sms, s);
  }
  if (sh.threads <= 256) return bwd_rows<T, R, DRO, 2, 2, 256, WIDE ? 1 : 2>(p, c, sh, sms, s);
  // Up to 5120 columns 168 registers a thread; more columns take 512 threads at 128, which spill 324 to
  // 436 bytes each (16384 x 5120 bf16 224 us, 16384 x 6144 536 us).
  if constexpr (WIDE) {
    if (sh.threads <= 320) return bwd_rows<T, R, DRO, 2, 4, 320, 1>(p, c, sh, sms, s);
  }
  return bwd_rows<T, R, DRO, 2, 4, 512, 1>(p, c, sh, sms, s);
}

template <typename T, typename R, bool DRO, int NV, int MAXT, int MINB>
cudaError_t bwd_elems(const NormBwdParams &p, const RowShape &sh, int sms, cudaStream_t s) {
  const int groups = sh.threads / (32 * sh.wpr);
  const int64_t fit = (int64_t)sms * std::max(MINB, MAXT * MINB / sh.threads);
  const int64_t blocks = std::min(std::min((p.rows + groups - 1) / groups, fit), bwd_blocks_for(p.rows, sms));
  k_norm_bwd_elems<T, R, DRO, NV, MAXT, MINB><<<(unsigned)blocks, sh.threads, 0, s>>>(p, sh.wpr);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : norm_parts(p, blocks, s);
}

template <typename T, typename R, bool DRO>
cudaError_t bwd_scalar(const NormBwdParams &p, int sms, cudaStream_t s) {
  const RowShape sh = elem_shape(p.dim);
  if (sh.nv == 8)
    return sh.threads <= 256 ? bwd_elems<T, R, DRO, 8, 256, 2>(p, sh, sms, s) : bwd_elems<T, R, DRO, 8, 512, 1>(p, sh, sms, s);
  return bwd_elems<T, R, DRO, 16, 512, 1>(p, sh, sms, s);
}

template <typename T, typename R>
cudaError_t norm_bwd_t(const NormBwdParams &p, int sms, cudaStream_t s) {
  const Cut c = cut_of(p.dim, {{p.s, sizeof(R)}, {p.dy, sizeof(T)}, {p.dres_out, sizeof(R)}, {p.dx, sizeof(T)}, {p.dres, sizeof(R)}});
  const bool vec = c.ok && c.period == 0 && a16(p.w);
  if ((vec && p.dim <= kWidestBwd) || (c.ok && c.period && p.dim + 7 <= kWidestBwd))
    return p.dres_out ? bwd_vec<T, R, true>(p, c, sms, s) : bwd_vec<T, R, false>(p, c, sms, s);
  if (p.dim > kWidestBwd) {
    const int64_t splits = bwd_blocks_for((p.rows + 31) / 32, sms);
    float2 *stats = reinterpret_cast<float2 *>(p.part + splits * 2 * p.dim);
    if (vec) k_norm_bwd_wide<T, R, 8><<<(unsigned)p.rows, kWideThreads, 0, s>>>(p, stats);
    else k_norm_bwd_wide<T, R, 1><<<(unsigned)p.rows, kWideThreads, 0, s>>>(p, stats);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    k_norm_cols<T, R><<<dim3((unsigned)((p.dim + 255) / 256), (unsigned)splits), 256, 0, s>>>(p, stats);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : norm_parts(p, splits, s);
  }
  return p.dres_out ? bwd_scalar<T, R, true>(p, sms, s) : bwd_scalar<T, R, false>(p, sms, s);
}

}  // namespace

cudaError_t launch_norm(int io_dtype, int res_dtype, const NormParams &p, int sms, cudaStream_t s) {
  if (io_dtype == SSM_F32) return norm_t<float, float>(p, sms, s);
  return res_dtype == SSM_F32 ? norm_t<uint16_t, float>(p, sms, s) : norm_t<uint16_t, uint16_t>(p, sms, s);
}

size_t norm_bwd_part_floats(int64_t rows, int64_t dim, int sms) {
  return (size_t)bwd_blocks_for(rows, sms) * 2 * (size_t)dim + (dim > kWidestBwd ? 2 * (size_t)rows : 0);
}

cudaError_t launch_norm_bwd(int io_dtype, int res_dtype, const NormBwdParams &p, int sms, cudaStream_t s) {
  if (io_dtype == SSM_F32) return norm_bwd_t<float, float>(p, sms, s);
  return res_dtype == SSM_F32 ? norm_bwd_t<uint16_t, float>(p, sms, s) : norm_bwd_t<uint16_t, uint16_t>(p, sms, s);
}

}  // namespace ssm
