// Gated recurrence, token-major activations [batch][L][dim]: the channels of one
// token are contiguous, as a projection leaves them.
//
// Memory bound like the channel-major form.  A lane takes a pair of channels, so
// every step is one f32x2 operation and a warp's access to a token is 128 bytes of
// bf16 (256 of fp32); it walks kTokSteps / kTokWarps consecutive steps, held in
// registers.  The warps of a block split a tile of kTokSteps steps of 64 channels and
// join their runs through shared memory; tiles of the same channels hand their runs on
// through the workspace (one tile: no waiting).
#include "ssm_gscan.cuh"

namespace ssm {

namespace {

constexpr int kTokWarps = 8;
constexpr int kTokThreads = 32 * kTokWarps;
constexpr int kTokRun = kTokSteps / kTokWarps;  // steps per warp
static_assert(kTokGroup <= 2 * kTokWarps, "a warp waits for two tiles at most");

// a pair of channels of one token as loaded
template <typename T> struct Raw;
template <> struct Raw<uint16_t> {
  uint32_t v;
  __device__ __forceinline__ f2 get() const { return pack2(bf16_lo(v), bf16_hi(v)); }
};
template <> struct Raw<float> {
  float2 v;
  __device__ __forceinline__ f2 get() const { return pack2(v.x, v.y); }
};

// The lane's channels: neighbours (2l, 2l + 1) where pairs are aligned, else l and
// l + 32, each access a warp-wide run either way.
struct Pair {
  int64_t d0, d1;
  bool in0, in1, vec;
};
__device__ __forceinline__ Pair pair_of(const GsParams &p, int64_t cg, int lane) {
  Pair c;
  c.vec = p.vec != 0;
  c.d0 = cg * kTokChannels + (c.vec ? 2 * lane : lane);
  c.d1 = c.d0 + (c.vec ? 1 : 32);
  c.in0 = c.d0 < p.dim;
  c.in1 = c.d1 < p.dim;
  return c;
}

template <typename T>
__device__ __forceinline__ Raw<T> load_pair(const void *base, int64_t tok, const GsParams &p, const Pair &c, bool in) {
  Raw<T> r;
  const T *q = static_cast<const T *>(base) + tok * p.dim;
  if constexpr (sizeof(T) == 2) {
    r.v = 0u;
    if (c.vec) {
      if (in && c.in0) r.v = __ldcs(reinterpret_cast<const uint32_t *>(q + c.d0));
    } else {
      if (in && c.in0) r.v = q[c.d0];
      if (in && c.in1) r.v |= (uint32_t)q[c.d1] << 16;
    }
  } else {
    r.v = make_float2(0.f, 0.f);
    if (c.vec) {
      if (in && c.in0) r.v = __ldcs(reinterpret_cast<const float2 *>(q + c.d0));
    } else {
      if (in && c.in0) r.v.x = q[c.d0];
      if (in && c.in1) r.v.y = q[c.d1];
    }
  }
  return r;
}

template <typename T>
__device__ __forceinline__ void store_pair(void *base, int64_t tok, const GsParams &p, const Pair &c, bool in, f2 v) {
  T *q = static_cast<T *>(base) + tok * p.dim;
  float a, b;
  unpack2(v, a, b);
  if (!in) return;
  if (c.vec) {
    if (c.in0) {
      if constexpr (sizeof(T) == 2) __stcs(reinterpret_cast<uint32_t *>(q + c.d0), pack_bf16x2(a, b));
      else __stcs(reinterpret_cast<float2 *>(q + c.d0), make_float2(a, b));
    }
  } else {
    if (c.in0) IO<T>::store1(q, c.d0, a);
    if (c.in1) IO<T>::store1(q, c.d1, b);
  }
}

// fp32 values of the lane's channels from a [..][dim] row (0 where absent), and back
__device__ __forceinline__ f2 load_f32(const float *row, const Pair &c) {
  return pack2(row && c.in0 ? row[c.d0] : 0.f, row && c.in1 ? row[c.d1] : 0.f);
}
__device__ __forceinline__ void store_f32(float *row, const Pair &c, f2 v) {
  float a, b;
  unpack2(v, a, b);
  if (c.in0) row[c.d0] = a;
  if (c.in1) row[c.d1] = b;
}

// runs of the lane's two channels
struct Run2 {
  f2 A, N, B;
};
__device__ __forceinline__ void split(const Run2 &r, Run &x, Run &y) {
  unpack2(r.A, x.A, y.A);
  unpack2(r.N, x.N, y.N);
  unpack2(r.B, x.B, y.B);
}
template <bool ST>
__device__ __forceinline__ f2 run_on2(const Run2 &r, f2 v) {
  Run x, y;
  float a, b;
  split(r, x, y);
  unpack2(v, a, b);
  return pack2(run_on<ST>(x, a), run_on<ST>(y, b));
}
template <bool ST>
__device__ __forceinline__ Run2 join2(const Run2 &own, const Run2 &other) {
  Run a, b, c, d;
  split(own, a, b);
  split(other, c, d);
  const Run x = join<ST>(a, c), y = join<ST>(b, d);
  return {pack2(x.A, y.A), pack2(x.N, y.N), pack2(x.B, y.B)};
}

// bit i: a sequence starts at the warp's step i
template <bool ST>
__device__ __forceinline__ unsigned warp_starts(const GsParams &p, int64_t b, int64_t t0, int lane) {
  if constexpr (!ST) return 0u;
  const int64_t t = t0 + lane;
  return __ballot_sync(0xffffffffu, lane < kTokRun && t < p.L && p.starts[b * p.L + t]);
}

// a start cuts the run, whatever its gates hold (NaN times 0)
template <bool ST>
__device__ __forceinline__ void cut_at_start(Run2 &r, unsigned st) {
  if constexpr (ST) {
    if (st) {
      r.A = splat2(0.f);
      r.N = splat2(-1.f);
    }
  }
}

struct TokShared {
  unsigned slot;
  f2 A[kTokWarps][32], N[kTokWarps][32], B[kTokWarps][32];  // the warps' runs
  unsigned long long run[kTokGroup][64];                    // the runs of the group's earlier tiles
  f2 in[32];                                                // the state entering the tile
  f2 other[kTokWarps][32];
  __device__ __forceinline__ Run2 of(int w, int lane) const { return {A[w][lane], N[w][lane], B[w][lane]}; }
};

// Look-back of the whole block (see the channel-major form): `c` is the tile's index in
// the direction of the walk, sm holds the warps' runs in that direction (warp 0 first, or
// last with FROM_BEHIND).  Returns the value entering the warp's own run; `out` receives
// in warp 0 the value leaving the tile.
template <bool ST, bool FROM_BEHIND>
__device__ __forceinline__ f2 tile_in(const GsParams &p, TokShared &sm, int64_t chain, int64_t c, f2 first, int w,
                                      int lane, f2 &out) {
  const int64_t groups = (p.tiles + kTokGroup - 1) / kTokGroup, g = c / kTokGroup;
  const int in = (int)(c - g * kTokGroup);
  unsigned long long *runs = p.runs + chain * p.tiles * kTokChannels;
  unsigned *states = p.states + chain * groups * kTokChannels;
  const bool last = c == p.tiles - 1, last_in_group = in == kTokGroup - 1;
  Run2 tile;
  if (w == 0) {
    tile = sm.of(FROM_BEHIND ? kTokWarps - 1 : 0, lane);
#pragma unroll
    for (int j = 1; j < kTokWarps; ++j) tile = join2<ST>(sm.of(FROM_BEHIND ? kTokWarps - 1 - j : j, lane), tile);
    if (!last && !last_in_group) {
      Run x, y;
      split(tile, x, y);
      put_run(runs + c * kTokChannels + lane, x);
      put_run(runs + c * kTokChannels + 32 + lane, y);
    }
  }
  unsigned long long started = 0;
  unsigned n = 0;
#pragma unroll
  for (int j = w; j < kTokGroup; j += kTokWarps) {
    if (j < in) {
      const unsigned long long *q = runs + (g * kTokGroup + j) * kTokChannels + lane;
      unsigned long long x, y;
      while ((x = look64(q)) == 0ull)
        if (!spun(started, n, p.err)) break;
      while ((y = look64(q + 32)) == 0ull)
        if (!spun(started, n, p.err)) break;
      sm.run[j][lane] = x;
      sm.run[j][32 + lane] = y;
    }
  }
  f2 h = first;
  if (w == 0 && g > 0) {
    const unsigned *q = states + (g - 1) * kTokChannels + lane;
    unsigned x, y;
    while ((x = look32(q)) == 0u)
      if (!spun(started, n, p.err)) break;
    while ((y = look32(q + 32)) == 0u)
      if (!spun(started, n, p.err)) break;
    h = pack2(of_word(x), of_word(y));
  }
  if (in > 0) __syncthreads();
  if (w == 0) {
    float h0, h1;
    unpack2(h, h0, h1);
    for (int j = 0; j < in; ++j) {
      h0 = run_on<ST>(of_words(sm.run[j][lane]), h0);
      h1 = run_on<ST>(of_words(sm.run[j][32 + lane]), h1);
    }
    h = pack2(h0, h1);
    sm.in[lane] = h;
    out = run_on2<ST>(tile, h);
    if (!last && last_in_group) {
      float x, y;
      unpack2(out, x, y);
      put_state(states + g * kTokChannels + lane, x);
      put_state(states + g * kTokChannels + 32 + lane, y);
    }
  }
  __syncthreads();
  h = sm.in[lane];
#pragma unroll
  for (int j = 0; j < kTokWarps - 1; ++j) {
    const int i = FROM_BEHIND ? kTokWarps - 1 - j : j;
    if (FROM_BEHIND ? i <= w : i >= w) break;
    h = run_on2<ST>(sm.of(i, lane), h);
  }
  return h;
}

template <typename T, bool TIED, bool Z, bool ST>
__global__ void __launch_bounds__(kTokThreads) k_tok_fwd(GsParams p) {
  __shared__ TokShared sm;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t cgs = gs_tok_groups(p.dim), chains = p.batch * cgs;
  const int64_t ticket = p.tiles > 1 ? take_ticket(p.ticket, &sm.slot) : blockIdx.x;
  const int64_t c = ticket / chains, chain = ticket - c * chains, b = chain / cgs, cg = chain - b * cgs;
  const Pair ch = pair_of(p, cg, lane);
  const int64_t t0 = c * kTokSteps + w * kTokRun;
  Raw<T> u[kTokRun], f[kTokRun], z[Z ? kTokRun : 1];
#pragma unroll
  for (int i = 0; i < kTokRun; ++i) {
    const int64_t tok = b * p.L + t0 + i;
    const bool in = t0 + i < p.L;
    f[i] = load_pair<T>(p.f, tok, p, ch, in);
    u[i] = load_pair<T>(p.u, tok, p, ch, in);
    if constexpr (Z) z[i] = load_pair<T>(p.z, tok, p, ch, in);
  }
  const unsigned st = warp_starts<ST>(p, b, t0, lane);
  const f2 b2 = mul2(load_f32(p.bias, ch), splat2(kLog2e));
  const f2 first = load_f32(p.h0 ? p.h0 + b * p.dim : nullptr, ch);
  f2 ng[kTokRun];
  Run2 r = {splat2(1.f), splat2(0.f), splat2(0.f)};
#pragma unroll
  for (int i = 0; i < kTokRun; ++i) {
    ng[i] = t0 + i < p.L ? neg_gate2(f[i].get(), b2) : splat2(0.f);  // a step past the end holds the state
    if constexpr (ST) {
      if ((st >> i) & 1u) r.B = splat2(0.f);
    }
    r.B = state_step<TIED>(r.B, ng[i], u[i].get());
    r.N = fma2(ng[i], r.A, r.N);
    r.A = fma2(ng[i], r.A, r.A);
  }
  cut_at_start<ST>(r, st);
  sm.A[w][lane] = r.A;
  sm.N[w][lane] = r.N;
  sm.B[w][lane] = r.B;
  __syncthreads();
  f2 out;
  f2 h = tile_in<ST, false>(p, sm, chain, c, first, w, lane, out);
  if (w == 0) {
    if (p.ckpt) store_f32(p.ckpt + (b * p.tiles + c) * p.dim, ch, h);
    if (p.last && c == p.tiles - 1) store_f32(p.last + b * p.dim, ch, out);
  }
  if (!p.y) return;
#pragma unroll
  for (int i = 0; i < kTokRun; ++i) {
    if constexpr (ST) {
      if ((st >> i) & 1u) h = splat2(0.f);
    }
    h = state_step<TIED>(h, ng[i], u[i].get());
    f2 o = h;
    if constexpr (Z) {
      const f2 zv = z[i].get();
      o = mul2(h, mul2(zv, sigmoid2(zv)));
    }
    store_pair<T>(p.y, b * p.L + t0 + i, p, ch, t0 + i < p.L, o);
  }
}

template <typename T, bool TIED, bool Z, bool ST>
__global__ void __launch_bounds__(kTokThreads, 2) k_tok_bwd(GsParams p) {
  __shared__ TokShared sm;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t cgs = gs_tok_groups(p.dim), chains = p.batch * cgs;
  const int64_t ticket = p.tiles > 1 ? take_ticket(p.ticket, &sm.slot) : blockIdx.x;
  const int64_t cb = ticket / chains, chain = ticket - cb * chains, b = chain / cgs, cg = chain - b * cgs;
  const int64_t c = p.tiles - 1 - cb;  // from behind
  const Pair ch = pair_of(p, cg, lane);
  const int64_t t0 = c * kTokSteps + w * kTokRun;
  Raw<T> u[kTokRun], f[kTokRun], g[kTokRun], z[Z ? kTokRun : 1];
#pragma unroll
  for (int i = 0; i < kTokRun; ++i) {
    const int64_t tok = b * p.L + t0 + i;
    const bool in = t0 + i < p.L;
    f[i] = load_pair<T>(p.f, tok, p, ch, in);
    u[i] = load_pair<T>(p.u, tok, p, ch, in);
    g[i] = load_pair<T>(p.dout, tok, p, ch, in);
    if constexpr (Z) z[i] = load_pair<T>(p.z, tok, p, ch, in);
  }
  const unsigned st = warp_starts<ST>(p, b, t0, lane);
  const f2 b2 = mul2(load_f32(p.bias, ch), splat2(kLog2e));
  const float *hrow = c > 0 ? p.ckpt + (b * p.tiles + c) * p.dim : p.h0 ? p.h0 + b * p.dim : nullptr;
  f2 h = load_f32(hrow, ch);
  const f2 first = load_f32(p.dlast ? p.dlast + b * p.dim : nullptr, ch);
  // the states: runs of the warps before this one, then its own steps.  A and N are
  // shared with the gradient's runs below.
  f2 ng[kTokRun];
  Run2 r = {splat2(1.f), splat2(0.f), splat2(0.f)};
#pragma unroll
  for (int i = 0; i < kTokRun; ++i) {
    ng[i] = t0 + i < p.L ? neg_gate2(f[i].get(), b2) : splat2(0.f);
    if constexpr (ST) {
      if ((st >> i) & 1u) r.B = splat2(0.f);
    }
    r.B = state_step<TIED>(r.B, ng[i], u[i].get());
    r.N = fma2(ng[i], r.A, r.N);
    r.A = fma2(ng[i], r.A, r.A);
  }
  cut_at_start<ST>(r, st);
  // the gradient's run from behind
  f2 R = splat2(0.f), dh[kTokRun];
#pragma unroll
  for (int i = kTokRun - 1; i >= 0; --i) {
    dh[i] = g[i].get();
    if constexpr (Z) {
      const f2 zv = z[i].get();
      dh[i] = mul2(dh[i], mul2(zv, sigmoid2(zv)));
    }
    const f2 s = add2(dh[i], R);
    R = fma2(ng[i], s, s);
    if constexpr (ST) {
      if ((st >> i) & 1u) R = splat2(0.f);
    }
  }
  sm.A[w][lane] = r.A;
  sm.N[w][lane] = r.N;
  sm.B[w][lane] = R;
  sm.other[w][lane] = r.B;
  __syncthreads();
  for (int i = 0; i < w; ++i) h = run_on2<ST>({sm.A[i][lane], sm.N[i][lane], sm.other[i][lane]}, h);
  f2 out;
  f2 P = tile_in<ST, true>(p, sm, chain, cb, first, w, lane, out);
  if (w == 0 && p.dh0 && c == 0) store_f32(p.dh0 + b * p.dim, ch, out);
  f2 wt[kTokRun];
#pragma unroll
  for (int i = 0; i < kTokRun; ++i) {
    if constexpr (ST) {
      if ((st >> i) & 1u) h = splat2(0.f);
    }
    const f2 uv = u[i].get(), ag = gate_slope2(f[i].get(), b2, ng[i]);
    wt[i] = mul2(TIED ? fma2(uv, splat2(-1.f), h) : h, ag);
    h = state_step<TIED>(h, ng[i], uv);
    if constexpr (Z) {  // dz = dout h s (1 + z (1 - s))
      const f2 zv = z[i].get(), s = sigmoid2(zv);
      const f2 k = fma2(zv, fma2(s, splat2(-1.f), splat2(1.f)), splat2(1.f));
      store_pair<T>(p.dz, b * p.L + t0 + i, p, ch, t0 + i < p.L, mul2(mul2(g[i].get(), h), mul2(s, k)));
    }
  }
  f2 sum = splat2(0.f);
#pragma unroll
  for (int i = kTokRun - 1; i >= 0; --i) {
    const bool in = t0 + i < p.L;
    const f2 G = add2(dh[i], P), df = mul2(G, wt[i]);
    store_pair<T>(p.du, b * p.L + t0 + i, p, ch, in, TIED ? mul2(mul2(G, ng[i]), splat2(-1.f)) : G);
    store_pair<T>(p.df, b * p.L + t0 + i, p, ch, in, df);
    if (in) sum = add2(sum, df);
    P = fma2(ng[i], G, G);
    if constexpr (ST) {
      if ((st >> i) & 1u) P = splat2(0.f);
    }
  }
  if (p.dbias_part) {
    __syncthreads();  // every warp has read the states' runs
    sm.other[w][lane] = sum;
    __syncthreads();
    if (w == 0) {
      f2 t = splat2(0.f);
#pragma unroll
      for (int i = 0; i < kTokWarps; ++i) t = add2(t, sm.other[i][lane]);
      store_f32(p.dbias_part + (b * p.tiles + c) * p.dim, ch, t);
    }
  }
}

template <typename T, bool TIED, bool Z, bool ST>
cudaError_t launch_t(bool bwd, const GsParams &p, cudaStream_t s) {
  const int64_t n = p.batch * gs_tok_groups(p.dim) * p.tiles;
  if (n > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (bwd) k_tok_bwd<T, TIED, Z, ST><<<(unsigned)n, kTokThreads, 0, s>>>(p);
  else k_tok_fwd<T, TIED, Z, ST><<<(unsigned)n, kTokThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_io(bool bwd, const GsParams &p, cudaStream_t s) {
  const int v = (p.untied ? 0 : 4) | (p.z ? 2 : 0) | (p.starts ? 1 : 0);
  switch (v) {
    case 0: return launch_t<T, false, false, false>(bwd, p, s);
    case 1: return launch_t<T, false, false, true>(bwd, p, s);
    case 2: return launch_t<T, false, true, false>(bwd, p, s);
    case 3: return launch_t<T, false, true, true>(bwd, p, s);
    case 4: return launch_t<T, true, false, false>(bwd, p, s);
    case 5: return launch_t<T, true, false, true>(bwd, p, s);
    case 6: return launch_t<T, true, true, false>(bwd, p, s);
    default: return launch_t<T, true, true, true>(bwd, p, s);
  }
}

}  // namespace

cudaError_t launch_gs_tok_fwd(int io_dtype, const GsParams &p, cudaStream_t s) {
  return io_dtype == SSM_BF16 ? launch_io<uint16_t>(false, p, s) : launch_io<float>(false, p, s);
}
cudaError_t launch_gs_tok_bwd(int io_dtype, const GsParams &p, cudaStream_t s) {
  return io_dtype == SSM_BF16 ? launch_io<uint16_t>(true, p, s) : launch_io<float>(true, p, s);
}

}  // namespace ssm
