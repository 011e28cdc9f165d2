// Gated recurrence, channel-major activations [batch][dim][L]: each row (one
// channel of one batch element) is contiguous in time.
//
// Memory bound: 2 bytes a value in bf16 for each of u, f, z, y (forward) and
// u, f, z, dout, du, df, dz (backward), against about 13 and 30 instruction
// slots and 4 and 5 special-function results a value.  A lane takes 32
// contiguous bytes (one whole sector) of each tensor with one load, as pairs
// (t, t + S/2) on which the gates, the two half runs and the output run as f32x2
// operations; the 32 lanes' runs are joined by shuffles.
//
// Two schedules.  k_rows_*: a warp walks its row, one 32-lane pass after
// another, the state in a register; rows shorter than a pass share a warp.
// k_tiles_*: few long rows; eight warps take a tile of eight passes, tiles of a
// row hand their runs on through the workspace.
#include "ssm_gscan.cuh"

namespace ssm {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRowThreads = 128;

template <typename T>
struct Geo {
  static constexpr int S = kGsLaneBytes / (int)sizeof(T);  // steps per lane
  static constexpr int H = S / 2;                          // pairs per lane
  static constexpr int PASS = 32 * S;                      // steps per warp run
  static constexpr int W = kGsLaneBytes / 4;               // words of a lane's chunk
};

// value i of a lane's chunk
template <typename T>
__device__ __forceinline__ float at(const uint32_t *w, int i) {
  if constexpr (sizeof(T) == 2) return (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
  else return __uint_as_float(w[i]);
}
template <typename T>
__device__ __forceinline__ f2 pair_at(const uint32_t *w, int q) {
  return pack2(at<T>(w, q), at<T>(w, q + Geo<T>::H));
}

// the lane's S steps from src, zeros from `rem` on (rem may be negative)
template <typename T>
__device__ __forceinline__ void load_chunk(uint32_t (&w)[8], const T *src, int64_t rem, int vec) {
  constexpr int S = Geo<T>::S;
  if (vec == 2 && rem >= S) {
    asm volatile("ld.global.cs.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(src));
  } else if (vec && rem >= S) {
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const uint4 q = __ldcs(reinterpret_cast<const uint4 *>(src) + v);
      w[4 * v] = q.x; w[4 * v + 1] = q.y; w[4 * v + 2] = q.z; w[4 * v + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0u;
#pragma unroll
    for (int e = 0; e < S; ++e)
      if (e < rem) {
        if constexpr (sizeof(T) == 2) w[e >> 1] |= (uint32_t)src[e] << (16 * (e & 1));
        else w[e] = __float_as_uint(src[e]);
      }
  }
}

// stores the lane's S steps, given as pairs
template <typename T>
__device__ __forceinline__ void store_chunk(T *dst, int64_t rem, int vec, const f2 (&v)[Geo<T>::H]) {
  constexpr int S = Geo<T>::S, H = Geo<T>::H;
  float o[S];
#pragma unroll
  for (int q = 0; q < H; ++q) unpack2(v[q], o[q], o[q + H]);
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 2) w[i] = pack_bf16x2(o[2 * i], o[2 * i + 1]);
    else w[i] = __float_as_uint(o[i]);
  }
  if (vec == 2 && rem >= S) {
    asm volatile("st.global.cs.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else if (vec && rem >= S) {
    __stcs(reinterpret_cast<uint4 *>(dst), make_uint4(w[0], w[1], w[2], w[3]));
    __stcs(reinterpret_cast<uint4 *>(dst) + 1, make_uint4(w[4], w[5], w[6], w[7]));
  } else {
#pragma unroll
    for (int e = 0; e < S; ++e)
      if (e < rem) {
        if constexpr (sizeof(T) == 2) dst[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        else dst[e] = __uint_as_float(w[e]);
      }
  }
}

// bit e: a sequence starts at the lane's step e
template <int S>
__device__ __forceinline__ unsigned load_starts(const uint8_t *src, int64_t rem, int vec) {
  unsigned m = 0;
  if (vec && rem >= S) {
#pragma unroll
    for (int v = 0; v < S / 4; ++v) {
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(src) + v);
      const uint32_t x = ((w & 0x7f7f7f7fu) + 0x7f7f7f7fu) | w;  // bit 7 of every nonzero byte
      m |= (((x >> 7) & 1u) | ((x >> 14) & 2u) | ((x >> 21) & 4u) | ((x >> 28) & 8u)) << (4 * v);
    }
  } else {
#pragma unroll
    for (int e = 0; e < S; ++e)
      if (e < rem && src[e]) m |= 1u << e;
  }
  return m;
}

// ---- forward ----------------------------------------------------------------------
template <typename T, bool Z, bool ST>
struct FwdChunk {
  uint32_t u[8], f[8], z[Z ? 8 : 1];
  unsigned st;
  __device__ __forceinline__ void load(const GsParams &p, int64_t row, int64_t b, int64_t t0) {
    const int64_t rem = p.L - t0, at0 = row * p.L + t0;
    load_chunk<T>(f, static_cast<const T *>(p.f) + at0, rem, p.vec);
    load_chunk<T>(u, static_cast<const T *>(p.u) + at0, rem, p.vec);
    if constexpr (Z) load_chunk<T>(z, static_cast<const T *>(p.z) + at0, rem, p.vec);
    if constexpr (ST) st = load_starts<Geo<T>::S>(p.starts + b * p.L + t0, rem, p.start_vec);
    else st = 0;
  }
};

// -g of the lane's steps; steps past the row's end leave the state alone (g = 0)
template <typename T>
__device__ __forceinline__ void lane_gates(f2 (&ng)[Geo<T>::H], const uint32_t *f, f2 b2, int64_t rem) {
  constexpr int H = Geo<T>::H;
#pragma unroll
  for (int q = 0; q < H; ++q) ng[q] = neg_gate2(pair_at<T>(f, q), b2);
  if (rem < Geo<T>::S) {
#pragma unroll
    for (int q = 0; q < H; ++q) ng[q] = zero_at(ng[q], q >= rem, q + H >= rem);
  }
}

// The lane's two half runs from zero, the steps q and the steps q + H.
struct Halves {
  Run lo, hi;
};
template <typename T, bool TIED, bool ST>
__device__ __forceinline__ Halves lane_run(const f2 (&ng)[Geo<T>::H], const uint32_t *u, unsigned st) {
  constexpr int H = Geo<T>::H;
  f2 A = splat2(1.f), N = splat2(0.f), B = splat2(0.f);
#pragma unroll
  for (int q = 0; q < H; ++q) {
    if constexpr (ST) B = zero_at(B, (st >> q) & 1u, (st >> (q + H)) & 1u);
    B = state_step<TIED>(B, ng[q], pair_at<T>(u, q));
    N = fma2(ng[q], A, N);
    A = fma2(ng[q], A, A);
  }
  if constexpr (ST) {  // a start cuts the run, whatever its later gates hold (NaN times 0)
    const bool lo = (st & ((1u << H) - 1u)) != 0u, hi = (st >> H) != 0u;
    A = put_at(A, lo, hi, 0.f);
    N = put_at(N, lo, hi, -1.f);
  }
  Halves h;
  unpack2(A, h.lo.A, h.hi.A);
  unpack2(N, h.lo.N, h.hi.N);
  unpack2(B, h.lo.B, h.hi.B);
  return h;
}

// Runs of the lanes of a row (W of them, the lane being number sl) joined up to and
// including each lane's own
template <bool ST>
__device__ __forceinline__ void scan_up(Run &r, int sl, int W) {
  for (int o = 1; o < W; o <<= 1) {
    const Run q = {__shfl_up_sync(kAll, r.A, o, W), __shfl_up_sync(kAll, r.N, o, W), __shfl_up_sync(kAll, r.B, o, W)};
    if (sl >= o) r = join<ST>(r, q);
  }
}
// the same from behind: the runs of the lane and of all after it, for the gradient
template <bool ST>
__device__ __forceinline__ void scan_down(Run &r, int sl, int W) {
  for (int o = 1; o < W; o <<= 1) {
    const Run q = {__shfl_down_sync(kAll, r.A, o, W), __shfl_down_sync(kAll, r.N, o, W),
                   __shfl_down_sync(kAll, r.B, o, W)};
    if (sl + o < W) r = join<ST>(r, q);
  }
}
__device__ __forceinline__ Run run_above(const Run &r, int W) {
  return {__shfl_up_sync(kAll, r.A, 1, W), __shfl_up_sync(kAll, r.N, 1, W), __shfl_up_sync(kAll, r.B, 1, W)};
}
__device__ __forceinline__ Run run_below(const Run &r, int W) {
  return {__shfl_down_sync(kAll, r.A, 1, W), __shfl_down_sync(kAll, r.N, 1, W), __shfl_down_sync(kAll, r.B, 1, W)};
}
__device__ __forceinline__ Run run_of(const Run &r, int lane, int W) {
  return {__shfl_sync(kAll, r.A, lane, W), __shfl_sync(kAll, r.N, lane, W), __shfl_sync(kAll, r.B, lane, W)};
}

// the lane's outputs from the state h entering its first half run
template <typename T, bool TIED, bool Z, bool ST>
__device__ __forceinline__ void lane_out(const GsParams &p, int64_t row, int64_t t0, const FwdChunk<T, Z, ST> &c,
                                         const f2 (&ng)[Geo<T>::H], float hin, const Run &lo) {
  constexpr int H = Geo<T>::H;
  if (!p.y) return;
  f2 h = pack2(hin, run_on<ST>(lo, hin)), o[H];
#pragma unroll
  for (int q = 0; q < H; ++q) {
    if constexpr (ST) h = zero_at(h, (c.st >> q) & 1u, (c.st >> (q + H)) & 1u);
    h = state_step<TIED>(h, ng[q], pair_at<T>(c.u, q));
    if constexpr (Z) {
      const f2 z = pair_at<T>(c.z, q);
      o[q] = mul2(h, mul2(z, sigmoid2(z)));
    } else {
      o[q] = h;
    }
  }
  store_chunk<T>(static_cast<T *>(p.y) + row * p.L + t0, p.L - t0, p.vec, o);
}

template <typename T, bool TIED, bool Z, bool ST>
__global__ void __launch_bounds__(kRowThreads) k_rows_fwd(GsParams p, int W) {
  using G = Geo<T>;
  const int lane = threadIdx.x & 31, sl = lane & (W - 1);
  const int64_t warp = ((int64_t)blockIdx.x * kRowThreads + threadIdx.x) >> 5;
  const int64_t rows = p.batch * p.dim;
  int64_t row = warp * (32 / W) + lane / W;
  if (warp * (32 / W) >= rows) return;  // whole warps leave together
  const bool live = row < rows;
  if (!live) row = rows - 1;            // idle lanes read the last row and write nothing
  const int64_t b = row / p.dim, d = row - b * p.dim;
  const f2 b2 = splat2(p.bias ? p.bias[d] * kLog2e : 0.f);
  float carry = p.h0 ? p.h0[row] : 0.f;
  const int64_t chunks = gs_row_chunks(p.L, sizeof(T));
  FwdChunk<T, Z, ST> c;
  c.load(p, row, b, (int64_t)sl * G::S);
  for (int64_t k = 0; k < chunks; ++k) {
    const int64_t t0 = k * G::PASS + (int64_t)sl * G::S, rem = p.L - t0;
    FwdChunk<T, Z, ST> next;
    if (k + 1 < chunks) next.load(p, row, b, t0 + G::PASS);
    if (p.ckpt && k > 0 && lane == 0) p.ckpt[row * chunks + k] = carry;
    f2 ng[G::H];
    lane_gates<T>(ng, c.f, b2, rem);
    const Halves hv = lane_run<T, TIED, ST>(ng, c.u, c.st);
    Run r = join<ST>(hv.hi, hv.lo);
    scan_up<ST>(r, sl, W);
    const Run before = run_above(r, W);
    const float hin = sl == 0 ? carry : run_on<ST>(before, carry);
    carry = run_on<ST>(run_of(r, W - 1, W), carry);
    if (live && rem > 0) lane_out<T, TIED, Z, ST>(p, row, t0, c, ng, hin, hv.lo);
    if (k + 1 < chunks) c = next;
  }
  if (p.last && live && sl == 0) p.last[row] = carry;
}

// ---- look-back over tiles of a row ---------------------------------------------------
// Called by one warp of tile `c` of a row (time index; from behind in the backward)
// with the tile's own run in every lane: publishes it, and returns the state entering the
// tile.  The tiles of a group of kGsRowGroup are joined in the order of their index
// whatever the order they finish in, starting from the state that the last tile of the
// group before published; so the result does not depend on timing.
template <bool ST>
__device__ __forceinline__ float look_back(const GsParams &p, int64_t row, int64_t c, float first, const Run &tile) {
  const int lane = threadIdx.x & 31;
  const int64_t groups = (p.tiles + kGsRowGroup - 1) / kGsRowGroup, g = c / kGsRowGroup;
  const int in = (int)(c - g * kGsRowGroup);
  unsigned long long *runs = p.runs + row * p.tiles;
  unsigned *states = p.states + row * groups;
  const bool last_in_group = in == kGsRowGroup - 1;
  if (lane == 0 && !last_in_group) put_run(runs + c, tile);
  // lane i waits for the run of the group's tile i, lane 31 (never a predecessor's) for the state
  unsigned long long w = 0ull, started = 0;
  unsigned n = 0, v = 0u;
  if (lane < in) {
    while ((w = look64(runs + g * kGsRowGroup + lane)) == 0ull)
      if (!spun(started, n, p.err)) break;
  } else if (lane == 31 && g > 0) {
    while ((v = look32(states + g - 1)) == 0u)
      if (!spun(started, n, p.err)) break;
  }
  __syncwarp();
  Run r = lane < in ? of_words(w) : no_run();
  const float base = __shfl_sync(kAll, of_word(v), 31);
  scan_up<ST>(r, lane, 32);
  const float h = run_on<ST>(run_of(r, 31, 32), g > 0 ? base : first);
  if (lane == 0 && last_in_group) put_state(states + g, run_on<ST>(tile, h));
  return h;
}

constexpr int kTileThreads = 32 * kGsTileWarps;

template <typename T, bool TIED, bool Z, bool ST>
__global__ void __launch_bounds__(kTileThreads) k_tiles_fwd(GsParams p) {
  using G = Geo<T>;
  __shared__ unsigned slot;
  __shared__ Run sr[kGsTileWarps];
  __shared__ float sh[kGsTileWarps];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t rows = p.batch * p.dim;
  const int64_t ticket = take_ticket(p.ticket, &slot);
  const int64_t c = ticket / rows, row = ticket - c * rows;
  const int64_t b = row / p.dim, d = row - b * p.dim;
  const f2 b2 = splat2(p.bias ? p.bias[d] * kLog2e : 0.f);
  const int64_t chunk = c * kGsTileWarps + w, t0 = chunk * G::PASS + (int64_t)lane * G::S, rem = p.L - t0;
  FwdChunk<T, Z, ST> ch;
  ch.load(p, row, b, t0);
  f2 ng[G::H];
  lane_gates<T>(ng, ch.f, b2, rem);
  const Halves hv = lane_run<T, TIED, ST>(ng, ch.u, ch.st);
  Run r = join<ST>(hv.hi, hv.lo);
  scan_up<ST>(r, lane, 32);
  const Run before = run_above(r, 32);
  if (lane == 31) sr[w] = r;
  __syncthreads();
  if (w == 0) {
    Run tile = sr[0];
#pragma unroll
    for (int i = 1; i < kGsTileWarps; ++i) tile = join<ST>(sr[i], tile);
    float h = look_back<ST>(p, row, c, p.h0 ? p.h0[row] : 0.f, tile);
#pragma unroll
    for (int i = 0; i < kGsTileWarps; ++i) {
      if (lane == 0) sh[i] = h;
      h = run_on<ST>(sr[i], h);
    }
    if (lane == 0 && c == p.tiles - 1 && p.last) p.last[row] = h;
  }
  __syncthreads();
  const float hw = sh[w];
  const int64_t chunks = gs_row_chunks(p.L, sizeof(T));
  if (p.ckpt && lane == 0 && chunk > 0 && chunk < chunks) p.ckpt[row * chunks + chunk] = hw;
  if (rem > 0) lane_out<T, TIED, Z, ST>(p, row, t0, ch, ng, lane == 0 ? hw : run_on<ST>(before, hw), hv.lo);
}

// ---- backward ---------------------------------------------------------------------------
// Per lane: -g, d (the gradient reaching h directly) and, from a walk of the states, dz
// (stored at once) and w = (h_{t-1} - u) a g (untied h_{t-1} a g), which leave
// du = g G and df = G w to the walk of the gradient from behind.
template <typename T, bool Z, bool ST>
struct BwdChunk : FwdChunk<T, Z, ST> {
  uint32_t g[8];
  __device__ __forceinline__ void load(const GsParams &p, int64_t row, int64_t b, int64_t t0) {
    FwdChunk<T, Z, ST>::load(p, row, b, t0);
    load_chunk<T>(g, static_cast<const T *>(p.dout) + row * p.L + t0, p.L - t0, p.vec);
  }
};

// d of the lane's steps, and the gradient's half runs from zero
template <typename T, bool Z, bool ST>
__device__ __forceinline__ f2 lane_grad_run(f2 (&dh)[Geo<T>::H], const BwdChunk<T, Z, ST> &c,
                                            const f2 (&ng)[Geo<T>::H]) {
  constexpr int H = Geo<T>::H;
#pragma unroll
  for (int q = 0; q < H; ++q) {
    dh[q] = pair_at<T>(c.g, q);
    if constexpr (Z) {
      const f2 z = pair_at<T>(c.z, q);
      dh[q] = mul2(dh[q], mul2(z, sigmoid2(z)));
    }
  }
  f2 R = splat2(0.f);
#pragma unroll
  for (int q = H - 1; q >= 0; --q) {
    const f2 s = add2(dh[q], R);
    R = fma2(ng[q], s, s);
    if constexpr (ST) R = zero_at(R, (c.st >> q) & 1u, (c.st >> (q + H)) & 1u);
  }
  return R;
}

// the half runs on the gradient: those on the state with R in the place of B
__device__ __forceinline__ Halves grad_halves(const Halves &h, f2 R) {
  Halves g = h;
  unpack2(R, g.lo.B, g.hi.B);
  return g;
}

// The lane's gradients, from the state entering it (hin) and the gradient reaching its
// last step from behind (pin); returns the sum of its df.
template <typename T, bool TIED, bool Z, bool ST>
__device__ __forceinline__ float lane_grads(const GsParams &p, int64_t row, int64_t t0, const BwdChunk<T, Z, ST> &c,
                                            const f2 (&ng)[Geo<T>::H], const f2 (&dh)[Geo<T>::H], f2 b2, float hin,
                                            float pin, const Run &lo, const Run &ghi, bool write) {
  constexpr int H = Geo<T>::H, S = Geo<T>::S;
  const int64_t at0 = row * p.L + t0, rem = p.L - t0;
  f2 wt[H];
  {
    f2 h = pack2(hin, run_on<ST>(lo, hin)), o[H];
#pragma unroll
    for (int q = 0; q < H; ++q) {
      if constexpr (ST) h = zero_at(h, (c.st >> q) & 1u, (c.st >> (q + H)) & 1u);
      const f2 u = pair_at<T>(c.u, q), ag = gate_slope2(pair_at<T>(c.f, q), b2, ng[q]);
      wt[q] = mul2(TIED ? fma2(u, splat2(-1.f), h) : h, ag);
      h = state_step<TIED>(h, ng[q], u);
      if constexpr (Z) {  // dz = dout h s (1 + z (1 - s))
        const f2 z = pair_at<T>(c.z, q), s = sigmoid2(z);
        const f2 k = fma2(z, fma2(s, splat2(-1.f), splat2(1.f)), splat2(1.f));
        o[q] = mul2(mul2(pair_at<T>(c.g, q), h), mul2(s, k));
      }
    }
    if constexpr (Z) {
      if (write) store_chunk<T>(static_cast<T *>(p.dz) + at0, rem, p.vec, o);
    }
  }
  f2 P = pack2(run_on<ST>(ghi, pin), pin), du[H], sum = splat2(0.f);
#pragma unroll
  for (int q = H - 1; q >= 0; --q) {
    const f2 G = add2(dh[q], P);
    du[q] = TIED ? mul2(mul2(G, ng[q]), splat2(-1.f)) : G;
    wt[q] = mul2(G, wt[q]);
    P = fma2(ng[q], G, G);
    if constexpr (ST) P = zero_at(P, (c.st >> q) & 1u, (c.st >> (q + H)) & 1u);
  }
  if (rem < S) {
#pragma unroll
    for (int q = 0; q < H; ++q) wt[q] = zero_at(wt[q], q >= rem, q + H >= rem);
  }
#pragma unroll
  for (int q = 0; q < H; ++q) sum = add2(sum, wt[q]);
  if (write) {
    store_chunk<T>(static_cast<T *>(p.du) + at0, rem, p.vec, du);
    store_chunk<T>(static_cast<T *>(p.df) + at0, rem, p.vec, wt);
  }
  float s0, s1;
  unpack2(sum, s0, s1);
  return s0 + s1;
}

template <typename T, bool TIED, bool Z, bool ST>
__global__ void __launch_bounds__(kRowThreads, 4) k_rows_bwd(GsParams p, int W) {
  using G = Geo<T>;
  const int lane = threadIdx.x & 31, sl = lane & (W - 1);
  const int64_t warp = ((int64_t)blockIdx.x * kRowThreads + threadIdx.x) >> 5;
  const int64_t rows = p.batch * p.dim;
  int64_t row = warp * (32 / W) + lane / W;
  if (warp * (32 / W) >= rows) return;
  const bool live = row < rows;
  if (!live) row = rows - 1;
  const int64_t b = row / p.dim, d = row - b * p.dim;
  const f2 b2 = splat2(p.bias ? p.bias[d] * kLog2e : 0.f);
  float pc = p.dlast ? p.dlast[row] : 0.f, db = 0.f;
  const int64_t chunks = gs_row_chunks(p.L, sizeof(T));
  for (int64_t k = chunks - 1; k >= 0; --k) {
    const int64_t t0 = k * G::PASS + (int64_t)sl * G::S, rem = p.L - t0;
    BwdChunk<T, Z, ST> c;
    c.load(p, row, b, t0);
    const float h0 = k > 0 ? p.ckpt[row * chunks + k] : (p.h0 ? p.h0[row] : 0.f);
    f2 ng[G::H], dh[G::H];
    lane_gates<T>(ng, c.f, b2, rem);
    const Halves hv = lane_run<T, TIED, ST>(ng, c.u, c.st);
    const Halves gv = grad_halves(hv, lane_grad_run<T, Z, ST>(dh, c, ng));
    Run r = join<ST>(hv.hi, hv.lo), g = join<ST>(gv.lo, gv.hi);
    scan_up<ST>(r, sl, W);
    scan_down<ST>(g, sl, W);
    const Run before = run_above(r, W), after = run_below(g, W);
    const float hin = sl == 0 ? h0 : run_on<ST>(before, h0);
    const float pin = sl == W - 1 ? pc : run_on<ST>(after, pc);
    pc = run_on<ST>(run_of(g, 0, W), pc);
    db += lane_grads<T, TIED, Z, ST>(p, row, t0, c, ng, dh, b2, hin, pin, hv.lo, gv.hi, live && rem > 0);
  }
  if (p.dh0 && live && sl == 0) p.dh0[row] = pc;
  if (p.dbias_part) {
    for (int o = 1; o < W; o <<= 1) db += __shfl_xor_sync(kAll, db, o, W);
    if (live && sl == 0) p.dbias_part[row] = db;
  }
}

template <typename T, bool TIED, bool Z, bool ST>
__global__ void __launch_bounds__(kTileThreads, 2) k_tiles_bwd(GsParams p) {
  using G = Geo<T>;
  __shared__ unsigned slot;
  __shared__ Run sr[kGsTileWarps];
  __shared__ float sp[kGsTileWarps], sdb[kGsTileWarps];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t rows = p.batch * p.dim;
  const int64_t ticket = take_ticket(p.ticket, &slot);
  const int64_t cb = ticket / rows, row = ticket - cb * rows, c = p.tiles - 1 - cb;  // from behind
  const int64_t b = row / p.dim, d = row - b * p.dim;
  const f2 b2 = splat2(p.bias ? p.bias[d] * kLog2e : 0.f);
  const int64_t chunks = gs_row_chunks(p.L, sizeof(T));
  const int64_t chunk = c * kGsTileWarps + w, t0 = chunk * G::PASS + (int64_t)lane * G::S, rem = p.L - t0;
  BwdChunk<T, Z, ST> ch;
  ch.load(p, row, b, t0);
  const float h0 = chunk >= chunks ? 0.f : chunk > 0 ? p.ckpt[row * chunks + chunk] : (p.h0 ? p.h0[row] : 0.f);
  f2 ng[G::H], dh[G::H];
  lane_gates<T>(ng, ch.f, b2, rem);
  const Halves hv = lane_run<T, TIED, ST>(ng, ch.u, ch.st);
  const Halves gv = grad_halves(hv, lane_grad_run<T, Z, ST>(dh, ch, ng));
  Run r = join<ST>(hv.hi, hv.lo), g = join<ST>(gv.lo, gv.hi);
  scan_up<ST>(r, lane, 32);
  scan_down<ST>(g, lane, 32);
  const Run before = run_above(r, 32), after = run_below(g, 32);
  const float hin = lane == 0 ? h0 : run_on<ST>(before, h0);
  if (lane == 0) sr[w] = g;
  __syncthreads();
  if (w == 0) {
    Run tile = sr[kGsTileWarps - 1];
#pragma unroll
    for (int i = kGsTileWarps - 2; i >= 0; --i) tile = join<ST>(sr[i], tile);
    float P = look_back<ST>(p, row, cb, p.dlast ? p.dlast[row] : 0.f, tile);
#pragma unroll
    for (int i = kGsTileWarps - 1; i >= 0; --i) {
      if (lane == 0) sp[i] = P;
      P = run_on<ST>(sr[i], P);
    }
    if (lane == 0 && c == 0 && p.dh0) p.dh0[row] = P;
  }
  __syncthreads();
  const float pw = sp[w];
  float db = lane_grads<T, TIED, Z, ST>(p, row, t0, ch, ng, dh, b2, hin, lane == 31 ? pw : run_on<ST>(after, pw),
                                        hv.lo, gv.hi, rem > 0);
  if (p.dbias_part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) db += __shfl_xor_sync(kAll, db, o);
    if (lane == 0) sdb[w] = db;
    __syncthreads();
    if (threadIdx.x == 0) {
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < kGsTileWarps; ++i) t += sdb[i];
      p.dbias_part[(b * p.tiles + c) * p.dim + d] = t;
    }
  }
}

// ---- launches -----------------------------------------------------------------------------
template <typename T, bool TIED, bool Z, bool ST>
cudaError_t launch_t(bool bwd, int path, const GsParams &p, cudaStream_t s) {
  const int64_t rows = p.batch * p.dim;
  if (path == SSM_PATH_LOOKBACK) {
    const int64_t n = rows * p.tiles;
    if (n > 0x7fffffff) return cudaErrorInvalidConfiguration;
    if (bwd) k_tiles_bwd<T, TIED, Z, ST><<<(unsigned)n, kTileThreads, 0, s>>>(p);
    else k_tiles_fwd<T, TIED, Z, ST><<<(unsigned)n, kTileThreads, 0, s>>>(p);
    return cudaGetLastError();
  }
  int W = 32;  // lanes per row: the fewest that hold a short row
  while (W > 1 && (int64_t)(W / 2) * Geo<T>::S >= p.L) W /= 2;
  const int64_t warps = (rows + 32 / W - 1) / (32 / W), blocks = (warps * 32 + kRowThreads - 1) / kRowThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (bwd) k_rows_bwd<T, TIED, Z, ST><<<(unsigned)blocks, kRowThreads, 0, s>>>(p, W);
  else k_rows_fwd<T, TIED, Z, ST><<<(unsigned)blocks, kRowThreads, 0, s>>>(p, W);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_io(bool bwd, int path, const GsParams &p, cudaStream_t s) {
  const int v = (p.untied ? 0 : 4) | (p.z ? 2 : 0) | (p.starts ? 1 : 0);
  switch (v) {
    case 0: return launch_t<T, false, false, false>(bwd, path, p, s);
    case 1: return launch_t<T, false, false, true>(bwd, path, p, s);
    case 2: return launch_t<T, false, true, false>(bwd, path, p, s);
    case 3: return launch_t<T, false, true, true>(bwd, path, p, s);
    case 4: return launch_t<T, true, false, false>(bwd, path, p, s);
    case 5: return launch_t<T, true, false, true>(bwd, path, p, s);
    case 6: return launch_t<T, true, true, false>(bwd, path, p, s);
    default: return launch_t<T, true, true, true>(bwd, path, p, s);
  }
}

}  // namespace

cudaError_t launch_gs_rows_fwd(int io_dtype, int path, const GsParams &p, cudaStream_t s) {
  return io_dtype == SSM_BF16 ? launch_io<uint16_t>(false, path, p, s) : launch_io<float>(false, path, p, s);
}
cudaError_t launch_gs_rows_bwd(int io_dtype, int path, const GsParams &p, cudaStream_t s) {
  return io_dtype == SSM_BF16 ? launch_io<uint16_t>(true, path, p, s) : launch_io<float>(true, path, p, s);
}

}  // namespace ssm
