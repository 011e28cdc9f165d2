// Gated recurrence, channel-major activations [batch][dim][L]: each row (one
// channel of one batch element) is contiguous in time.
//
// Memory bound: 2 bytes a value in bf16 for each of u, f, z, y (forward) and
// u, f, z, dout, du, df, dz (backward), against 4 special-function results a value (2 for the gate, 2
// for SiLU's sigmoid), 6 in the backward's tiles, whose two walks form the sigmoid each for themselves.
// A warp copies its next steps into shared memory ahead (cp.async: 16-byte pieces, or 4-byte
// words or elements where the tensors themselves are not aligned, always a contiguous run a
// warp), reads
// 32 bytes a lane from there (a run of 16 bf16 or 8 fp32 steps), as pairs (t, t + S/2) on
// which the gates, the two half runs and the output run as f32x2 operations; the 32 lanes'
// runs are joined by shuffles.  Rows that are not whole 16-byte pieces (CUT) are cut at the
// aligned places: the first chunk begins a few steps before its row, and steps outside the
// row have gate 0 and are not stored.  Measured forward + backward, 2 x 5120 x 4001 bf16: 82
// + 164 us, and 144 + 311 us from tensors off a 4-byte boundary, which go by elements; 2 x 1536 x 3001
// fp32: 32 + 64 us, 45 + 79 us by 4-byte words.  A variant of its own, as aligned rows lose 10 % to
// the extra tests.
//
// Two schedules.  k_rows_*: a warp walks its row, one 32-lane pass after another, the state
// in a register; rows shorter than a pass share a warp.  k_tiles_*: few long rows; the eight
// warps of a block take a tile of eight passes, the tiles of a row hand their runs on through
// the workspace.
#include "ssm_gscan.cuh"

#include <algorithm>

namespace ssm {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRowThreads = 128;

template <typename T>
struct Geo {
  static constexpr int S = kGsLaneBytes / (int)sizeof(T);  // steps per lane
  static constexpr int H = S / 2;                          // pairs per lane
  static constexpr int PASS = 32 * S;                      // steps per warp run
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

// ---- a warp's piece of one tensor in shared memory: 32 chunks of 32 bytes -------------
// The two 16-byte units of a chunk change places in every other group of four lanes, so that
// eight lanes reading their first (or second) units meet eight different bank groups.
constexpr int kSlot = 1024;
__device__ __forceinline__ uint32_t unit_at(int lane, int h) { return 16 * (2 * lane + (h ^ ((lane >> 2) & 1))); }
// byte offset of word w (0..7) of a lane's chunk
__device__ __forceinline__ uint32_t word_at(int lane, int w) { return unit_at(lane, w >> 2) + 4 * (w & 3); }

// Which lanes share the row: W of them from lane `base`, this one being number sl.
struct Lanes {
  int W, base, sl;
};

// Copies the row's steps [t, t + W * S) (those below L; zeros beyond) to the group's chunks;
// a negative t begins in the row before.  The row's chunks begin `early` steps before it, at
// an aligned place.  mode 2: 16-byte pieces, 1: 4-byte words, 0: elements (not asynchronous).
template <typename T, bool CUT>
__device__ __forceinline__ void fill_slot(unsigned char *slot, const T *row, int64_t t, int64_t L, int early, int mode,
                                          const Lanes &g) {
  const uint32_t s = (uint32_t)__cvta_generic_to_shared(slot);
  const int n = (int)(L - t < g.W * Geo<T>::S ? L - t : g.W * Geo<T>::S);  // steps there are
  const T *src = row + t;
  if (mode == 2) {
    constexpr int E = 16 / (int)sizeof(T);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int u = j * g.W + g.sl;
      // of a piece that the row's end cuts, the row's part
      const int m = CUT ? min(max(n - u * E, 0), E) : u * E < n ? E : 0;
      copy16(s + unit_at(g.base + (u >> 1), u & 1), m ? src + u * E : row - early, (uint32_t)(m * (int)sizeof(T)));
    }
  } else if (mode == 1) {
    constexpr int E = 4 / (int)sizeof(T);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int w = j * g.W + g.sl;
      const bool in = w * E < n;
      copy4(s + word_at(g.base + (w >> 3), w & 7), in ? src + w * E : row, in);
    }
  } else {
    constexpr int S = Geo<T>::S;
    T v[S];
#pragma unroll
    for (int j = 0; j < S; ++j) {
      const int e = j * g.W + g.sl;
      v[j] = e < n ? src[e] : T(0);
    }
#pragma unroll
    for (int j = 0; j < S; ++j) {
      const int e = j * g.W + g.sl, l = e / S, k = e % S;
      *reinterpret_cast<T *>(slot + word_at(g.base + l, k * (int)sizeof(T) / 4) + (k * (int)sizeof(T) & 3)) = v[j];
    }
  }
}

// the lane's chunk
__device__ __forceinline__ void get_chunk(uint32_t (&w)[8], const unsigned char *slot, int lane) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 q = *reinterpret_cast<const uint4 *>(slot + unit_at(lane, h));
    w[4 * h] = q.x; w[4 * h + 1] = q.y; w[4 * h + 2] = q.z; w[4 * h + 3] = q.w;
  }
}

// Stores the group's steps [t, t + W * S) below L from the lanes' pairs.  Unaligned rows go
// through `slot` (whose chunks the lanes have read) so that the warp stores contiguous runs;
// a row's steps are written by its own lanes only, `live` being the same in all of them.
template <typename T, bool CUT>
__device__ __forceinline__ void put_chunk(unsigned char *slot, T *row, int64_t t, int64_t L, int mode, bool v32,
                                          const Lanes &g, const f2 (&v)[Geo<T>::H], bool live) {
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
  if (mode == 2) {
    T *dst = row + t + g.sl * S;
    const int64_t t0 = t + g.sl * S, rem = live ? L - t0 : 0;
    if (CUT && (t0 < 0 || (rem < S && rem % (S / 2)))) {  // cut by the row's start or end: its own steps one by one
      const int lead = t0 < 0 ? (int)-t0 : 0;
#pragma unroll
      for (int e = 0; e < S; ++e)
        if (e >= lead && e < rem) {
          if constexpr (sizeof(T) == 2) dst[e] = (T)(w[e >> 1] >> (16 * (e & 1)));
          else dst[e] = __uint_as_float(w[e]);
        }
      return;
    }
    if (v32 && rem >= S) {
      asm volatile("st.global.cs.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                   "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                   : "memory");
    } else {  // whole 16-byte pieces
      if (rem > 0) __stcs(reinterpret_cast<uint4 *>(dst), make_uint4(w[0], w[1], w[2], w[3]));
      if (rem > S / 2) __stcs(reinterpret_cast<uint4 *>(dst) + 1, make_uint4(w[4], w[5], w[6], w[7]));
    }
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
    *reinterpret_cast<uint4 *>(slot + unit_at(g.base + g.sl, h)) = make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
  __syncwarp();
  const int n = live ? (int)(L - t < g.W * S ? L - t : g.W * S) : 0;
  T *dst = row + t;
  if (mode == 1) {
    constexpr int E = 4 / (int)sizeof(T);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = j * g.W + g.sl;
      if (k * E < n && (!CUT || k * E + t >= 0))
        __stcs(reinterpret_cast<uint32_t *>(dst + k * E), *reinterpret_cast<const uint32_t *>(slot + word_at(g.base + (k >> 3), k & 7)));
    }
  } else {
#pragma unroll
    for (int j = 0; j < S; ++j) {
      const int e = j * g.W + g.sl, l = e / S, k = e % S;
      if (e < n && (!CUT || e + t >= 0))
        dst[e] = *reinterpret_cast<const T *>(slot + word_at(g.base + l, k * (int)sizeof(T) / 4) + (k * (int)sizeof(T) & 3));
    }
  }
}

// bit e: a sequence starts at the lane's step e
template <int S>
__device__ __forceinline__ unsigned load_starts(const uint8_t *src, int64_t rem, int lead, int vec) {
  unsigned m = 0;
  if (vec && rem >= S && lead == 0) {
#pragma unroll
    for (int v = 0; v < S / 4; ++v) {
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(src) + v);
      const uint32_t x = ((w & 0x7f7f7f7fu) + 0x7f7f7f7fu) | w;  // bit 7 of every nonzero byte
      m |= (((x >> 7) & 1u) | ((x >> 14) & 2u) | ((x >> 21) & 4u) | ((x >> 28) & 8u)) << (4 * v);
    }
  } else {
#pragma unroll
    for (int e = 0; e < S; ++e)
      if (e >= lead && e < rem && src[e]) m |= 1u << e;
  }
  return m;
}

// ---- forward ----------------------------------------------------------------------
// Slots of one stage of a warp: f, u, z (forward), f, u, z, dout (backward).
constexpr int kSlotF = 0, kSlotU = kSlot, kSlotZ = 2 * kSlot;
template <bool Z, bool BWD>
constexpr int kStage = kSlot * (2 + (Z ? 1 : 0) + (BWD ? 1 : 0));
template <bool Z>
constexpr int kSlotG = kSlot * (Z ? 3 : 2);

// steps of the row's first chunk that lie before the row
template <bool CUT>
__device__ __forceinline__ int lead_of(const GsParams &p, int64_t row) {
  return CUT ? (int)(row * p.L) & p.cut : 0;
}

// chunks counted from t = 0; they lie lead_of(row) steps earlier
template <typename T, bool Z, bool BWD, bool CUT>
__device__ __forceinline__ void fill_stage(unsigned char *st, const GsParams &p, int64_t row, int64_t t, const Lanes &g) {
  const int64_t at0 = row * p.L;
  const int early = lead_of<CUT>(p, row);
  t -= early;
  fill_slot<T, CUT>(st + kSlotF, static_cast<const T *>(p.f) + at0, t, p.L, early, p.vec, g);
  fill_slot<T, CUT>(st + kSlotU, static_cast<const T *>(p.u) + at0, t, p.L, early, p.vec, g);
  if constexpr (Z) fill_slot<T, CUT>(st + kSlotZ, static_cast<const T *>(p.z) + at0, t, p.L, early, p.vec, g);
  if constexpr (BWD) fill_slot<T, CUT>(st + kSlotG<Z>, static_cast<const T *>(p.dout) + at0, t, p.L, early, p.vec, g);
}

// A chunk's first `lead` steps, which are not the row's, set to zero in every slot of a stage
template <typename T, bool Z, bool BWD>
__device__ __forceinline__ void drop_lead(unsigned char *stage, int lane, int lead) {
  if (lead == 0) return;
  for (int s = 0; s < kStage<Z, BWD>; s += kSlot)
    for (int e = 0; e < lead; ++e)
      *reinterpret_cast<T *>(stage + s + word_at(lane, e * (int)sizeof(T) / 4) + (e * (int)sizeof(T) & 3)) = T(0);
}

// The gates of the lane's steps; steps outside the row leave the state alone.  Returns whether the
// warp has nearly closed ones.
template <typename T>
__device__ __forceinline__ bool lane_gates(f2 (&c)[Geo<T>::H], const unsigned char *st, int lane, f2 b2, int64_t rem,
                                           int lead) {
  constexpr int H = Geo<T>::H;
  uint32_t f[8];
  get_chunk(f, st + kSlotF, lane);
  float least = 1.f;
#pragma unroll
  for (int q = 0; q < H; ++q) c[q] = gate2(pair_at<T>(f, q), b2, least);
  const bool closed = __any_sync(kAll, least < kClosed);
  if (closed) {
#pragma unroll
    for (int q = 0; q < H; ++q) c[q] = signed_gate2(pair_at<T>(f, q), b2);
  }
  if (rem < Geo<T>::S || lead > 0) {
#pragma unroll
    for (int q = 0; q < H; ++q) c[q] = hold_at(c[q], q >= rem || q < lead, q + H >= rem || q + H < lead);
  }
  return closed;
}

// The lane's two half runs from zero, the steps q and the steps q + H; with BWD, R of the
// gradient's from behind, whose d is dh.
struct Halves {
  Run lo, hi;
};
template <typename T, bool TIED, bool ST, bool BWD>
__device__ __forceinline__ Halves lane_run(bool closed, const f2 (&c)[Geo<T>::H], const unsigned char *stage, int lane,
                                           unsigned st, const f2 *dh, f2 &R) {
  constexpr int H = Geo<T>::H;
  uint32_t u[8];
  get_chunk(u, stage + kSlotU, lane);
  f2 A = splat2(1.f), N = splat2(0.f), B = splat2(0.f);
  R = splat2(0.f);
  by_gates(closed, [&](auto kind) {
    constexpr bool C = decltype(kind)::value;
#pragma unroll
    for (int q = 0; q < H; ++q) {
      if constexpr (ST) B = zero_at(B, (st >> q) & 1u, (st >> (q + H)) & 1u);
      B = state_step<TIED, C>(B, c[q], pair_at<T>(u, q));
      run_step<C>(A, N, c[q]);
    }
    if constexpr (BWD) {
#pragma unroll
      for (int q = H - 1; q >= 0; --q) {
        R = grad_step<C>(add2(dh[q], R), c[q]);
        if constexpr (ST) R = zero_at(R, (st >> q) & 1u, (st >> (q + H)) & 1u);
      }
    }
  });
  if constexpr (ST) {  // a start cuts the run, whatever its later gates hold (NaN times 0)
    const bool lo = (st & ((1u << H) - 1u)) != 0u, hi = (st >> H) != 0u;
    A = put_at(A, lo, hi, kStart);
    N = put_at(N, lo, hi, -1.f);
  }
  Halves h;
  unpack2(A, h.lo.A, h.hi.A);
  unpack2(N, h.lo.N, h.hi.N);
  unpack2(B, h.lo.B, h.hi.B);
  h.lo.N = end_run(h.lo.A, h.lo.N);
  h.hi.N = end_run(h.hi.A, h.hi.N);
  return h;
}

// Runs of the lanes of a row (W of them, the lane being number sl) joined up to and
// including each lane's own
template <bool ST>
__device__ __forceinline__ void scan_up(Run &r, int sl, int W) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    if (o >= W) break;  // the same in every lane
    const Run q = {__shfl_up_sync(kAll, r.A, o, W), __shfl_up_sync(kAll, r.N, o, W), __shfl_up_sync(kAll, r.B, o, W)};
    if (sl >= o) r = join<ST>(r, q);
  }
}
// the same from behind: the runs of the lane and of all after it, for the gradient
template <bool ST>
__device__ __forceinline__ void scan_down(Run &r, int sl, int W) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    if (o >= W) break;  // the same in every lane
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

// the lane's outputs from the state entering its first half run
template <typename T, bool TIED, bool Z, bool ST, bool CUT>
__device__ __forceinline__ void lane_out(const GsParams &p, int64_t row, int64_t t, unsigned char *stage, const Lanes &g,
                                         unsigned st, bool closed, const f2 (&c)[Geo<T>::H], float hin, const Run &lo,
                                         bool live) {
  constexpr int H = Geo<T>::H;
  if (!p.y) return;
  const int lane = g.base + g.sl;
  f2 h = pack2(hin, run_on<ST>(lo, hin)), o[H];
  uint32_t u[8], z[8];
  get_chunk(u, stage + kSlotU, lane);
  if constexpr (Z) get_chunk(z, stage + kSlotZ, lane);
  by_gates(closed, [&](auto kind) {
    constexpr bool C = decltype(kind)::value;
#pragma unroll
    for (int q = 0; q < H; ++q) {
      if constexpr (ST) h = zero_at(h, (st >> q) & 1u, (st >> (q + H)) & 1u);
      h = state_step<TIED, C>(h, c[q], pair_at<T>(u, q));
      if constexpr (Z) {
        const f2 zv = pair_at<T>(z, q);
        o[q] = mul2(h, mul2(zv, sigmoid2(zv)));
      } else {
        o[q] = h;
      }
    }
  });
  put_chunk<T, CUT>(stage + kSlotU, static_cast<T *>(p.y) + row * p.L, t, p.L, p.vec, p.v32, g, o, live);
}

// A warp's rows: W lanes each
__device__ __forceinline__ Lanes lanes_of(int W) {
  const int lane = threadIdx.x & 31;
  return {W, lane & ~(W - 1), lane & (W - 1)};
}

constexpr int kRowStages = 3;  // the pass worked on and two on their way

// FULL: 32 lanes a row; otherwise short rows of one chunk a lane, `short_lanes` lanes each.
template <typename T, bool TIED, bool Z, bool ST, bool FULL, bool CUT>
__global__ void __launch_bounds__(kRowThreads, sizeof(T) == 2 ? 5 : 6) k_rows_fwd(GsParams p, int short_lanes) {
  using G = Geo<T>;
  const int W = FULL ? 32 : short_lanes;
  extern __shared__ __align__(16) unsigned char smem[];
  unsigned char *ring = smem + (threadIdx.x >> 5) * kRowStages * kStage<Z, false>;
  const Lanes g = lanes_of(W);
  const int lane = threadIdx.x & 31;
  const int64_t warp = ((int64_t)blockIdx.x * kRowThreads + threadIdx.x) >> 5;
  const int64_t rows = p.batch * p.dim;
  int64_t row = warp * (32 / W) + lane / W;
  if (warp * (32 / W) >= rows) return;  // whole warps leave together
  const bool live = row < rows;
  if (!live) row = rows - 1;            // idle lanes read the last row and write nothing
  const unsigned b = (unsigned)row / (unsigned)p.dim, d = (unsigned)row - b * (unsigned)p.dim;  // the host checks that rows fit
  const int64_t chunks = FULL ? gs_row_chunks(p.L, sizeof(T)) : 1;
  const int early = lead_of<CUT>(p, row);
#pragma unroll
  for (int j = 0; j < kRowStages - 1; ++j) {
    if (j < chunks) fill_stage<T, Z, false, CUT>(ring + j * kStage<Z, false>, p, row, j * (int64_t)G::PASS, g);
    copies_commit();
  }
  const f2 b2 = splat2(p.bias ? p.bias[d] * kLog2e : 0.f);
  float carry = p.h0 ? p.h0[row] : 0.f;
  int at = 0, ahead = kRowStages - 1;
  for (int64_t k = 0; k < chunks; ++k) {
    const int64_t t = k * G::PASS - early, t0 = t + (int64_t)g.sl * G::S, rem = p.L - t0;
    const int lead = CUT && t0 < 0 ? (int)-t0 : 0;
    unsigned char *stage = ring + at * kStage<Z, false>;
    if (k + kRowStages - 1 < chunks)
      fill_stage<T, Z, false, CUT>(ring + ahead * kStage<Z, false>, p, row, (k + kRowStages - 1) * (int64_t)G::PASS, g);
    copies_commit();
    unsigned st = 0;
    if constexpr (ST) st = load_starts<G::S>(p.starts + b * p.L + t0, rem, lead, p.start_vec);
    copies_wait<kRowStages - 1>();
    __syncwarp();
    if (p.ckpt && k > 0 && lane == 0) p.ckpt[row * chunks + k] = carry;
    f2 c[G::H], none;
    drop_lead<T, Z, false>(stage, lane, lead);
    const bool closed = lane_gates<T>(c, stage, lane, b2, rem, lead);
    const Halves hv = lane_run<T, TIED, ST, false>(closed, c, stage, lane, st, nullptr, none);
    Run r = join<ST>(hv.hi, hv.lo);
    scan_up<ST>(r, g.sl, W);
    const Run before = run_above(r, W);
    const float hin = g.sl == 0 ? carry : run_on<ST>(before, carry);
    carry = run_on<ST>(run_of(r, W - 1, W), carry);
    lane_out<T, TIED, Z, ST, CUT>(p, row, t, stage, g, st, closed, c, hin, hv.lo, live);
    __syncwarp();  // every lane is done with the stage before it is filled again
    at = at + 1 == kRowStages ? 0 : at + 1;
    ahead = ahead + 1 == kRowStages ? 0 : ahead + 1;
  }
  if (p.last && live && g.sl == 0) p.last[row] = carry;
}

// ---- look-back over tiles of a row ---------------------------------------------------
// Called by one warp of tile `c` of a row (time index; from behind in the backward)
// with the runs of the tile's warps: publishes the tile's run, and returns the state
// entering it.  The tiles of a group of p.group are joined in the order of their index whatever
// the order they finish in, starting from the state that the last tile of the group before
// published; so the result does not depend on timing.  `w` holds what the lane saw of the
// word it needs when it looked ahead (peek): lane i the run of the group's tile i, lane 31
// (never a predecessor's) the state.
__device__ __forceinline__ const void *look_at(const GsParams &p, int64_t row, unsigned c) {
  const int lane = threadIdx.x & 31;
  const unsigned g = c / p.group, in = c - g * p.group;
  if (lane < in) return p.runs + row * p.tiles + g * p.group + lane;
  if (lane == 31 && g > 0) return p.states + row * p.groups + g - 1;
  return nullptr;
}
__device__ __forceinline__ unsigned long long peek(const void *q) {
  if (!q) return 0ull;
  return (threadIdx.x & 31) == 31 ? look32(static_cast<const unsigned *>(q))
                                  : look64(static_cast<const unsigned long long *>(q));
}
template <bool ST, bool FROM_BEHIND>
__device__ __forceinline__ float look_back(const GsParams &p, int64_t row, unsigned c, float first, const Run *runs,
                                           const void *q, unsigned long long w) {
  const int lane = threadIdx.x & 31;
  const unsigned g = c / p.group, in = c - g * p.group;
  const bool last_in_group = in == p.group - 1;
  Run tile = no_run();
#pragma unroll
  for (int i = 0; i < kGsTileWarps; ++i) tile = join<ST>(runs[FROM_BEHIND ? kGsTileWarps - 1 - i : i], tile);
  // the row's first tile hands on its state in the place of its run, so that no other tile
  // reads the state entering the row (which the last one may overwrite)
  if (c == 0) tile = Run{0.f, -1.f, run_on<ST>(tile, first)};
  if (lane == 0 && !last_in_group) put_run(p.runs + row * p.tiles + c, tile);
  unsigned long long started = 0;
  unsigned n = 0;
  auto wait = [&]() {
    while (w == 0ull) {
      w = peek(q);
      if (w == 0ull && !spun(started, n, p.err)) break;
    }
  };
  // the runs first: they do not wait for anyone's state
  Run r = no_run();
  if (in > 0) {
    if (lane < in) {
      wait();
      r = of_words(w);
    }
    __syncwarp();
    scan_up<ST>(r, lane, 32);
    r = run_of(r, 31, 32);
  }
  float h = first;
  if (g > 0) {
    if (lane == 31) wait();
    __syncwarp();
    h = __shfl_sync(kAll, of_word((unsigned)w), 31);
  }
  if (in > 0) h = run_on<ST>(r, h);
  if (lane == 0 && last_in_group) put_state(p.states + row * p.groups + g, run_on<ST>(tile, h));
  return h;
}

constexpr int kTileThreads = 32 * kGsTileWarps;

// Tickets and runs of this tile and the one before: what is written over lies two tiles back,
// and every warp has passed a barrier since it read it, so one barrier a tile is enough.
struct TileShared {
  Taken ticket[2];
  Run run[2][kGsTileWarps];
  float in[kGsTileWarps], db[kGsTileWarps];
};

// The value entering the warp's own run, after the barrier that shows the warps' runs;
// FROM_BEHIND: the walk starts at the last warp.  `first` enters the row's first tile (0
// in the others); the value leaving the tile is published, and goes to `end` where it leaves the row.  With one
// tile a group every warp reads the state itself and walks the runs before its own; else
// warp 0 looks back for all.  q, seen: as in look_back (one tile a group: in every warp, the
// state of the tile before, in every lane).
template <bool ST, bool FROM_BEHIND>
__device__ __forceinline__ float tile_in(const GsParams &p, TileShared &sm, const Run *runs, int64_t row, unsigned c,
                                         float first, const void *q, unsigned long long seen, float *end) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int mine = FROM_BEHIND ? kGsTileWarps - 1 - w : w;
  auto nth = [](int i) { return FROM_BEHIND ? kGsTileWarps - 1 - i : i; };
  if (p.group == 1) {
    float h = first;
    if (q) {
      unsigned long long started = 0;
      unsigned n = 0, v = (unsigned)seen;
      while (v == 0u) {
        v = look32(static_cast<const unsigned *>(q));
        if (v == 0u && !spun(started, n, p.err)) break;
      }
      h = of_word(v);
    }
#pragma unroll
    for (int i = 0; i < kGsTileWarps - 1; ++i) {
      if (i < mine) h = run_on<ST>(runs[nth(i)], h);
    }
    if (mine == kGsTileWarps - 1 && lane == 0) {
      const float out = run_on<ST>(runs[w], h);
      if (c + 1 < p.tiles) put_state(p.states + row * p.groups + c, out);
      else if (end) end[row] = out;
    }
    return h;
  }
  if (w == 0) {
    float h = look_back<ST, FROM_BEHIND>(p, row, c, first, runs, q, seen);
#pragma unroll
    for (int i = 0; i < kGsTileWarps; ++i) {
      if (lane == 0) sm.in[nth(i)] = h;
      h = run_on<ST>(runs[nth(i)], h);
    }
    if (lane == 0 && c + 1 == p.tiles && end) end[row] = h;
  }
  __syncthreads();
  return sm.in[w];
}
// where a tile's state comes from, and what is seen there ahead
__device__ __forceinline__ const void *tile_look(const GsParams &p, int64_t row, unsigned c, unsigned long long &seen) {
  const void *q = nullptr;
  seen = 0ull;
  if (p.group == 1) {
    if (c > 0) {
      q = p.states + row * p.groups + c - 1;
      seen = look32(static_cast<const unsigned *>(q));
    }
  } else if (threadIdx.x < 32) {
    q = look_at(p, row, c);
    seen = peek(q);
  }
  return q;
}

// Blocks stay and take tile after tile: the next tile's ticket is drawn and its steps are on
// their way while the current one waits for the state entering it.
template <typename T, bool TIED, bool Z, bool ST, bool CUT>
__global__ void __launch_bounds__(kTileThreads, 3) k_tiles_fwd(GsParams p) {
  using G = Geo<T>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ TileShared sm;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  unsigned char *ring = smem + w * 2 * kStage<Z, false>;
  const Lanes lanes = {32, 0, lane};
  const unsigned chains = (unsigned)(p.batch * p.dim), total = chains * (unsigned)p.tiles;
  const int64_t chunks = gs_row_chunks(p.L, sizeof(T));
  const Taken now = first_ticket(p.ticket, sm.ticket[0], chains, (unsigned)p.dim);
  if (now.id >= total) return;
  Place at = now.place;
  fill_stage<T, Z, false, CUT>(ring, p, at.chain, ((int64_t)at.time * kGsTileWarps + w) * G::PASS, lanes);
  copies_commit();
  for (int stg = 0;; stg ^= 1) {
    const int64_t row = at.chain, chunk = (int64_t)at.time * kGsTileWarps + w, t = chunk * G::PASS - lead_of<CUT>(p, row);
    const int64_t t0 = t + lane * G::S, rem = p.L - t0;
    const int lead = CUT && t0 < 0 ? (int)-t0 : 0;
    unsigned char *stage = ring + stg * kStage<Z, false>;
    unsigned drawn = 0;
    if (threadIdx.x == 0) drawn = atomicAdd(p.ticket, 1u);
    unsigned long long seen;
    const void *q = tile_look(p, row, at.time, seen);
    const f2 b2 = splat2(p.bias ? p.bias[at.rest] * kLog2e : 0.f);
    const float first = at.time == 0 && p.h0 ? p.h0[row] : 0.f;
    unsigned st = 0;
    if constexpr (ST) st = load_starts<G::S>(p.starts + at.batch * p.L + t0, rem, lead, p.start_vec);
    copies_wait<0>();
    __syncwarp();
    f2 c[G::H], none;
    drop_lead<T, Z, false>(stage, lane, lead);
    const bool closed = lane_gates<T>(c, stage, lane, b2, rem, lead);
    const Halves hv = lane_run<T, TIED, ST, false>(closed, c, stage, lane, st, nullptr, none);
    Run r = join<ST>(hv.hi, hv.lo);
    scan_up<ST>(r, lane, 32);
    const Run before = run_above(r, 32);
    if (lane == 31) sm.run[stg][w] = r;
    if (threadIdx.x == 0) hand_out(sm.ticket[stg], drawn, chains, (unsigned)p.dim);
    __syncthreads();
    const Taken next = sm.ticket[stg];
    if (next.id < total)
      fill_stage<T, Z, false, CUT>(ring + (stg ^ 1) * kStage<Z, false>, p, next.place.chain,
                              ((int64_t)next.place.time * kGsTileWarps + w) * G::PASS, lanes);
    copies_commit();
    const float hw = tile_in<ST, false>(p, sm, sm.run[stg], row, at.time, first, q, seen, p.last);
    if (p.ckpt && lane == 0 && chunk > 0 && chunk < chunks) p.ckpt[row * chunks + chunk] = hw;
    lane_out<T, TIED, Z, ST, CUT>(p, row, t, stage, lanes, st, closed, c, lane == 0 ? hw : run_on<ST>(before, hw), hv.lo,
                                  t < p.L);
    __syncwarp();
    if (next.id >= total) break;
    at = next.place;
  }
}

// ---- backward ---------------------------------------------------------------------------
// Per lane: the gates, d (the gradient reaching h directly) and, from a walk of the states, dz
// (stored at once) and w, which leaves df to the walk of the gradient from behind.

// d of the lane's steps
template <typename T, bool Z>
__device__ __forceinline__ void lane_direct(f2 (&dh)[Geo<T>::H], const unsigned char *stage, int lane) {
  constexpr int H = Geo<T>::H;
  uint32_t g[8], z[8];
  get_chunk(g, stage + kSlotG<Z>, lane);
  if constexpr (Z) get_chunk(z, stage + kSlotZ, lane);
#pragma unroll
  for (int q = 0; q < H; ++q) {
    dh[q] = pair_at<T>(g, q);
    if constexpr (Z) {
      const f2 zv = pair_at<T>(z, q);
      dh[q] = mul2(dh[q], mul2(zv, sigmoid2(zv)));
    }
  }
}

// the half runs on the gradient: those on the state with R in the place of B
__device__ __forceinline__ Halves grad_halves(const Halves &h, f2 R) {
  Halves g = h;
  unpack2(R, g.lo.B, g.hi.B);
  return g;
}

// The steps of the state and of the gradient with du and df, which is G (h - u) a g (untied
// G h a g): the product of -c (h - u), left in w by the state's step, and of what the gradient's
// makes of G, a G where c is a -g and -g G where it is an a.  The token-major kernel, with twice
// the steps a lane in its registers, forms them otherwise (its form here: 4 x 5120 x 8192 bf16
// backward 513 instead of 472 us).
template <bool TIED>
__device__ __forceinline__ f2 state_step_bwd(f2 h, f2 c, f2 u, f2 &w) {
  const f2 m = open2(c);
  w = mul2(c, TIED ? fma2(h, splat2(-1.f), u) : mul2(h, splat2(-1.f)));
  const f2 to = fma2(w, splat2(-1.f), TIED ? pick2(m, h, u) : h & m);
  return TIED ? to : add2(to, u);
}
template <bool TIED>
__device__ __forceinline__ f2 grad_step_bwd(f2 G, f2 c, f2 w, f2 &du, f2 &df) {
  const f2 m = open2(c), near = G & m, P = fma2(c, G, near), gG = fma2(c, G, fma2(G, splat2(-1.f), near));  // gG: -g G
  df = mul2(w, pick2(m, P, gG));
  du = TIED ? mul2(gG, splat2(-1.f)) : G;
  return P;
}

// The lane's gradients, from the state entering it (hin) and the gradient reaching its
// last step from behind (pin); returns the sum of its df.
template <typename T, bool TIED, bool Z, bool ST, bool CUT>
__device__ __forceinline__ float lane_grads(const GsParams &p, int64_t row, int64_t t, unsigned char *stage,
                                            const Lanes &l, unsigned st, const f2 (&c)[Geo<T>::H],
                                            const f2 (&dh)[Geo<T>::H], float hin, float pin, const Run &lo,
                                            const Run &ghi, bool live) {
  constexpr int H = Geo<T>::H, S = Geo<T>::S;
  const int lane = l.base + l.sl;
  const int64_t at0 = row * p.L, rem = p.L - t - l.sl * S;
  f2 wt[H];
  {
    f2 h = pack2(hin, run_on<ST>(lo, hin)), o[H];
    uint32_t u[8], z[8], g[8];
    get_chunk(u, stage + kSlotU, lane);
    if constexpr (Z) {
      get_chunk(z, stage + kSlotZ, lane);
      get_chunk(g, stage + kSlotG<Z>, lane);
    }
#pragma unroll
    for (int q = 0; q < H; ++q) {
      if constexpr (ST) h = zero_at(h, (st >> q) & 1u, (st >> (q + H)) & 1u);
      h = state_step_bwd<TIED>(h, c[q], pair_at<T>(u, q), wt[q]);
      if constexpr (Z) {  // dz = dout h s (1 + z (1 - s))
        const f2 zv = pair_at<T>(z, q), s = sigmoid2(zv);
        const f2 k = fma2(zv, fma2(s, splat2(-1.f), splat2(1.f)), splat2(1.f));
        o[q] = mul2(mul2(pair_at<T>(g, q), h), mul2(s, k));
      }
    }
    if constexpr (Z) put_chunk<T, CUT>(stage + kSlotZ, static_cast<T *>(p.dz) + at0, t, p.L, p.vec, p.v32, l, o, live);
  }
  f2 P = pack2(run_on<ST>(ghi, pin), pin), du[H], sum = splat2(0.f);
#pragma unroll
  for (int q = H - 1; q >= 0; --q) {
    P = grad_step_bwd<TIED>(add2(dh[q], P), c[q], wt[q], du[q], wt[q]);
    if constexpr (ST) P = zero_at(P, (st >> q) & 1u, (st >> (q + H)) & 1u);
  }
  put_chunk<T, CUT>(stage + kSlotU, static_cast<T *>(p.du) + at0, t, p.L, p.vec, p.v32, l, du, live);
  put_chunk<T, CUT>(stage + kSlotF, static_cast<T *>(p.df) + at0, t, p.L, p.vec, p.v32, l, wt, live);
  const int64_t lead = CUT && l.sl * S + t < 0 ? -(t + l.sl * S) : 0;
  if (rem < S || lead > 0) {
#pragma unroll
    for (int q = 0; q < H; ++q) wt[q] = zero_at(wt[q], q >= rem || q < lead, q + H >= rem || q + H < lead);
  }
#pragma unroll
  for (int q = 0; q < H; ++q) sum = add2(sum, wt[q]);
  float s0, s1;
  unpack2(sum, s0, s1);
  return s0 + s1;
}

constexpr int kRowBwdStages = 2;

template <typename T, bool TIED, bool Z, bool ST, bool FULL, bool CUT>
__global__ void __launch_bounds__(kRowThreads, sizeof(T) == 2 ? 3 : 4) k_rows_bwd(GsParams p, int short_lanes) {
  using G = Geo<T>;
  const int W = FULL ? 32 : short_lanes;
  extern __shared__ __align__(16) unsigned char smem[];
  unsigned char *ring = smem + (threadIdx.x >> 5) * kRowBwdStages * kStage<Z, true>;
  const Lanes l = lanes_of(W);
  const int lane = threadIdx.x & 31;
  const int64_t warp = ((int64_t)blockIdx.x * kRowThreads + threadIdx.x) >> 5;
  const int64_t rows = p.batch * p.dim;
  int64_t row = warp * (32 / W) + lane / W;
  if (warp * (32 / W) >= rows) return;
  const bool live = row < rows;
  if (!live) row = rows - 1;
  const unsigned b = (unsigned)row / (unsigned)p.dim, d = (unsigned)row - b * (unsigned)p.dim;
  const int64_t chunks = FULL ? gs_row_chunks(p.L, sizeof(T)) : 1;
  const int early = lead_of<CUT>(p, row);
  fill_stage<T, Z, true, CUT>(ring, p, row, (chunks - 1) * (int64_t)G::PASS, l);
  copies_commit();
  const f2 b2 = splat2(p.bias ? p.bias[d] * kLog2e : 0.f);
  float pc = p.dlast ? p.dlast[row] : 0.f, db = 0.f;
  int at = 0;
  for (int64_t k = chunks - 1; k >= 0; --k, at ^= 1) {
    const int64_t t = k * G::PASS - early, t0 = t + (int64_t)l.sl * G::S, rem = p.L - t0;
    const int lead = CUT && t0 < 0 ? (int)-t0 : 0;
    unsigned char *stage = ring + at * kStage<Z, true>;
    if (k > 0) fill_stage<T, Z, true, CUT>(ring + (at ^ 1) * kStage<Z, true>, p, row, (k - 1) * (int64_t)G::PASS, l);
    copies_commit();
    const float h0 = k > 0 ? p.ckpt[row * chunks + k] : (p.h0 ? p.h0[row] : 0.f);
    unsigned st = 0;
    if constexpr (ST) st = load_starts<G::S>(p.starts + b * p.L + t0, rem, lead, p.start_vec);
    copies_wait<1>();
    __syncwarp();
    f2 c[G::H], dh[G::H], R;
    drop_lead<T, Z, true>(stage, lane, lead);
    lane_direct<T, Z>(dh, stage, lane);
    const bool closed = lane_gates<T>(c, stage, lane, b2, rem, lead);
    const Halves hv = lane_run<T, TIED, ST, true>(closed, c, stage, lane, st, dh, R), gv = grad_halves(hv, R);
    Run r = join<ST>(hv.hi, hv.lo), g = join<ST>(gv.lo, gv.hi);
    scan_up<ST>(r, l.sl, W);
    scan_down<ST>(g, l.sl, W);
    const Run before = run_above(r, W), after = run_below(g, W);
    const float hin = l.sl == 0 ? h0 : run_on<ST>(before, h0);
    const float pin = l.sl == W - 1 ? pc : run_on<ST>(after, pc);
    pc = run_on<ST>(run_of(g, 0, W), pc);
    db += lane_grads<T, TIED, Z, ST, CUT>(p, row, t, stage, l, st, c, dh, hin, pin, hv.lo, gv.hi, live);
    __syncwarp();  // every lane is done with the stage before it is filled again
  }
  if (p.dh0 && live && l.sl == 0) p.dh0[row] = pc;
  if (p.dbias_part) {
    for (int o = 1; o < W; o <<= 1) db += __shfl_xor_sync(kAll, db, o, W);
    if (live && l.sl == 0) p.dbias_part[row] = db;
  }
}

template <typename T, bool TIED, bool Z, bool ST, bool CUT>
__global__ void __launch_bounds__(kTileThreads, 2) k_tiles_bwd(GsParams p) {
  using G = Geo<T>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ TileShared sm;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  unsigned char *ring = smem + w * 2 * kStage<Z, true>;
  const Lanes lanes = {32, 0, lane};
  const unsigned chains = (unsigned)(p.batch * p.dim), total = chains * (unsigned)p.tiles;
  const int64_t chunks = gs_row_chunks(p.L, sizeof(T));
  // the warp's chunk of a tile taken from behind; a tile's chunks past the row's end are empty
  auto chunk_of = [&](unsigned time) { return (int64_t)(p.tiles - 1 - time) * kGsTileWarps + w; };
  const Taken now = first_ticket(p.ticket, sm.ticket[0], chains, (unsigned)p.dim);
  if (now.id >= total) return;
  Place at = now.place;
  fill_stage<T, Z, true, CUT>(ring, p, at.chain, chunk_of(at.time) * G::PASS, lanes);
  copies_commit();
  for (int stg = 0;; stg ^= 1) {
    const int64_t row = at.chain, chunk = chunk_of(at.time), t = chunk * G::PASS - lead_of<CUT>(p, row);
    const int64_t t0 = t + lane * G::S, rem = p.L - t0;
    const int lead = CUT && t0 < 0 ? (int)-t0 : 0;
    unsigned char *stage = ring + stg * kStage<Z, true>;
    unsigned drawn = 0;
    if (threadIdx.x == 0) drawn = atomicAdd(p.ticket, 1u);
    unsigned long long seen;
    const void *q = tile_look(p, row, at.time, seen);
    const f2 b2 = splat2(p.bias ? p.bias[at.rest] * kLog2e : 0.f);
    const float first = at.time == 0 && p.dlast ? p.dlast[row] : 0.f;
    const float h0 = chunk >= chunks ? 0.f : chunk > 0 ? p.ckpt[row * chunks + chunk] : (p.h0 ? p.h0[row] : 0.f);
    unsigned st = 0;
    if constexpr (ST) st = load_starts<G::S>(p.starts + at.batch * p.L + t0, rem, lead, p.start_vec);
    copies_wait<0>();
    __syncwarp();
    f2 c[G::H], dh[G::H], R;
    drop_lead<T, Z, true>(stage, lane, lead);
    lane_direct<T, Z>(dh, stage, lane);
    const bool closed = lane_gates<T>(c, stage, lane, b2, rem, lead);
    const Halves hv = lane_run<T, TIED, ST, true>(closed, c, stage, lane, st, dh, R), gv = grad_halves(hv, R);
    Run r = join<ST>(hv.hi, hv.lo), g = join<ST>(gv.lo, gv.hi);
    scan_up<ST>(r, lane, 32);
    scan_down<ST>(g, lane, 32);
    const Run before = run_above(r, 32), after = run_below(g, 32);
    const float hin = lane == 0 ? h0 : run_on<ST>(before, h0);
    if (lane == 0) sm.run[stg][w] = g;
    if (threadIdx.x == 0) hand_out(sm.ticket[stg], drawn, chains, (unsigned)p.dim);
    __syncthreads();
    const Taken next = sm.ticket[stg];
    if (next.id < total)
      fill_stage<T, Z, true, CUT>(ring + (stg ^ 1) * kStage<Z, true>, p, next.place.chain, chunk_of(next.place.time) * G::PASS,
                             lanes);
    copies_commit();
    const float pw = tile_in<ST, true>(p, sm, sm.run[stg], row, at.time, first, q, seen, p.dh0);
    float db = lane_grads<T, TIED, Z, ST, CUT>(p, row, t, stage, lanes, st, c, dh, hin,
                                          lane == 31 ? pw : run_on<ST>(after, pw), hv.lo, gv.hi, t < p.L);
    if (p.dbias_part) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) db += __shfl_xor_sync(kAll, db, o);
      if (lane == 0) sm.db[w] = db;
      __syncthreads();
      if (threadIdx.x == 0) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kGsTileWarps; ++i) s += sm.db[i];
        p.dbias_part[((int64_t)at.batch * p.tiles + (p.tiles - 1 - at.time)) * p.dim + at.rest] = s;
      }
    }
    __syncwarp();
    if (next.id >= total) break;
    at = next.place;
  }
}

// ---- launches -----------------------------------------------------------------------------
template <typename K>
cudaError_t with_smem(K kern, int smem) {
  return smem > 40 * 1024 ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) : cudaSuccess;
}

// CUT: rows whose chunks begin at aligned places before them (p.cut); short rows take that
// variant always.
template <typename T, bool TIED, bool Z, bool ST, bool CUT>
cudaError_t launch_t(bool bwd, int path, const GsParams &p, cudaStream_t s) {
  const int64_t rows = p.batch * p.dim;
  cudaError_t e;
  if (path == SSM_PATH_LOOKBACK) {
    const int smem = kGsTileWarps * 2 * (bwd ? kStage<Z, true> : kStage<Z, false>);
    auto kern = bwd ? k_tiles_bwd<T, TIED, Z, ST, CUT> : k_tiles_fwd<T, TIED, Z, ST, CUT>;
    if ((e = with_smem(kern, smem)) != cudaSuccess) return e;
    const int64_t n = std::min<int64_t>(rows * p.tiles, (int64_t)p.sms * (bwd ? 2 : 3));
    kern<<<(unsigned)n, kTileThreads, smem, s>>>(p);
    return cudaGetLastError();
  }
  int W = 32;  // lanes per row: the fewest that hold a short row
  while (W > 1 && (int64_t)(W / 2) * Geo<T>::S >= gs_row_span(p.L, sizeof(T))) W /= 2;
  const int64_t warps = (rows + 32 / W - 1) / (32 / W), blocks = (warps * 32 + kRowThreads - 1) / kRowThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const int smem = kRowThreads / 32 * (bwd ? kRowBwdStages * kStage<Z, true> : kRowStages * kStage<Z, false>);
  auto kern = W == 32 ? (bwd ? k_rows_bwd<T, TIED, Z, ST, true, CUT> : k_rows_fwd<T, TIED, Z, ST, true, CUT>)
                      : (bwd ? k_rows_bwd<T, TIED, Z, ST, false, true> : k_rows_fwd<T, TIED, Z, ST, false, true>);
  if ((e = with_smem(kern, smem)) != cudaSuccess) return e;
  kern<<<(unsigned)blocks, kRowThreads, smem, s>>>(p, W);
  return cudaGetLastError();
}

template <typename T, bool CUT>
cudaError_t launch_cut(bool bwd, int path, const GsParams &p, cudaStream_t s) {
  const int v = (p.untied ? 0 : 4) | (p.z ? 2 : 0) | (p.starts ? 1 : 0);
  switch (v) {
    case 0: return launch_t<T, false, false, false, CUT>(bwd, path, p, s);
    case 1: return launch_t<T, false, false, true, CUT>(bwd, path, p, s);
    case 2: return launch_t<T, false, true, false, CUT>(bwd, path, p, s);
    case 3: return launch_t<T, false, true, true, CUT>(bwd, path, p, s);
    case 4: return launch_t<T, true, false, false, CUT>(bwd, path, p, s);
    case 5: return launch_t<T, true, false, true, CUT>(bwd, path, p, s);
    case 6: return launch_t<T, true, true, false, CUT>(bwd, path, p, s);
    default: return launch_t<T, true, true, true, CUT>(bwd, path, p, s);
  }
}

template <typename T>
cudaError_t launch_io(bool bwd, int path, const GsParams &p, cudaStream_t s) {
  return p.cut ? launch_cut<T, true>(bwd, path, p, s) : launch_cut<T, false>(bwd, path, p, s);
}

}  // namespace

cudaError_t launch_gs_rows_fwd(int io_dtype, int path, const GsParams &p, cudaStream_t s) {
  return io_dtype == SSM_BF16 ? launch_io<uint16_t>(false, path, p, s) : launch_io<float>(false, path, p, s);
}
cudaError_t launch_gs_rows_bwd(int io_dtype, int path, const GsParams &p, cudaStream_t s) {
  return io_dtype == SSM_BF16 ? launch_io<uint16_t>(true, path, p, s) : launch_io<float>(true, path, p, s);
}

}  // namespace ssm
