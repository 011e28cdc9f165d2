// Gated recurrence, token-major activations [batch][L][dim]: the channels of one
// token are contiguous, as a projection leaves them.
//
// Memory bound like the channel-major form, against 4 special-function results a value (backward 6: both
// walks form SiLU's sigmoid).  A lane takes a pair of channels, so every
// step is one f32x2 operation, and walks Tok<T>::RUN consecutive steps; the four warps of a block
// split a tile of 64 channels by four such runs and join them through shared memory; tiles of
// the same channels hand their runs on through the workspace.  Blocks stay and take tile after
// tile: the next tile's ticket is drawn and its values are on their way into shared memory
// (cp.async, each warp its own steps) while the current one is worked on.
#include "ssm_gscan.cuh"

#include <algorithm>

namespace ssm {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kTokThreads = 32 * kTokWarps;
constexpr int kTokFwdBlocks = 4, kTokBwdBlocks = 3;  // an SM: their shared memory and registers fit

template <typename T>
struct Tok {
  static constexpr int RUN = gs_tok_steps(sizeof(T)) / kTokWarps;  // steps per warp
  static constexpr int ROW = kTokChannels * (int)sizeof(T);        // bytes of a token's channels
  static constexpr int SLOT = RUN * ROW;                           // a warp's piece of one tensor
};
static_assert(Tok<uint16_t>::SLOT == 2048 && Tok<float>::SLOT == 2048, "slots are laid out alike");

template <bool Z, bool BWD>
constexpr int kWarpStage = 2048 * (2 + (Z ? 1 : 0) + (BWD ? 1 : 0));
constexpr int kTokF = 0, kTokU = 2048, kTokZ = 4096;
template <bool Z>
constexpr int kTokG = Z ? 6144 : 4096;

// the lane's pair of channels at step i of a slot
template <typename T>
__device__ __forceinline__ f2 pair_at(const unsigned char *slot, int i, int lane) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t v = *reinterpret_cast<const uint32_t *>(slot + i * Tok<T>::ROW + 4 * lane);
    return pack2(bf16_lo(v), bf16_hi(v));
  } else {
    return *reinterpret_cast<const f2 *>(slot + i * Tok<T>::ROW + 8 * lane);
  }
}

// Copies the warp's steps (n of them, from src: the first one's first channel of the group)
// into a slot, zeros for steps and channels that are not there.  ch: channels of the group
// there are.  16-byte pieces (mode 2); out of line, to keep the tile's code short: 4-byte
// words (mode 1) and elements (mode 0, not asynchronous).
template <typename T>
__device__ __noinline__ void fill_slot_narrow(unsigned char *slot, const T *src, int n, int ch, int64_t dim, int mode, int lane) {
  constexpr int RUN = Tok<T>::RUN, ROW = Tok<T>::ROW;
  if (mode == 1) {
    constexpr int E = 4 / (int)sizeof(T), PER = ROW / 128;  // rounds a token
    uint32_t s = (uint32_t)__cvta_generic_to_shared(slot) + 4 * lane;
    const T *q = src + lane * E;
    if (n == RUN && ch == kTokChannels) {
#pragma unroll
      for (int t = 0; t < RUN; ++t) {
#pragma unroll
        for (int h = 0; h < PER; ++h) copy4(s + 128 * (t * PER + h), q + 32 * E * h, true);
        q += dim;
      }
    } else {
#pragma unroll 2
      for (int t = 0; t < RUN; ++t) {
#pragma unroll
        for (int h = 0; h < PER; ++h) {
          const bool in = t < n && (h * 32 + lane) * E < ch;
          copy4(s + 128 * (t * PER + h), in ? q + 32 * E * h : src, in);
        }
        q += dim;
      }
    }
  } else {
    const T *q = src + lane;
    T v[RUN][2];
#pragma unroll
    for (int t = 0; t < RUN; ++t) {
      v[t][0] = t < n && lane < ch ? q[0] : T(0);
      v[t][1] = t < n && lane + 32 < ch ? q[32] : T(0);
      q += dim;
    }
#pragma unroll
    for (int t = 0; t < RUN; ++t) {
      T *d = reinterpret_cast<T *>(slot + t * ROW) + lane;
      d[0] = v[t][0];
      d[32] = v[t][1];
    }
  }
}
template <typename T>
__device__ __forceinline__ void fill_slot(unsigned char *slot, const T *src, int n, int ch, int64_t dim, int mode, int lane) {
  if (mode != 2) return fill_slot_narrow<T>(slot, src, n, ch, dim, mode, lane);
  constexpr int E = 16 / (int)sizeof(T), PER = Tok<T>::ROW / 16, STEP = 32 / PER;  // pieces a token, tokens a round
  const uint32_t s = (uint32_t)__cvta_generic_to_shared(slot) + 16 * lane;
  const int t = lane / PER, c = lane % PER * E;
  const T *q = src + t * dim + c;
  if (n == Tok<T>::RUN && ch == kTokChannels) {
#pragma unroll
    for (int j = 0; j < Tok<T>::RUN / STEP; ++j) {
      copy16(s + 512 * j, q, 16u);
      q += STEP * dim;
    }
  } else {
    const int left = c < ch ? n - t : 0;
#pragma unroll 1
    for (int j = 0; j < Tok<T>::RUN / STEP; ++j) {
      const bool in = j * STEP < left;
      copy16(s + 512 * j, in ? q : src, in ? 16u : 0u);
      q += STEP * dim;
    }
  }
}

// fp32 values of the lane's channels from a [..][dim] row (0 where absent), and back
struct Pair {
  int64_t d;       // the first one's channel
  bool in0, in1;
};
__device__ __forceinline__ f2 load_f32(const float *row, const Pair &c) {
  return pack2(row && c.in0 ? row[c.d] : 0.f, row && c.in1 ? row[c.d + 1] : 0.f);
}
__device__ __forceinline__ void store_f32(float *row, const Pair &c, f2 v) {
  float a, b;
  unpack2(v, a, b);
  if (c.in0) row[c.d] = a;
  if (c.in1) row[c.d + 1] = b;
}
// A step's pair to q, the lane's first channel.  all: the whole run is there and pairs are
// aligned (one access; c.in0 as the predicate), else by elements, `in` telling whether the
// step is there.
template <typename T>
__device__ __forceinline__ void put_pair(T *q, const Pair &c, bool all, bool in, f2 v) {
  float a, b;
  unpack2(v, a, b);
  if (all) {
    if constexpr (sizeof(T) == 2) {
      const uint32_t w = pack_bf16x2(a, b);
      if (c.in0) __stcs(reinterpret_cast<uint32_t *>(q), w);
    } else {
      if (c.in0) __stcs(reinterpret_cast<float2 *>(q), make_float2(a, b));
    }
  } else {
    if (in && c.in0) IO<T>::store1(q, 0, a);
    if (in && c.in1) IO<T>::store1(q, 1, b);
  }
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
template <typename T, bool ST>
__device__ __forceinline__ unsigned warp_starts(const GsParams &p, int64_t tok, int n, int lane) {
  if constexpr (!ST) return 0u;
  return __ballot_sync(kAll, lane < n && p.starts[tok + lane]);
}

// a start cuts the run, whatever its gates hold (NaN times 0)
template <bool ST>
__device__ __forceinline__ void cut_at_start(Run2 &r, unsigned st) {
  if constexpr (ST) {
    if (st) {
      r.A = splat2(kStart);
      r.N = splat2(-1.f);
    }
  }
}

// The next tile's ticket and the warps' runs, of this tile and the one before: what is written
// over lies two tiles back, and every warp has passed a barrier since it read it, so one barrier
// a tile is enough.  The other tile's place also takes the joined runs of a group's earlier
// tiles, with a barrier more at the tile's end.
struct TokShared {
  Taken ticket[2];
  f2 A[2][kTokWarps][32], N[2][kTokWarps][32], B[2][kTokWarps][32];
  __device__ __forceinline__ Run2 of(int k, int w, int lane) const { return {A[k][w][lane], N[k][w][lane], B[k][w][lane]}; }
  __device__ __forceinline__ void put(int k, int w, int lane, const Run2 &r) {
    A[k][w][lane] = r.A;
    N[k][w][lane] = r.N;
    B[k][w][lane] = r.B;
  }
};
struct TokSharedBwd : TokShared {
  f2 state[2][kTokWarps][32];  // B of the state's runs
  f2 sum[kTokWarps][32];
};

// a pair of states as one word of 64 bits
__device__ __forceinline__ void put_pair_state(unsigned long long *q, f2 v) {
  float x, y;
  unpack2(v, x, y);
  const unsigned long long w = ((unsigned long long)as_word(y) << 32) | as_word(x);
  asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(q), "l"(w) : "memory");
}
__device__ __forceinline__ f2 of_pair(unsigned long long w) { return pack2(of_word((unsigned)w), of_word((unsigned)(w >> 32))); }
__device__ __forceinline__ unsigned long long wait64(const unsigned long long *q, unsigned long long w, unsigned *err) {
  unsigned long long started = 0;
  unsigned n = 0;
  while (w == 0ull) {
    w = look64(q);
    if (w == 0ull && !spun(started, n, err)) break;
  }
  return w;
}

// Where the state that the tile's group starts from is (null in the first group)
__device__ __forceinline__ const unsigned long long *state_of(const GsParams &p, int64_t chain, unsigned c, int lane) {
  const unsigned g = c / p.group;
  if (g == 0) return nullptr;
  return reinterpret_cast<const unsigned long long *>(p.states) + (chain * p.groups + g - 1) * 32 + lane;
}

// Look-back of the whole block (see the channel-major form): `c` is the tile's index in
// the direction of the walk, sm holds the warps' runs in that direction (warp 0 first, or
// last with FROM_BEHIND), `q` and `seen` where the group's state is and what the lane saw of
// it when it looked ahead.  Returns the value entering the warp's own run; `out` receives, in
// the warp that the walk reaches last, the value leaving the tile.  The runs of the group's
// earlier tiles are joined in the order of their index, a quarter by each warp, before the
// state is waited for: from there to the state leaving the tile it is a few steps.
template <bool ST, bool FROM_BEHIND>
__device__ __forceinline__ f2 tile_in(const GsParams &p, TokShared &sm, int cur, int64_t chain, unsigned c, f2 first, int w,
                                      int lane, const unsigned long long *q, unsigned long long seen, f2 &out) {
  const unsigned g = c / p.group, in = c - g * p.group;
  const bool last = c == p.tiles - 1, last_in_group = in == p.group - 1;
  const int mine = FROM_BEHIND ? kTokWarps - 1 - w : w;  // the warp's place in the walk
  auto nth = [](int j) { return FROM_BEHIND ? kTokWarps - 1 - j : j; };
  if (p.group > 1) {
    unsigned long long *runs = p.runs + chain * p.tiles * kTokChannels;
    if (mine == 0 && !last && !last_in_group) {
      Run2 tile = sm.of(cur, nth(0), lane);
#pragma unroll
      for (int j = 1; j < kTokWarps; ++j) tile = join2<ST>(sm.of(cur, nth(j), lane), tile);
      Run x, y;
      split(tile, x, y);
      if (c == 0) {  // the state itself, as in the channel-major form
        float f0, f1;
        unpack2(first, f0, f1);
        x = Run{0.f, -1.f, run_on<ST>(x, f0)};
        y = Run{0.f, -1.f, run_on<ST>(y, f1)};
      }
      put_run(runs + (int64_t)c * kTokChannels + 2 * lane, x);
      put_run(runs + (int64_t)c * kTokChannels + 2 * lane + 1, y);
    }
    if (in > 0) {
      constexpr unsigned AT = 4;  // words of tiles on their way at once
      const unsigned part = (p.group + kTokWarps - 1) / kTokWarps, end = min(in, (mine + 1) * part);
      Run x = no_run(), y = no_run();
#pragma unroll 1
      for (unsigned j0 = mine * part; j0 < end; j0 += AT) {
        const unsigned long long *a = runs + ((int64_t)g * p.group + j0) * kTokChannels + 2 * lane;
        unsigned long long v[AT][2];
#pragma unroll
        for (unsigned j = 0; j < AT; ++j) {
          const bool there = j0 + j < end;
          v[j][0] = there ? look64(a + j * kTokChannels) : ~0ull;
          v[j][1] = there ? look64(a + j * kTokChannels + 1) : ~0ull;
        }
#pragma unroll
        for (unsigned j = 0; j < AT; ++j) {
          if (j0 + j >= end) break;
          x = join<ST>(of_words(wait64(a + j * kTokChannels, v[j][0], p.err)), x);
          y = join<ST>(of_words(wait64(a + j * kTokChannels + 1, v[j][1], p.err)), y);
        }
      }
      sm.put(cur ^ 1, mine, lane, {pack2(x.A, y.A), pack2(x.N, y.N), pack2(x.B, y.B)});
      __syncthreads();
    }
  }
  f2 h = first;
  if (q) h = of_pair(wait64(q, seen, p.err));
  if (in > 0) {
#pragma unroll
    for (int j = 0; j < kTokWarps; ++j) h = run_on2<ST>(sm.of(cur ^ 1, j, lane), h);
  }
#pragma unroll
  for (int j = 0; j < kTokWarps - 1; ++j) {
    if (j < mine) h = run_on2<ST>(sm.of(cur, nth(j), lane), h);
  }
  if (mine == kTokWarps - 1) {
    out = run_on2<ST>(sm.of(cur, w, lane), h);
    if (!last && last_in_group)
      put_pair_state(reinterpret_cast<unsigned long long *>(p.states) + (chain * p.groups + g) * 32 + lane, out);
  }
  return h;
}

// A tile's place in the tensors, for one warp
template <typename T, bool FROM_BEHIND>
struct Where {
  int64_t time, t0, tok;  // tile along time, the warp's first step, and its token
  int n;                  // steps of the warp there are
  int ch;                 // channels of the group there are
  int64_t first;          // element index of the warp's first step and the group's first channel
  __device__ __forceinline__ Where(const GsParams &p, const Place &a, int w) {
    time = FROM_BEHIND ? p.tiles - 1 - a.time : a.time;
    t0 = time * gs_tok_steps(sizeof(T)) + w * Tok<T>::RUN;
    tok = (int64_t)a.batch * p.L + t0;
    const int64_t left = p.L - t0, c = p.dim - (int64_t)a.rest * kTokChannels;
    n = left < 0 ? 0 : left < Tok<T>::RUN ? (int)left : Tok<T>::RUN;
    ch = c < kTokChannels ? (int)c : kTokChannels;
    first = tok * p.dim + (int64_t)a.rest * kTokChannels;
  }
};

template <typename T, bool Z, bool BWD>
__device__ __forceinline__ void fill_stage(unsigned char *st, const GsParams &p, const Where<T, BWD> &a, int lane) {
  // a warp with no steps copies nothing from, but its pointers have to be inside
  const int64_t at = a.n > 0 ? a.first : 0;
  fill_slot<T>(st + kTokF, static_cast<const T *>(p.f) + at, a.n, a.ch, p.dim, p.vec, lane);
  fill_slot<T>(st + kTokU, static_cast<const T *>(p.u) + at, a.n, a.ch, p.dim, p.vec, lane);
  if constexpr (Z) fill_slot<T>(st + kTokZ, static_cast<const T *>(p.z) + at, a.n, a.ch, p.dim, p.vec, lane);
  if constexpr (BWD) fill_slot<T>(st + kTokG<Z>, static_cast<const T *>(p.dout) + at, a.n, a.ch, p.dim, p.vec, lane);
}

// The gates of the warp's steps and their run on the state; steps past the end hold it.  With BWD,
// R of the gradient's run from behind, whose d is dh.
template <typename T, bool TIED, bool ST, bool BWD>
__device__ __forceinline__ Run2 warp_run(f2 (&c)[Tok<T>::RUN], const unsigned char *stage, int n, f2 b2, unsigned st, int lane,
                                         const f2 *dh, f2 &R) {
  constexpr int RUN = Tok<T>::RUN;
  Run2 r = {splat2(1.f), splat2(0.f), splat2(0.f)};
  R = splat2(0.f);
  float least = 1.f;
#pragma unroll
  for (int i = 0; i < RUN; ++i) c[i] = gate2(pair_at<T>(stage + kTokF, i, lane), b2, least);
  const bool closed = __any_sync(kAll, least < kClosed);
  if (closed) {
#pragma unroll
    for (int i = 0; i < RUN; ++i) c[i] = signed_gate2(pair_at<T>(stage + kTokF, i, lane), b2);
  }
  if (n < RUN) {
#pragma unroll
    for (int i = 0; i < RUN; ++i) c[i] = hold_at(c[i], i >= n, i >= n);
  }
  by_gates(closed, [&](auto kind) {
    constexpr bool C = decltype(kind)::value;
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
      if constexpr (ST) {
        if ((st >> i) & 1u) r.B = splat2(0.f);
      }
      r.B = state_step<TIED, C>(r.B, c[i], pair_at<T>(stage + kTokU, i, lane));
      run_step<C>(r.A, r.N, c[i]);
    }
    if constexpr (BWD) {
#pragma unroll
      for (int i = RUN - 1; i >= 0; --i) {
        R = grad_step<C>(add2(dh[i], R), c[i]);
        if constexpr (ST) {
          if ((st >> i) & 1u) R = splat2(0.f);
        }
      }
    }
  });
  float a0, a1, n0, n1;
  unpack2(r.A, a0, a1);
  unpack2(r.N, n0, n1);
  r.N = pack2(end_run(a0, n0), end_run(a1, n1));
  cut_at_start<ST>(r, st);
  return r;
}

template <typename T, bool TIED, bool Z, bool ST>
__global__ void __launch_bounds__(kTokThreads, kTokFwdBlocks) k_tok_fwd(GsParams p) {
  constexpr int RUN = Tok<T>::RUN, STAGE = kWarpStage<Z, false>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ TokShared sm;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  unsigned char *ring = smem + w * 2 * STAGE;
  const unsigned cgs = (unsigned)gs_tok_groups(p.dim), chains = (unsigned)p.batch * cgs, total = chains * (unsigned)p.tiles;
  const Taken now = first_ticket(p.ticket, sm.ticket[0], chains, cgs);
  if (now.id >= total) return;
  Place at = now.place;
  fill_stage<T, Z, false>(ring, p, Where<T, false>(p, at, w), lane);
  copies_commit();
  for (int stg = 0;; stg ^= 1) {
    const Where<T, false> a(p, at, w);
    const unsigned char *stage = ring + stg * STAGE;
    unsigned drawn = total;
    if (threadIdx.x == 0 && p.ticket) drawn = atomicAdd(p.ticket, 1u);
    const unsigned long long *q = state_of(p, at.chain, at.time, lane);
    const unsigned long long seen = q ? look64(q) : 0ull;
    const Pair ch = {(int64_t)at.rest * kTokChannels + 2 * lane, 2 * lane < a.ch, 2 * lane + 1 < a.ch};
    const f2 b2 = mul2(load_f32(p.bias, ch), splat2(kLog2e));
    const f2 first = load_f32(p.h0 && at.time == 0 ? p.h0 + at.batch * p.dim : nullptr, ch);
    const unsigned st = warp_starts<T, ST>(p, a.tok, a.n, lane);
    copies_wait<0>();
    __syncwarp();
    f2 c[RUN], none;
    const Run2 r = warp_run<T, TIED, ST, false>(c, stage, a.n, b2, st, lane, nullptr, none);
    sm.put(stg, w, lane, r);
    if (threadIdx.x == 0) hand_out(sm.ticket[stg], drawn, chains, cgs);
    __syncthreads();
    const Taken next = sm.ticket[stg];
    f2 out;
    f2 h = tile_in<ST, false>(p, sm, stg, at.chain, at.time, first, w, lane, q, seen, out);
    if (next.id < total) fill_stage<T, Z, false>(ring + (stg ^ 1) * STAGE, p, Where<T, false>(p, next.place, w), lane);
    copies_commit();
    if (p.ckpt && w == 0) store_f32(p.ckpt + ((int64_t)at.batch * p.tiles + at.time) * p.dim, ch, h);
    if (p.last && w == kTokWarps - 1 && at.time == p.tiles - 1) store_f32(p.last + at.batch * p.dim, ch, out);
    if (p.y) {
      auto walk = [&](bool all) {
        T *y = static_cast<T *>(p.y) + a.first + 2 * lane;
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
          if constexpr (ST) {
            if ((st >> i) & 1u) h = splat2(0.f);
          }
          h = state_step<TIED, true>(h, c[i], pair_at<T>(stage + kTokU, i, lane));
          f2 o = h;
          if constexpr (Z) {
            const f2 zv = pair_at<T>(stage + kTokZ, i, lane);
            o = mul2(h, mul2(zv, sigmoid2(zv)));
          }
          put_pair<T>(y, ch, all, i < a.n, o);
          y += p.dim;
        }
      };
      if (p.v32 && a.n == RUN) walk(true);
      else walk(false);
    }
    if (next.id >= total) break;
    at = next.place;
    if (p.group > 1) __syncthreads();  // every warp is done with the group's runs
  }
}

// The step of the state with w = -(h - u) a g (untied -h a g), a g being g - g^2 or a - a^2, and the
// step of the gradient with du = g G (untied G) and df = -w G.  That one's choice by the sign of c is
// a product with 1 or 0: fewer registers than a mask (8 x 4096 x 2048 packed backward 267 us, with
// masks 286, and 288 as the channel-major kernels form them).
template <bool TIED>
__device__ __forceinline__ f2 state_step_bwd(f2 h, f2 c, f2 u, f2 &w) {
  const f2 n = c | 0x8000000080000000ull;
  w = mul2(TIED ? fma2(u, splat2(-1.f), h) : h, fma2(n, n, n));
  return state_step<TIED, true>(h, c, u);
}
template <bool TIED>
__device__ __forceinline__ f2 grad_step_bwd(f2 G, f2 c, f2 w, f2 &du, f2 &df) {
  float lo, hi;
  asm("set.lt.f32.s32 %0, %1, 0;" : "=f"(lo) : "r"((int)(unsigned)c));
  asm("set.lt.f32.s32 %0, %1, 0;" : "=f"(hi) : "r"((int)(unsigned)(c >> 32)));
  const f2 near = mul2(G, pack2(lo, hi)), nG = mul2(G, splat2(-1.f));
  du = TIED ? fma2(c, nG, fma2(near, splat2(-1.f), G)) : G;
  df = mul2(nG, w);
  return fma2(c, G, near);
}

template <typename T, bool TIED, bool Z, bool ST>
__global__ void __launch_bounds__(kTokThreads, kTokBwdBlocks) k_tok_bwd(GsParams p) {
  constexpr int RUN = Tok<T>::RUN, STAGE = kWarpStage<Z, true>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ TokSharedBwd sm;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  unsigned char *ring = smem + w * 2 * STAGE;
  const unsigned cgs = (unsigned)gs_tok_groups(p.dim), chains = (unsigned)p.batch * cgs, total = chains * (unsigned)p.tiles;
  const Taken now = first_ticket(p.ticket, sm.ticket[0], chains, cgs);
  if (now.id >= total) return;
  Place at = now.place;
  fill_stage<T, Z, true>(ring, p, Where<T, true>(p, at, w), lane);
  copies_commit();
  for (int stg = 0;; stg ^= 1) {
    const Where<T, true> a(p, at, w);
    const unsigned char *stage = ring + stg * STAGE;
    unsigned drawn = total;
    if (threadIdx.x == 0 && p.ticket) drawn = atomicAdd(p.ticket, 1u);
    const unsigned long long *q = state_of(p, at.chain, at.time, lane);
    const unsigned long long seen = q ? look64(q) : 0ull;
    const Pair ch = {(int64_t)at.rest * kTokChannels + 2 * lane, 2 * lane < a.ch, 2 * lane + 1 < a.ch};
    const f2 b2 = mul2(load_f32(p.bias, ch), splat2(kLog2e));
    const float *hrow = a.time > 0 ? p.ckpt + ((int64_t)at.batch * p.tiles + a.time) * p.dim
                                   : p.h0 ? p.h0 + at.batch * p.dim : nullptr;
    f2 h = load_f32(hrow, ch);
    const f2 first = load_f32(p.dlast && at.time == 0 ? p.dlast + at.batch * p.dim : nullptr, ch);
    const unsigned st = warp_starts<T, ST>(p, a.tok, a.n, lane);
    copies_wait<0>();
    __syncwarp();
    // the state's run, and the gradient's from behind, which shares A and N with it
    f2 c[RUN], dh[RUN], R;
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
      dh[i] = pair_at<T>(stage + kTokG<Z>, i, lane);
      if constexpr (Z) {
        const f2 zv = pair_at<T>(stage + kTokZ, i, lane);
        dh[i] = mul2(dh[i], mul2(zv, sigmoid2(zv)));
      }
    }
    const Run2 r = warp_run<T, TIED, ST, true>(c, stage, a.n, b2, st, lane, dh, R);
    sm.put(stg, w, lane, {r.A, r.N, R});
    sm.state[stg][w][lane] = r.B;
    if (threadIdx.x == 0) hand_out(sm.ticket[stg], drawn, chains, cgs);
    __syncthreads();
    const Taken next = sm.ticket[stg];
    f2 out;
    f2 P = tile_in<ST, true>(p, sm, stg, at.chain, at.time, first, w, lane, q, seen, out);
    if (next.id < total) fill_stage<T, Z, true>(ring + (stg ^ 1) * STAGE, p, Where<T, true>(p, next.place, w), lane);
    copies_commit();
#pragma unroll
    for (int i = 0; i < kTokWarps - 1; ++i) {
      if (i < w) h = run_on2<ST>({sm.A[stg][i][lane], sm.N[stg][i][lane], sm.state[stg][i][lane]}, h);
    }
    if (p.dh0 && w == 0 && a.time == 0) store_f32(p.dh0 + at.batch * p.dim, ch, out);
    f2 sum = splat2(0.f);
    auto walk = [&](bool all) {
      f2 wt[RUN];
      const int64_t e0 = a.first + 2 * lane;
      T *dz = static_cast<T *>(p.dz) + e0;
#pragma unroll
      for (int i = 0; i < RUN; ++i) {
        if constexpr (ST) {
          if ((st >> i) & 1u) h = splat2(0.f);
        }
        h = state_step_bwd<TIED>(h, c[i], pair_at<T>(stage + kTokU, i, lane), wt[i]);
        if constexpr (Z) {  // dz = dout h s (1 + z (1 - s))
          const f2 zv = pair_at<T>(stage + kTokZ, i, lane), s = sigmoid2(zv);
          const f2 k = fma2(zv, fma2(s, splat2(-1.f), splat2(1.f)), splat2(1.f));
          put_pair<T>(dz, ch, all, i < a.n, mul2(mul2(pair_at<T>(stage + kTokG<Z>, i, lane), h), mul2(s, k)));
          dz += p.dim;
        }
      }
      T *du = static_cast<T *>(p.du) + e0 + RUN * p.dim, *df = static_cast<T *>(p.df) + e0 + RUN * p.dim;
#pragma unroll
      for (int i = RUN - 1; i >= 0; --i) {
        du -= p.dim;
        df -= p.dim;
        const bool in = i < a.n;
        f2 du_i, df_i;
        P = grad_step_bwd<TIED>(add2(dh[i], P), c[i], wt[i], du_i, df_i);
        put_pair<T>(du, ch, all, in, du_i);
        put_pair<T>(df, ch, all, in, df_i);
        if (all || in) sum = add2(sum, df_i);
        if constexpr (ST) {
          if ((st >> i) & 1u) P = splat2(0.f);
        }
      }
    };
    if (p.v32 && a.n == RUN) walk(true);
    else walk(false);
    if (p.dbias_part) {
      sm.sum[w][lane] = sum;
      __syncthreads();
      if (w == 0) {
        f2 t = splat2(0.f);
#pragma unroll
        for (int i = 0; i < kTokWarps; ++i) t = add2(t, sm.sum[i][lane]);
        store_f32(p.dbias_part + ((int64_t)at.batch * p.tiles + a.time) * p.dim, ch, t);
      }
    }
    if (next.id >= total) break;
    at = next.place;
    if (p.group > 1) __syncthreads();  // every warp is done with the group's runs
  }
}

template <typename T, bool TIED, bool Z, bool ST>
cudaError_t launch_t(bool bwd, const GsParams &p, cudaStream_t s) {
  const int64_t n = p.batch * gs_tok_groups(p.dim) * p.tiles;
  const int smem = kTokWarps * 2 * (bwd ? kWarpStage<Z, true> : kWarpStage<Z, false>);
  auto kern = bwd ? k_tok_bwd<T, TIED, Z, ST> : k_tok_fwd<T, TIED, Z, ST>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // without tickets (one tile a chain) every block has one tile
  const int64_t blocks = p.ticket ? std::min<int64_t>(n, (int64_t)p.sms * (bwd ? kTokBwdBlocks : kTokFwdBlocks)) : n;
  kern<<<(unsigned)blocks, kTokThreads, smem, s>>>(p);
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
