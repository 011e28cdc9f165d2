// Device code shared by the gated recurrence's kernels (ssm_gscan_rows.cu,
// ssm_gscan_tok.cu, ssm_gscan.cu).  Not part of the public interface.
//
//   g_t = sigmoid(-(f_t + bias)),  a_t = 1 - g_t
//   h_t = a_t h_{t-1} + g_t u_t   (untied: + u_t),  h_{t-1} := 0 at a start
//   y_t = h_t SiLU(z_t)
// Backward, with d_t = dout_t SiLU(z_t) and P_t = a_t G_t (0 at a start):
//   G_t = d_t + P_{t+1},  du = g G (untied: G),  dz = dout h SiLU'(z),
//   df = G (h_{t-1} - u) a g   (untied: G h_{t-1} a g),  dh0 = P_0.
//
// A run of steps acts on the state entering it as h -> A h + B, and on the
// gradient entering it from behind as P -> A P + R, with the same A = prod a_t.
// A lane walks its own steps from zero for its run, the runs before it are
// joined, and it walks its steps again from the state that enters them.
//
// A gate close to 1 (a memory of 1e5 steps) must not lose its 1 - a = g to the
// rounding of a, nor a run its 1 - A: a_t is never formed on the way (h and P move
// by x - g x in one rounding), and a run carries A and N = A - 1 side by side,
// each built without cancellation:
//   one step     A <- A - g A,   N <- N - g A
//   two runs     A = A1 A2,      N = N1 + A1 N2
// and is applied as x + N x + B while A > 1/2 and as A x + B below.  With A alone,
// rounded at every step, 1e5 steps of a constant a = 1 - 1e-5 came out 2e-4 off.
//
// A gate close to 0 must not lose its a to the rounding of g: 1 - g is off by 1e-7 or
// so, which is 1e-3 of a at f = -9 and all of it below -17.  So a step is kept as one number
// with every digit of what is small, the sign telling -g from the a of a nearly closed
// gate, and moves h from the nearer end: h + g (u - h), or u + a (h - u).
#pragma once

#include <type_traits>

#include "ssm_layer.cuh"

namespace ssm {

struct Run {
  float A, N, B;
};

// With packed sequences (ST) a run that holds a start has A = -0, and what came before it counts
// for nothing, infinities and NaN included.  Gates make no such A: they are not negative, so a
// product of theirs that underflows is +0, through which a NaN passes as through any other.
constexpr float kStart = -0.f;
__device__ __forceinline__ bool has_start(float A) { return __float_as_uint(A) == 0x80000000u; }

// The run applied to x.
template <bool ST>
__device__ __forceinline__ float run_on(const Run &r, float x) {
  const float far = fmaf(r.A, x, r.B), near = fmaf(r.N, x, x) + r.B;
  const float v = r.N > -0.5f ? near : far;
  if constexpr (ST) return has_start(r.A) ? r.B : v;
  return v;
}

// Two runs joined, `own` the one on the side the result comes out of: a start in it stays a
// start, whatever the other run holds, and one in the other stays one too (-0 times own's A).
template <bool ST>
__device__ __forceinline__ Run join(const Run &own, const Run &other) {
  Run r;
  r.B = run_on<ST>(own, other.B);
  r.A = own.A * other.A;
  r.N = fmaf(other.A, own.N, other.N);
  if constexpr (ST) {
    if (has_start(own.A)) {
      r.A = kStart;
      r.N = -1.f;
    }
  }
  return r;
}

__device__ __forceinline__ Run no_run() { return Run{1.f, 0.f, 0.f}; }

// one half of a pair zeroed where its bit says that a sequence starts
__device__ __forceinline__ f2 zero_at(f2 v, bool lo, bool hi) {
  float a, b;
  unpack2(v, a, b);
  return pack2(lo ? 0.f : a, hi ? 0.f : b);
}

__device__ __forceinline__ f2 put_at(f2 v, bool lo, bool hi, float x) {
  float a, b;
  unpack2(v, a, b);
  return pack2(lo ? x : a, hi ? x : b);
}

// The gate of a step as one number, the sign telling which: -g (-0 where e^f = inf), or a where
// the gate is nearly closed.  gate2 gives the first for every step, and the least e^f met (NaN
// apart), by which a warp sees whether any of its steps takes the second, from signed_gate2.
//
// kClosed: e^f below which a gate is nearly closed.  Above it 1 - g is a to 33 times g's error:
// 6e-6 at worst and 1e-6 as a rule, within what fp32 outputs are held to (1e-5).  Warps that have
// such gates do more: 4 x 5120 x 8192 bf16 forward takes 226 us with logits of N(b, 1), b from 0 to 6
// by channel, 245 us at b = 0 and 281 us at b = -4, where all warps have; with kClosed = 1/16 the
// first two take 230 and 260 us.
constexpr float kClosed = 0.03125f;
__device__ __forceinline__ f2 gate2(f2 f, f2 b2, float &least) {
  float x, y, d0, d1;
  unpack2(fma2(f, splat2(kLog2e), b2), x, y);
  x = ex2(x);
  y = ex2(y);
  asm("min.f32 %0, %0, %1, %2;" : "+f"(least) : "f"(x), "f"(y));
  unpack2(fma2(pack2(x, y), splat2(-1.f), splat2(-1.f)), d0, d1);
  return pack2(rcp_approx(d0), rcp_approx(d1));
}
__device__ __forceinline__ f2 signed_gate2(f2 f, f2 b2) {
  float x, y, d0, d1;
  unpack2(fma2(f, splat2(kLog2e), b2), x, y);
  x = ex2(x);
  y = ex2(y);
  unpack2(fma2(pack2(x, y), splat2(-1.f), splat2(-1.f)), d0, d1);
  return mul2(pack2(x < kClosed ? -x : 1.f, y < kClosed ? -y : 1.f), pack2(rcp_approx(d0), rcp_approx(d1)));
}
// every bit set in the halves where c is a -g, and a choice between two pairs by it
__device__ __forceinline__ f2 open2(f2 c) {
  const int lo = (int)(unsigned)c >> 31, hi = (int)(unsigned)(c >> 32) >> 31;
  return ((f2)(unsigned)hi << 32) | (unsigned)lo;
}
__device__ __forceinline__ f2 pick2(f2 m, f2 x, f2 y) { return (x & m) | (y & ~m); }
// a x
__device__ __forceinline__ f2 kept2(f2 x, f2 c) { return fma2(c, x, x & open2(c)); }
// steps that are not there hold the state: g = 0
__device__ __forceinline__ f2 hold_at(f2 c, bool lo, bool hi) { return put_at(c, lo, hi, -0.f); }

// 1 / (1 + e^-z) on a pair
__device__ __forceinline__ f2 sigmoid2(f2 z) {
  float x, y, d0, d1;
  unpack2(mul2(z, splat2(-kLog2e)), x, y);
  unpack2(add2(pack2(ex2(x), ex2(y)), splat2(1.f)), d0, d1);
  return pack2(rcp_approx(d0), rcp_approx(d1));
}

// One step of the state: a h + u, or with tied gates h + g (u - h) = u + a (h - u), from the end
// that the number at hand is the distance to.  C: of a warp that may have nearly closed gates.
template <bool TIED, bool C>
__device__ __forceinline__ f2 state_step(f2 h, f2 c, f2 u) {
  if constexpr (TIED) return fma2(c, fma2(u, splat2(-1.f), h), C ? pick2(open2(c), h, u) : h);
  return add2(C ? kept2(h, c) : fma2(c, h, h), u);
}
// One step of the gradient from behind, P from G
template <bool C>
__device__ __forceinline__ f2 grad_step(f2 G, f2 c) { return C ? kept2(G, c) : fma2(c, G, G); }
// A and N of a run, one step more.  N counts up to the first nearly closed gate only, A being below
// 1/2 from there on: end_run sees to that.
template <bool C>
__device__ __forceinline__ void run_step(f2 &A, f2 &N, f2 c) {
  N = fma2(c, A, N);
  A = C ? kept2(A, c) : fma2(c, A, A);
}
__device__ __forceinline__ float end_run(float A, float N) { return A < 0.4f ? -1.f : N; }
// f(C), for a warp that has nearly closed gates and for one that has not
template <typename F>
__device__ __forceinline__ void by_gates(bool closed, F f) {
  if (closed) f(std::true_type{});
  else f(std::false_type{});
}

// ---- what tiles hand on to one another ----------------------------------------
// A word of the workspace is 0 until its value is there: values are stored with
// every bit inverted, and the one pattern that would invert to 0 (a NaN) is
// replaced by another NaN.  A word is written and read whole, so no fence is
// needed: the value is its own flag.
__device__ __forceinline__ unsigned as_word(float v) {
  const unsigned b = __float_as_uint(v);
  return b == 0xffffffffu ? 0x80000000u /* ~0x7fffffff, a NaN */ : ~b;
}
__device__ __forceinline__ float of_word(unsigned w) { return __uint_as_float(~w); }
// A run as 64 bits: B, and N (> -1/2) with its sign, or else A without one, which is at most 1/2
// then: a 2 stands for a start.
__device__ __forceinline__ void put_run(unsigned long long *p, const Run &r) {
  const float e = r.N > -0.5f ? -fabsf(r.N) : has_start(r.A) ? 2.f : fabsf(r.A);
  const unsigned long long v = ((unsigned long long)as_word(r.B) << 32) | as_word(e);
  asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}
__device__ __forceinline__ Run of_words(unsigned long long v) {
  Run r;
  const float e = of_word((unsigned)v);
  r.B = of_word((unsigned)(v >> 32));
  const bool n = (__float_as_uint(e) >> 31) != 0u, start = e == 2.f;
  r.N = n ? e : start ? -1.f : e - 1.f;
  r.A = n ? 1.f + e : start ? kStart : e;
  return r;
}
__device__ __forceinline__ void put_state(unsigned *p, float h) {
  asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(as_word(h)) : "memory");
}
__device__ __forceinline__ unsigned long long look64(const unsigned long long *p) {
  unsigned long long v;
  asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ unsigned look32(const unsigned *p) {
  unsigned v;
  asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// The bounded wait for such words: spun(started, n, err) is false once the limit has passed or
// another wait of the call has given up; the error word is set then, and the caller goes on with
// what it has.
__device__ __forceinline__ bool spun(unsigned long long &started, unsigned &n, unsigned *err,
                                     unsigned long long limit_ns = kWaitLimitNs) {
  if (n++ == 0) {
    started = global_ns();
    return true;
  }
  __nanosleep(20);
  if ((n & 63u) != 0) return true;
  if (look32(err) != 0u) return false;
  if (global_ns() - started > limit_ns) {
    atomicOr(err, kErrWaitTimeout);
    return false;
  }
  return true;
}

// ---- copies ahead into shared memory ---------------------------------------------------
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, uint32_t bytes) {  // zeros after `bytes`
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4u : 0u) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Tile order.  Blocks take tiles by ticket, the tiles of one time index before those of
// the next, so a tile that is waited for was taken earlier and is running or done (a block
// draws its next ticket while it works on a tile, and finishes its tiles in order: the lowest
// unfinished ticket never waits).  Drawn two ahead, with the copies started an iteration
// earlier, the tiles that others wait for lay longer in a block's hands: 1 x 1024 x 2^20 took
// 2.01 instead of 1.80 ms.  One thread splits the ticket into the tile's time index, its chain (a row, or the channel
// group of a batch element), and that into the batch element and what is left, in 32 bits
// (the host checks that they fit): four 64-bit divisions in every thread cost more than the
// gates.
struct Place {
  unsigned time, chain, batch, rest;
};
__device__ __forceinline__ Place place_of(unsigned ticket, unsigned chains, unsigned per_batch) {
  Place q;
  q.time = ticket / chains;
  q.chain = ticket - q.time * chains;
  q.batch = q.chain / per_batch;
  q.rest = q.chain - q.batch * per_batch;
  return q;
}
// A ticket as thread 0 draws it and hands it out at a barrier of the block.
struct Taken {
  unsigned id;
  Place place;
};
__device__ __forceinline__ void hand_out(Taken &t, unsigned id, unsigned chains, unsigned per_batch) {
  t.id = id;
  t.place = place_of(id, chains, per_batch);
}
// the first one of a block; without a counter (one tile a chain) the block's index is its
// only ticket
__device__ __forceinline__ Taken first_ticket(unsigned *counter, Taken &shared, unsigned chains, unsigned per_batch) {
  if (threadIdx.x == 0) hand_out(shared, counter ? atomicAdd(counter, 1u) : blockIdx.x, chains, per_batch);
  __syncthreads();
  const Taken t = shared;
  __syncthreads();  // read before the next one takes its place
  return t;
}

}  // namespace ssm
