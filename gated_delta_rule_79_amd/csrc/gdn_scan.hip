// Selective state space scan: every channel j of the H heads carries dk
// values,
//
//   delta_t = softplus(dt_t + bias)            (or dt_t + bias)
//   S_t[n]  = e^{delta_t a[n]} S_{t-1}[n] + delta_t x_t b_t[n]
//   y_t     = (sum_n c_t[n] S_t[n] + d x_t) * silu(z_t)
//
// with b, c rows shared by all channels of a group (H / hb heads), its
// backward and its single-token step.
//
// A lane owns one channel and NS of its states, in registers for a whole walk
// over the tokens; a wave owns 64 channels of one group, so that the b and c
// values are the same for all its lanes and arrive as scalars.  More than NS
// states are shared out over WS waves of the workgroup, whose sums over n meet
// in LDS.  There is no product of two shared matrices here (the decay differs
// in every channel and state), so nothing for the matrix cores: the vector
// unit's exponential, two multiplications and two multiply-adds for every
// token, channel and state bound the walks.  A group of fewer than 64 channels
// leaves lanes idle: 4096 tokens of 128 heads of 16 channels take 207 us with
// rows of b and c for each head, 74 with one for all.
//
// Few or long sequences are cut into segments walked by workgroups of their
// own: one launch walks every segment from zero and leaves its last state and
// the sum of its delta (the segment's decay is e^{a sum}); one chains them;
// one walks the outputs from the states chained.  Packed sequences are cut
// on the grid of all tokens, whatever their bounds: a walk goes from run to
// run of one sequence and takes up each sequence's own initial state, so all
// workgroups have the same number of tokens and the host need not know the
// lengths.

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "gdn_device.hpp"
#include "gdn_internal.hpp"

namespace gdn {

namespace {

// Waves of a workgroup whose channel blocks take ws waves each.
constexpr int waves_of(int ws) { return ws > 4 ? ws : 4; }
constexpr float kLog2e = 1.44269504088896340736f, kLog2eLow = 1.92596303e-8f;  // and the rest
constexpr float kLn2 = 0.69314718055994530942f;

#define GDN_CONST __attribute__((address_space(4)))

// ------------------------------------------------------------- functions ---

// e^x for |x| <= 200, 0 or infinity where that passes them.  What the product
// x log2(e) loses goes back in, by its own rounding and by the constant's
// (without the latter e^-82 is off by 19 u).  No branches in these: they stand
// between the loads of every token.
__device__ inline float exp_full(float x) {
  const float t = x * kLog2e, lost = fmaf(x, kLog2eLow, fmaf(x, kLog2e, -t));
  return __builtin_amdgcn_exp2f(t) * fmaf(lost, kLn2, 1.f);
}

// softplus(v) = max(v, 0) + log(1 + u), u = e^{-|v|}: w = 1 + u is off by
// d = u - (w - 1), log(w + d) = log(w) + d to 2^-25 of the result.  (Of a NaN
// the maximum stays.)  Its least value is e^-83 = 9e-37: never zero, so that
// the least step times the lowest finite rate is a decay of zero (rate_of).
__device__ inline float softplus(float v) {
  const float u = exp_full(fmaxf(-fabsf(v), -83.f)), w = 1.f + u;
  return __builtin_elementwise_maximum(v, 0.f) +
         fmaf(kLn2, __builtin_amdgcn_logf(w), u - (w - 1.f));
}

// bf16 rows take the exponential as it is: its error, |v| 2^-24, is far below
// the rounding of rows in bf16, and in the fp32 sums da, dd and dt_bias's
// gradient the size of a term's own rounding.  Zero from about -89 down, so
// that v times it is none of the type's lowest value; of a NaN it is anything,
// its users keep the NaN.
template <typename IO>
__device__ inline float sigmoid(float v) {
  const float e = io<IO>::bytes == 2 ? __builtin_amdgcn_exp2f(-v * kLog2e)
                                     : exp_full(__builtin_amdgcn_fmed3f(-v, -200.f, 200.f));
  return __builtin_amdgcn_rcpf(1.f + e);
}

// ------------------------------------------------------------------ sizes ---

struct Args {
  int64_t T;          // tokens of a dense sequence, or of the packed row
  int D, Dg, nb;      // channels, channels of a group, 64-channel blocks of a group
  int units;          // nb times the groups
  int ublocks;        // workgroups of a segment
  int dk, dv, hb;
  int S, L;           // segments of a sequence (packed: of all), their tokens
  int nseq;
  int softplus;
  const int32_t* cu;
  const void *x, *dt, *b, *c, *z, *dy;
  const float *a, *d, *bias, *s0, *ds;
  void *y, *dx, *ddt, *dz;
  float *sf, *ds0;
  // workspace
  int* cut;           // [segments] the state behind the segment does not see its front
  float* h;           // [segments][D dk] state behind a segment; after the chaining, in front
  float* sum;         // [segments][D] sum of delta
  int* cutr;          // the same from the last token back
  float* g;
  float *mark, *msum; // [tokens / kTile][D dk], [..][D]: states inside segments
  float* part;        // [tokens][units][WS][2][NS] shares of db, dc
  float *pa, *pd, *pb;  // [segments][D dk], [segments][WS][D] twice
};

// A segment's tokens, counted over all sequences.
struct Span {
  int64_t lo, hi;
  int at;             // slot
  int chain;          // dense: the sequence
  bool first, last;   // of its sequence (packed: of all)
};

__device__ inline Span span_of(const Args& A, int at) {
  Span s;
  s.at = at;
  s.chain = at / A.S;
  const int k = at - s.chain * A.S;
  s.first = k == 0;
  s.last = k == A.S - 1;
  const int64_t base = s.chain * A.T, from = static_cast<int64_t>(k) * A.L;
  s.lo = base + (from < A.T ? from : A.T);
  s.hi = base + (s.last || from + A.L > A.T ? A.T : from + A.L);
  return s;
}

__device__ inline int64_t bound(const Args& A, int n) {
  return reinterpret_cast<const GDN_CONST int32_t*>(reinterpret_cast<uintptr_t>(A.cu))[n];
}

// smallest n with cu[n] >= t, A.nseq + 1 if there is none
__device__ inline int lower(const Args& A, int64_t t) {
  int lo = 0, hi = A.nseq + 1;
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (bound(A, m) >= t) hi = m;
    else lo = m + 1;
  }
  return lo;
}

// The tokens of one sequence in a segment.
struct Run {
  int seq;
  int64_t lo, hi;
  bool cont;   // they continue the segment in front
  bool ends;   // the sequence ends with them
};

// The runs of a segment: index 0 is what continues the segment in front (if
// there is such), 1 .. count are the sequences that begin here, empty ones
// among them.  Bounds outside the segment or out of order give runs inside it.
struct Runs {
  int n0, count;
  bool cont;
};

__device__ inline Runs runs_of(const Args& A, const Span& s) {
  Runs r;
  if (A.cu == nullptr) {
    r.n0 = s.chain;
    r.count = s.first ? 1 : 0;
    r.cont = !s.first;
    return r;
  }
  r.n0 = lower(A, s.lo);
  // (nothing lies in front of the first segment, whatever the bounds say)
  r.cont = !s.first && r.n0 > 0 && r.n0 <= A.nseq && bound(A, r.n0) > s.lo;
  const int end = s.last ? A.nseq : min(lower(A, s.hi), A.nseq);
  r.count = max(end - r.n0, 0);
  return r;
}

__device__ inline Run run_at(const Args& A, const Span& s, const Runs& r, int i) {
  Run t;
  t.cont = i == 0;
  if (A.cu == nullptr) {
    t.seq = s.chain;
    t.lo = s.lo;
    t.hi = s.hi;
    t.ends = s.last;
    return t;
  }
  t.seq = r.n0 + i - 1;
  const int64_t b = bound(A, t.seq), e = bound(A, t.seq + 1);
  t.lo = i == 0 || b < s.lo ? s.lo : b > s.hi ? s.hi : b;
  t.hi = e < t.lo ? t.lo : e > s.hi ? s.hi : e;
  t.ends = s.last || e <= s.hi;  // (nor anything behind the last)
  return t;
}

// ------------------------------------------------------------------ lanes ---

// Memory through buffer descriptors: a row's place is a scalar, a lane's the
// same 32-bit byte offset in every row, and what lies past the descriptor's
// bytes (rows behind a run, lanes without a channel) is read as zero and not
// written.
constexpr uint32_t kNowhere = 0x80000000u;

__device__ inline __amdgpu_buffer_rsrc_t buffer(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes),
                                           0x00027000);
}

// A rate in powers of two, kept finite so that no step at all (a token past
// its run) leaves a state as it is.  Of a rate of -inf any step that softplus
// gives leaves nothing all the same (9e-37 x 3.4e38 = 306 halvings); of steps
// given without it those from 4.4e-37 up.
__device__ inline float rate_of(float a) {
  const float a2 = a * kLog2e;
  return a2 < -3.4e38f ? -3.4e38f : a2;
}

// What a lane keeps of its channel.
template <int NS>
struct Lane {
  int unit, grp;      // channel block, group
  int n0, left;       // first state of the wave, states from it on
  int ch;             // channel (of the last one where the lane has none)
  bool live;
  uint32_t row;       // bytes in front of the channel in a row of x
  uint32_t state;     // bytes in front of (n0, channel) in a [H, dk, dv] state
  float a2[NS];       // a log2(e)
  float bias, d;
};

template <int NS, bool PAD>
__device__ inline void load_state(const Args& A, const Lane<NS>& l, const float* p, float* h) {
  const auto b = buffer(p, 4u * A.D * A.dk);
#pragma unroll
  for (int i = 0; i < NS; ++i)
    h[i] = !PAD || i < l.left
               ? __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, l.state, 4 * i * A.dv, 0))
               : 0.f;
}
template <int NS, bool PAD>
__device__ inline void store_state(const Args& A, const Lane<NS>& l, float* p, const float* h) {
  const auto b = buffer(p, 4u * A.D * A.dk);
#pragma unroll
  for (int i = 0; i < NS; ++i)
    if (!PAD || i < l.left)
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(h[i]), b, l.state, 4 * i * A.dv, 0);
}

template <typename IO, int NS, bool PAD>
__device__ inline Lane<NS> lane_of(const Args& A, int WS) {
  Lane<NS> l;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int unit = blockIdx.x % A.ublocks * (waves_of(WS) / WS) + wave / WS;
  l.unit = min(unit, A.units - 1);
  l.grp = l.unit / A.nb;
  const int j = (l.unit - l.grp * A.nb) * 64 + lane;
  l.live = unit < A.units && j < A.Dg;
  l.ch = l.grp * A.Dg + min(j, A.Dg - 1);
  l.n0 = (wave % WS) * NS;
  l.left = A.dk - l.n0;
  const int head = l.ch / A.dv;
  l.row = l.live ? l.ch * io<IO>::bytes : kNowhere;
  l.state = l.live ? 4u * (head * A.dk * A.dv + l.ch - head * A.dv + l.n0 * A.dv) : kNowhere;
  load_state<NS, PAD>(A, l, A.a, l.a2);
#pragma unroll
  for (int i = 0; i < NS; ++i) l.a2[i] = rate_of(l.a2[i]);
  l.bias = A.bias != nullptr ? A.bias[l.ch] : 0.f;
  l.d = A.d != nullptr ? A.d[l.ch] : 0.f;
  return l;
}

// N values of a token's b or c row, the same for all lanes and so scalars;
// they stay packed until they are used.  left: states from the first of them
// to the row's end; those past it are zeros.
template <typename IO, int N, bool PAD>
struct Row {
  uint32_t w[N * io<IO>::bytes / 4];
  int left;
  // from: the wave's part of the row (its last four states where it has fewer)
  __device__ inline void load(uintptr_t from, int states) {
    left = states;
#pragma unroll
    for (int q = 0; q < N; q += 4) {
      const int n = PAD ? min(q, states - 4) : q;
      const GDN_CONST uint32_t* s =
          reinterpret_cast<const GDN_CONST uint32_t*>(from + n * io<IO>::bytes);
#pragma unroll
      for (int i = 0; i < io<IO>::bytes; ++i) w[q * io<IO>::bytes / 4 + i] = s[i];
    }
  }
  __device__ inline float operator[](int n) const {
    uint32_t u;
    if constexpr (io<IO>::bytes == 4) u = w[n];
    else u = n & 1 ? w[n >> 1] & 0xffff0000u : w[n >> 1] << 16;
    return __uint_as_float(PAD && (n & ~3) >= left ? 0u : u);
  }
  // Unpacks anew from here on (kept unpacked, a row takes a register a value).
  __device__ inline void pack() {
#pragma unroll
    for (auto& x : w) asm volatile("" : "+s"(x));
  }
  // The loads are there when this returns: what is loaded next is not waited
  // for together with them (scalar loads end in any order, so the wait for
  // one is a wait for all).
  __device__ inline void arrive() const {
    asm volatile("" ::"s"(w[0]));
    __builtin_amdgcn_sched_barrier(0);
  }
};

// Values of a wave's channels in U tokens, as stored; left: tokens of the run
// from the first of them (rows past it are zeros).
template <typename IO, int U>
struct Rows {
  uint32_t v[U];
  __device__ inline void load(const Args& A, const void* p, int64_t tok, int left, uint32_t row) {
    const uint32_t bytes = A.D * io<IO>::bytes;
    const int most = max(min(left, U), 0);
    const auto b = buffer(static_cast<const char*>(p) + tok * bytes, most * bytes);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // (a scalar offset past the descriptor's end is not relied on)
      const uint32_t at = min(u, most) * bytes;
      if constexpr (io<IO>::bytes == 2) v[u] = __builtin_amdgcn_raw_buffer_load_b16(b, row, at, 0);
      else v[u] = __builtin_amdgcn_raw_buffer_load_b32(b, row, at, 0);
    }
  }
  __device__ inline float operator[](int u) const {
    return __uint_as_float(io<IO>::bytes == 2 ? v[u] << 16 : v[u]);
  }
};
// The rows of a run from token tok on, to be written.
template <typename IO, int U>
struct RowsOut {
  __amdgpu_buffer_rsrc_t b;
  int most;
  uint32_t bytes;
  __device__ inline RowsOut(const Args& A, void* p, int64_t tok, int left)
      : most(min(left, U)), bytes(A.D * io<IO>::bytes) {
    b = buffer(static_cast<char*>(p) + tok * bytes, most * bytes);
  }
  __device__ inline void store(int u, uint32_t row, float v) const {
    const uint32_t at = min(u, most) * bytes;
    if constexpr (io<IO>::bytes == 2)
      __builtin_amdgcn_raw_buffer_store_b16(
          __builtin_bit_cast(uint16_t, static_cast<__bf16>(v)), b, row, at, 0);
    else
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), b, row, at, 0);
  }
};

template <typename IO>
__device__ inline float load_x(const void* p, const Args& A, int64_t tok, int ch) {
  return io<IO>::load(static_cast<const char*>(p) + tok * A.D * io<IO>::bytes, ch);
}
template <typename IO>
__device__ inline void store_x(void* p, const Args& A, int64_t tok, int ch, float v) {
  io<IO>::store(static_cast<char*>(p) + tok * A.D * io<IO>::bytes, ch, v);
}

__device__ inline float step_of(const Args& A, float dt, float bias) {
  const float v = dt + bias, s = softplus(v);
  return A.softplus ? s : v;
}

__device__ inline float decay(float delta, float a2) {
  return __builtin_amdgcn_exp2f(delta * a2);
}

// Where the wave's part of a token's row of b or c begins, and the bytes from
// one token's to the next.
template <typename IO, int NS>
__device__ inline uintptr_t row_of(const Args& A, const Lane<NS>& l, const void* p, int64_t tok) {
  return reinterpret_cast<uintptr_t>(p) + ((tok * A.hb + l.grp) * A.dk + l.n0) * io<IO>::bytes;
}
template <typename IO>
__device__ inline int row_step(const Args& A) {
  return A.hb * A.dk * io<IO>::bytes;
}

// The state a run starts from.
template <int NS, bool PAD>
__device__ inline void enter(const Args& A, const Lane<NS>& l, const Span& s, const Run& r,
                             float* h) {
  const int64_t size = static_cast<int64_t>(A.D) * A.dk;
  if (r.cont) {
    load_state<NS, PAD>(A, l, A.h + s.at * size, h);
  } else if (A.s0 != nullptr) {
    load_state<NS, PAD>(A, l, A.s0 + r.seq * size, h);
  } else {
#pragma unroll
    for (int i = 0; i < NS; ++i) h[i] = 0.f;
  }
}

// A run's rows of b or c, fetched ahead of their tokens: a group of U tokens at
// once where that takes few scalars (one wait a group, which is what few waves
// feel), else one token.
template <typename IO, int NS, bool PAD, int U>
struct Ahead {
  static constexpr bool GROUP = NS * io<IO>::bytes <= 16;
  typedef Row<IO, NS, PAD> row;
  row next[GROUP ? U : 1], cur[GROUP ? U : 1];
  uintptr_t from;  // the group's first row
  int step, left;  // bytes of a row; states of the wave
  __device__ inline void start(uintptr_t p, int row_step, int states, int tokens) {
    from = p;
    step = row_step;
    left = states;
    if (tokens > 0) fetch(0, tokens);
  }
  // the group from token `at` on (or that token) of those that are left
  __device__ inline void fetch(int at, int tokens) {
#pragma unroll
    for (int u = 0; u < (GROUP ? U : 1); ++u) next[u].load(from + min(at + u, tokens - 1) * step, left);
  }
  __device__ inline void take() {
#pragma unroll
    for (int u = 0; u < (GROUP ? U : 1); ++u) cur[u] = next[u];
  }
  __device__ inline const row& operator[](int u) const { return cur[GROUP ? u : 0]; }
  __device__ inline void group_done() { from += U * step; }
};

// Walks a run in groups of four tokens, the next group's rows and the next
// token's b on their way: f(t, left, x, u, delta, b) for token u of the group
// at t.  Tokens past the run have x = delta = 0, which leaves a state as it is.
template <typename IO, int NS, bool PAD, typename F>
__device__ inline void walk(const Args& A, const Lane<NS>& l, const Run& r, F f) {
  constexpr int U = 4;
  typedef Ahead<IO, NS, PAD, U> ahead;
  Rows<IO, U> x, dt;
  ahead b;
  int left = static_cast<int>(r.hi - r.lo);
  x.load(A, A.x, r.lo, left, l.row);
  dt.load(A, A.dt, r.lo, left, l.row);
  b.start(row_of<IO>(A, l, A.b, r.lo), row_step<IO>(A), l.left, left);
  for (int64_t t = r.lo; left > 0; t += U, left -= U) {
    const Rows<IO, U> xs = x, dts = dt;
    x.load(A, A.x, t + U, left - U, l.row);
    dt.load(A, A.dt, t + U, left - U, l.row);
    float delta[U];
#pragma unroll
    for (int u = 0; u < U; ++u) delta[u] = u < left ? step_of(A, dts[u], l.bias) : 0.f;
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (ahead::GROUP) {
      b.take();
      b[0].arrive();
      b.fetch(U, left);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (!ahead::GROUP) {
        b.take();
        b[0].arrive();
        b.fetch(u + 1, left);
      }
      f(t, left, xs, u, delta[u], b[u]);
      __builtin_amdgcn_sched_barrier(0);
    }
    b.group_done();
  }
}

// --------------------------------------------------- segments' own states ---

// State behind a segment: from its last run, walked from its sequence's
// initial state or, where it continues the segment in front, from zero.
template <typename IO, int NS, bool PAD>
__global__ __launch_bounds__(512) void scan_local_kernel(Args A, int WS) {
  const int k = blockIdx.x / A.ublocks;
  const Span s = span_of(A, k + k / (A.S - 1));  // (no last segment of a sequence)
  const Runs rs = runs_of(A, s);
  const Lane<NS> l = lane_of<IO, NS, PAD>(A, WS);
  const int64_t size = static_cast<int64_t>(A.D) * A.dk;
  int i = rs.count;
  Run r{};
  for (; i >= (rs.cont ? 0 : 1); --i) {
    r = run_at(A, s, rs, i);
    if (r.hi > r.lo) break;
  }
  float h[NS], sum = 0.f;
#pragma unroll
  for (int n = 0; n < NS; ++n) h[n] = 0.f;
  const bool none = i < (rs.cont ? 0 : 1);
  if (!none) {
    if (!r.cont) enter<NS, PAD>(A, l, s, r, h);
    walk<IO, NS, PAD>(A, l, r, [&](int64_t, int, const Rows<IO, 4>& x, int u, float delta,
                                   const Row<IO, NS, PAD>& b) {
      const float dx = delta * x[u];
      sum += delta;
#pragma unroll
      for (int n = 0; n < NS; ++n) h[n] = fmaf(decay(delta, l.a2[n]), h[n], dx * b[n]);
    });
  }
  store_state<NS, PAD>(A, l, A.h + s.at * size, h);
  if (l.live && l.n0 == 0) A.sum[static_cast<int64_t>(s.at) * A.D + l.ch] = sum;
  if (blockIdx.x % A.ublocks == 0 && threadIdx.x == 0) A.cut[s.at] = none || !r.cont;
}

// Chains the segments' states, every one replaced by the state in front of its
// segment, and (second half of the grid) the gradients, every one replaced by
// the gradient of the state behind its segment.  A wave chains a share of the
// segments of 64 channels and states, the shares meet in LDS, and every wave
// goes over its own again: 128 segments of 65536 values take 21 us (three passes
// of 34 MB, 4.9 TB/s).
constexpr int kChainWaves = 16;
__global__ __launch_bounds__(64 * kChainWaves) void scan_chain_kernel(Args A, int64_t blocks) {
  constexpr int U = 8;
  __shared__ float decays[kChainWaves][64], values[kChainWaves][64];
  const int64_t size = static_cast<int64_t>(A.D) * A.dk, wide = (size + 63) / 64;
  const bool back = blockIdx.x >= blocks;
  const int64_t block = blockIdx.x - (back ? blocks : 0);
  const int64_t chain = block / wide, at = chain * A.S;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t e = min((block - chain * wide) * 64 + lane, size - 1);  // (the last one again)
  const int head = static_cast<int>(e / (A.dk * A.dv));
  const int ch = head * A.dv + static_cast<int>(e % A.dv);
  const float a2 = rate_of(A.a[e]);
  float* h = (back ? A.g : A.h) + at * size + e;
  const float* sum = A.sum + at * A.D + ch;
  const int* cut = (back ? A.cutr : A.cut) + at;
  // segment of the i-th place in the order of the chain; the last place's own
  // state is not asked for (and the forward's not there)
  const int last = A.S - 1;
  auto place = [&](int i) { return back ? last - i : i; };
  const int share = (A.S + kChainWaves - 1) / kChainWaves;
  const int lo = min(wave * share, A.S), hi = min(lo + share, A.S);
  // A decay below zero is a cut: nothing passes it, a NaN of another sequence
  // neither.
  auto join = [](float p, float state, float v) { return p < 0.f ? v : fmaf(p, state, v); };
  float v[U], p[U];
  auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = place(min(i0 + u, max(last - 1, 0)));
      v[u] = h[k * size];
      p[u] = cut[k] ? -1.f : decay(sum[static_cast<int64_t>(k) * A.D], a2);
    }
  };
  float all = 1.f, state = 0.f;
  for (int i = lo; i < hi; i += U) {
    load(i);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u >= hi) break;
      all = p[u] < 0.f || all < 0.f ? -1.f : all * p[u];
      state = join(p[u], state, v[u]);
    }
  }
  decays[wave][lane] = all;
  values[wave][lane] = state;
  __syncthreads();
  state = 0.f;
  for (int w = 0; w < wave; ++w) state = join(decays[w][lane], state, values[w][lane]);
  for (int i = lo; i < hi; i += U) {
    if (share > U) load(i);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u >= hi) break;
      if ((block - chain * wide) * 64 + lane < size) h[place(i + u) * size] = state;
      state = join(p[u], state, v[u]);
    }
  }
}

// ---------------------------------------------------------------- outputs ---

// The walk of the outputs.  WS > 1: every U tokens the waves of a channel
// block leave their sums over n in LDS and share the rows out.
template <typename IO, int NS, int WS, bool PAD, bool GATE>
__global__ __launch_bounds__(64 * waves_of(WS)) void scan_out_kernel(Args A) {
  constexpr int U = 4;
  const Span s = span_of(A, blockIdx.x / A.ublocks);
  const Runs rs = runs_of(A, s);
  const Lane<NS> l = lane_of<IO, NS, PAD>(A, WS);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t size = static_cast<int64_t>(A.D) * A.dk;
  __shared__ float meet[WS > 1 ? waves_of(WS) : 1][WS > 1 ? U : 1][64];
  for (int i = rs.cont ? 0 : 1; i <= rs.count; ++i) {
    const Run r = run_at(A, s, rs, i);
    float h[NS];
    enter<NS, PAD>(A, l, s, r, h);
    Rows<IO, U> x, dt, z{};
    typedef Ahead<IO, NS, PAD, U> ahead;
    ahead bs, cs;
    int left = static_cast<int>(r.hi - r.lo);
    x.load(A, A.x, r.lo, left, l.row);
    dt.load(A, A.dt, r.lo, left, l.row);
    if constexpr (GATE) z.load(A, A.z, r.lo, left, l.row);
    bs.start(row_of<IO>(A, l, A.b, r.lo), row_step<IO>(A), l.left, left);
    cs.start(row_of<IO>(A, l, A.c, r.lo), row_step<IO>(A), l.left, left);
    for (int64_t t = r.lo; left > 0; t += U, left -= U) {
      const Rows<IO, U> xs = x, dts = dt, zs = z;
      float y[U];
      x.load(A, A.x, t + U, left - U, l.row);
      dt.load(A, A.dt, t + U, left - U, l.row);
      if constexpr (GATE) z.load(A, A.z, t + U, left - U, l.row);
      auto ahead_of = [&](int at) {
        bs.take();
        cs.take();
        bs[0].arrive();
        bs.fetch(at, left);
        cs.fetch(at, left);
      };
      float delta[U];
#pragma unroll
      for (int u = 0; u < U; ++u) delta[u] = u < left ? step_of(A, dts[u], l.bias) : 0.f;
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (ahead::GROUP) ahead_of(U);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if constexpr (!ahead::GROUP) ahead_of(u + 1);
        const Row<IO, NS, PAD>&b = bs[u], &c = cs[u];
        const float dx = delta[u] * xs[u];
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          h[n] = fmaf(decay(delta[u], l.a2[n]), h[n], dx * b[n]);
          sum[n & 3] = fmaf(c[n], h[n], sum[n & 3]);
        }
        y[u] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
        __builtin_amdgcn_sched_barrier(0);
      }
      bs.group_done();
      cs.group_done();
      if constexpr (WS > 1) {
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) meet[wave][u][lane] = y[u];
        __syncthreads();
      }
      const RowsOut<IO, U> out(A, A.y, t, left);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (WS > 1 && u % WS != wave % WS) continue;
        float v = y[u];
        if constexpr (WS > 1) {
          v = meet[wave - wave % WS][u][lane];
#pragma unroll
          for (int k = 1; k < WS; ++k) v += meet[wave - wave % WS + k][u][lane];
        }
        v = fmaf(l.d, xs[u], v);
        if constexpr (GATE) v *= zs[u] * sigmoid<IO>(zs[u]);
        out.store(u, l.row, v);
      }
    }
    if (r.ends && A.sf != nullptr) store_state<NS, PAD>(A, l, A.sf + r.seq * size, h);
  }
}

// --------------------------------------------------------------- backward ---
//
// With dy_t the gradient of y_t in front of its gate and g_t that of S_t,
//
//   g_t[n] = c_t[n] dy_t + e^{delta_{t+1} a[n]} g_{t+1}[n]      (+ ds_final)
//   dc_t[n] = sum_j dy_t S_t[n],          db_t[n] = sum_j g_t[n] delta_t x_t
//   dx_t = delta_t sum_n g_t[n] b_t[n] + d dy_t
//   ddelta_t = sum_n g_t[n] (x_t b_t[n] + a[n] e^{delta_t a[n]} S_{t-1}[n])
//   da[n] = sum_t delta_t g_t[n] e^{delta_t a[n]} S_{t-1}[n]
//
// (j: the channels of a group).  The states are formed again: the walk of the
// segments leaves one for every tile of kScanTile tokens (from zero where the
// segment continues another; e^{a sum} of the state in front of the segment
// is added when it is read).  The gradient walk goes over the tiles from the
// last one back; a tile's states at every fourth token go to LDS, four
// tokens' decays and states stay in registers.

// As scan_local_kernel, over all runs: besides the segment's state its tiles'
// states, and what its first run makes of the gradient behind it.
template <typename IO, int NS, bool PAD, bool GATE>
__global__ __launch_bounds__(512) void scan_marks_kernel(Args A, int WS) {
  const Span s = span_of(A, blockIdx.x / A.ublocks);
  const Runs rs = runs_of(A, s);
  const Lane<NS> l = lane_of<IO, NS, PAD>(A, WS);
  const int64_t size = static_cast<int64_t>(A.D) * A.dk;
  float h[NS], g[NS], sum = 0.f, sumr = 0.f;
#pragma unroll
  for (int n = 0; n < NS; ++n) h[n] = g[n] = 0.f;
  bool cut = true, cutr = true;
  for (int i = rs.cont ? 0 : 1; i <= rs.count; ++i) {
    const Run r = run_at(A, s, rs, i);
    if (r.hi <= r.lo) continue;
    cut = !r.cont;
    sum = 0.f;
    if (r.cont) {
#pragma unroll
      for (int n = 0; n < NS; ++n) h[n] = 0.f;
    } else {
      enter<NS, PAD>(A, l, s, r, h);
    }
    float front[NS];  // decay from the run's start (only where it continues one)
#pragma unroll
    for (int n = 0; n < NS; ++n) front[n] = 1.f;
    auto mark = [&](int64_t t) {
      if (t == r.lo || (t - r.lo) % kScanTile != 0) return;
      const int64_t slot = t / kScanTile;
      store_state<NS, PAD>(A, l, A.mark + slot * size, h);
      if (l.live && l.n0 == 0) A.msum[slot * A.D + l.ch] = sum;
    };
    if (r.cont) {
      constexpr int U = 4;
      typedef Ahead<IO, NS, PAD, U> ahead;
      Rows<IO, U> dy, z{}, dys, zs{};
      ahead cs;
      const int all = static_cast<int>(r.hi - r.lo);
      dy.load(A, A.dy, r.lo, all, l.row);
      if constexpr (GATE) z.load(A, A.z, r.lo, all, l.row);
      cs.start(row_of<IO>(A, l, A.c, r.lo), row_step<IO>(A), l.left, all);
      walk<IO, NS, PAD>(A, l, r, [&](int64_t t, int left, const Rows<IO, U>& x, int u,
                                     float delta, const Row<IO, NS, PAD>& b) {
        if (u == 0) {
          mark(t);
          dys = dy;
          zs = z;
          dy.load(A, A.dy, t + U, left - U, l.row);
          if constexpr (GATE) z.load(A, A.z, t + U, left - U, l.row);
        }
        if (!ahead::GROUP || u == 0) {
          cs.take();
          cs.fetch(ahead::GROUP ? U : u + 1, left);
        }
        const Row<IO, NS, PAD>& c = cs[u];
        const float dx = delta * x[u];
        // (the gate first: of the type's lowest value it is zero, dy z infinite)
        const float v = GATE ? dys[u] * (zs[u] * sigmoid<IO>(zs[u])) : dys[u];
        sum += delta;
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          const float e = decay(delta, l.a2[n]);
          h[n] = fmaf(e, h[n], dx * b[n]);
          front[n] *= e;
          g[n] = fmaf(front[n], c[n] * v, g[n]);
        }
        if (u == U - 1) cs.group_done();
      });
    } else {
      walk<IO, NS, PAD>(A, l, r, [&](int64_t t, int, const Rows<IO, 4>& x, int u, float delta,
                                     const Row<IO, NS, PAD>& b) {
        if (u == 0) mark(t);
        const float dx = delta * x[u];
        sum += delta;
#pragma unroll
        for (int n = 0; n < NS; ++n) h[n] = fmaf(decay(delta, l.a2[n]), h[n], dx * b[n]);
      });
    }
    if (r.cont) {
      cutr = r.ends;
      sumr = sum;
      if (r.ends && A.ds != nullptr) {
        float v[NS];
        load_state<NS, PAD>(A, l, A.ds + r.seq * size, v);
#pragma unroll
        for (int n = 0; n < NS; ++n) g[n] = fmaf(front[n], v[n], g[n]);
      }
    }
  }
  if (A.S == 1) return;
  store_state<NS, PAD>(A, l, A.h + s.at * size, h);
  store_state<NS, PAD>(A, l, A.g + s.at * size, g);
  // (one run over the whole segment, or both directions are cut)
  if (l.live && l.n0 == 0) A.sum[static_cast<int64_t>(s.at) * A.D + l.ch] = cut ? sumr : sum;
  if (blockIdx.x % A.ublocks == 0 && threadIdx.x == 0) {
    A.cut[s.at] = cut;
    A.cutr[s.at] = cutr;
  }
}

template <int CTRL>
__device__ inline float lane_of_other(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}

// Sums over lanes of two values at once: each half of the lanes goes on with
// one of them.  (The matrix cores can add lanes up too, as products with unit
// vectors; their fp32 products take the vector unit's time: the gradient walk
// of 16384 tokens of 4096 channels went from 1000 to 1390 us.)
//
// Lanes 8 and 4 apart: r = a + a of the other lane, then the same of b in the
// banks of four lanes that have the bit, an add each, where a swap of halves
// takes two adds' time in front of its add; so these two steps, which halve
// the most values, come first.  Both adds are written out: a masked one keeps
// its old lanes only so, and the other would be torn up for a product that is
// one of its operands.  These instructions and the swaps read a register two
// states after its write at the earliest.  (The lane 4 apart differs in its
// lower bits too, which later steps add up.)
template <int BIT, int N>
__device__ inline void fold_banks(const float (&a)[N], const float (&b)[N], float (&r)[N]) {
  static_assert((BIT == 8 || BIT == 4) && (N == 8 || N == 4), "");
#define GDN_ADD(r, a, how, banks) "v_add_f32_dpp " r ", " a ", " a " " how " row_mask:0xf bank_mask:" banks "\n"
#define GDN_8(how, up)                                                                         \
  asm("s_nop 1\n" GDN_ADD("%0", "%8", how, "0xf") GDN_ADD("%1", "%9", how, "0xf")              \
          GDN_ADD("%2", "%10", how, "0xf") GDN_ADD("%3", "%11", how, "0xf")                    \
          GDN_ADD("%4", "%12", how, "0xf") GDN_ADD("%5", "%13", how, "0xf")                    \
          GDN_ADD("%6", "%14", how, "0xf") GDN_ADD("%7", "%15", how, "0xf")                    \
          GDN_ADD("%0", "%16", how, up) GDN_ADD("%1", "%17", how, up)                          \
          GDN_ADD("%2", "%18", how, up) GDN_ADD("%3", "%19", how, up)                          \
          GDN_ADD("%4", "%20", how, up) GDN_ADD("%5", "%21", how, up)                          \
          GDN_ADD("%6", "%22", how, up) GDN_ADD("%7", "%23", how, up) "s_nop 1"                \
      : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]),          \
        "=&v"(r[6]), "=&v"(r[7])                                                               \
      : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "v"(a[4]), "v"(a[5]), "v"(a[6]),           \
        "v"(a[7]), "v"(b[0]), "v"(b[1]), "v"(b[2]), "v"(b[3]), "v"(b[4]), "v"(b[5]),           \
        "v"(b[6]), "v"(b[7]))
#define GDN_4(how, up)                                                                         \
  asm("s_nop 1\n" GDN_ADD("%0", "%4", how, "0xf") GDN_ADD("%1", "%5", how, "0xf")              \
          GDN_ADD("%2", "%6", how, "0xf") GDN_ADD("%3", "%7", how, "0xf")                      \
          GDN_ADD("%0", "%8", how, up) GDN_ADD("%1", "%9", how, up)                            \
          GDN_ADD("%2", "%10", how, up) GDN_ADD("%3", "%11", how, up) "s_nop 1"                \
      : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3])                                     \
      : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "v"(b[0]), "v"(b[1]), "v"(b[2]), "v"(b[3]))
  if constexpr (N == 8) {
    if constexpr (BIT == 8) GDN_8("row_ror:8", "0xc");
    else GDN_8("row_half_mirror", "0xa");
  } else {
    if constexpr (BIT == 8) GDN_4("row_ror:8", "0xc");
    else GDN_4("row_half_mirror", "0xa");
  }
#undef GDN_4
#undef GDN_8
#undef GDN_ADD
}
__device__ inline float fold32(float a, float b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false,
                                                  false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ inline float fold16(float a, float b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false,
                                                  false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// Lanes 2 and 1 apart.
template <int BIT>
__device__ inline float fold(float a, float b) {
  const bool up = threadIdx.x & BIT;
  const float keep = up ? b : a, send = up ? a : b;
  return keep + lane_of_other<BIT == 2 ? 0x1b : 0xb1>(send);
}

// The gradient walk.
template <typename IO, int NS, int WS, bool PAD, bool GATE>
__global__ __launch_bounds__(64 * waves_of(WS), 2) void scan_grad_kernel(Args A) {
  constexpr int U = 4, Q = kScanTile / U, N = PAD || NS < 8 ? 4 : 8;
  __shared__ floatx4 marks[waves_of(WS)][Q][NS / 4][64];
  __shared__ float meet[WS > 1 ? waves_of(WS) : 1][WS > 1 ? U : 1][3][64];
  const Span s = span_of(A, blockIdx.x / A.ublocks);
  const Runs rs = runs_of(A, s);
  const Lane<NS> l = lane_of<IO, NS, PAD>(A, WS);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool real = blockIdx.x % A.ublocks * (waves_of(WS) / WS) + wave / WS < A.units;
  const int64_t size = static_cast<int64_t>(A.D) * A.dk;
  const int step = row_step<IO>(A);
  float da[NS], dd = 0.f, dbias = 0.f;
#pragma unroll
  for (int n = 0; n < NS; ++n) da[n] = 0.f;

  for (int i = rs.count; i >= (rs.cont ? 0 : 1); --i) {
    const Run r = run_at(A, s, rs, i);
    float g[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) g[n] = 0.f;
    if (!r.ends) load_state<NS, PAD>(A, l, A.g + s.at * size, g);
    else if (A.ds != nullptr) load_state<NS, PAD>(A, l, A.ds + r.seq * size, g);

    const int tiles = static_cast<int>((r.hi - r.lo + kScanTile - 1) / kScanTile);
    Rows<IO, U> next[4];  // the rows of the next block: x, dt, dy, z
    auto rows = [&](int64_t t, int left) {
      next[0].load(A, A.x, t, left, l.row);
      next[1].load(A, A.dt, t, left, l.row);
      next[2].load(A, A.dy, t, left, l.row);
      if constexpr (GATE) next[3].load(A, A.z, t, left, l.row);
    };
    if (tiles > 0) {
      const int64_t t = r.lo + (r.hi - r.lo - 1) / U * U;
      rows(t, static_cast<int>(r.hi - t));
    }
    for (int k = tiles - 1; k >= 0; --k) {
      const int64_t t0 = r.lo + k * kScanTile;
      const int count = static_cast<int>(r.hi - t0 < kScanTile ? r.hi - t0 : kScanTile);
      const int blocks = (count + U - 1) / U;
      {
        // the tile's states at every fourth token
        float h[NS];
        if (k == 0) {
          enter<NS, PAD>(A, l, s, r, h);
        } else {
          const int64_t slot = t0 / kScanTile;
          load_state<NS, PAD>(A, l, A.mark + slot * size, h);
          if (r.cont) {
            const float sum = A.msum[slot * A.D + l.ch];
            float f[NS];
            enter<NS, PAD>(A, l, s, r, f);
#pragma unroll
            for (int n = 0; n < NS; ++n) h[n] = fmaf(decay(sum, l.a2[n]), f[n], h[n]);
          }
        }
        Rows<IO, U> wx[Q - 1], wdt[Q - 1];
#pragma unroll
        for (int q = 0; q < Q - 1; ++q) {
          wx[q].load(A, A.x, t0 + q * U, count - (q + 1) * U > 0 ? U : 0, l.row);
          wdt[q].load(A, A.dt, t0 + q * U, count - (q + 1) * U > 0 ? U : 0, l.row);
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) {
#pragma unroll
          for (int n = 0; n < NS; n += 4)
            marks[wave][q][n / 4][lane] = floatx4{h[n], h[n + 1], h[n + 2], h[n + 3]};
          if (q + 1 >= blocks) break;
          const int64_t t = t0 + q * U;
          const Rows<IO, U>&x = wx[q < Q - 1 ? q : 0], &dt = wdt[q < Q - 1 ? q : 0];
          Row<IO, NS, PAD> next;
          const uintptr_t from = row_of<IO>(A, l, A.b, t);
          next.load(from, l.left);
          float delta[U];
#pragma unroll
          for (int u = 0; u < U; ++u) delta[u] = step_of(A, dt[u], l.bias);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const Row<IO, NS, PAD> b = next;
            b.arrive();
            next.load(from + min(u + 1, U - 1) * step, l.left);
            const float dx = delta[u] * x[u];
#pragma unroll
            for (int n = 0; n < NS; ++n) h[n] = fmaf(decay(delta[u], l.a2[n]), h[n], dx * b[n]);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
      for (int q = blocks - 1; q >= 0; --q) {
        // rows past the run are its last one's, with delta = x = dy = 0: the
        // state and its gradient pass through them unchanged
        const int64_t t = t0 + q * U;
        const int left = static_cast<int>(r.hi - t < U ? r.hi - t : U);
        const Rows<IO, U> x = next[0], pre = next[1], dout = next[2], z = next[GATE ? 3 : 0];
        rows(t - U, t > r.lo ? U : 0);  // (the block in front is a whole one)
        const uintptr_t fromb = row_of<IO>(A, l, A.b, t), fromc = row_of<IO>(A, l, A.c, t);
        float delta[U], dx[U], dy[U], slope[U], gb[U], ga[U], ys[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          delta[u] = u < left ? step_of(A, pre[u], l.bias) : 0.f;
          dx[u] = delta[u] * x[u];
          dy[u] = dout[u];
          if constexpr (GATE) {
            const float sg = sigmoid<IO>(z[u]);
            dy[u] *= z[u] * sg;
            slope[u] = dout[u] * (sg * (1.f + z[u] * (1.f - sg)));
          }
          gb[u] = ga[u] = ys[u] = 0.f;
        }
#pragma unroll
        for (int n0 = 0; n0 < NS; n0 += N) {
          Row<IO, N, PAD> b[U], c[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int at = min(u, left - 1) * step + n0 * io<IO>::bytes;
            b[u].load(fromb + at, l.left - n0);
            c[u].load(fromc + at, l.left - n0);
          }
          float e[U][N], h[U + 1][N];  // decays, states in front of and behind the tokens
#pragma unroll
          for (int n = 0; n < N; n += 4) {
            const floatx4 v = marks[wave][q][(n0 + n) / 4][lane];
#pragma unroll
            for (int m = 0; m < 4; ++m) h[0][n + m] = v[m];
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int n = 0; n < N; ++n) {
              e[u][n] = decay(delta[u], l.a2[n0 + n]);
              h[u + 1][n] = fmaf(e[u][n], h[u][n], dx[u] * b[u][n]);
            }
          }
#pragma unroll
          for (int u = 0; u < U; ++u) b[u].pack();
          float pair[2][N], four[2][N];  // of a token, of two tokens
#pragma unroll
          for (int u = U - 1; u >= 0; --u) {
            float vb[N], vc[N];
#pragma unroll
            for (int n = 0; n < N; ++n) {
              float& gn = g[n0 + n];
              gn = fmaf(c[u][n], dy[u], gn);
              vb[n] = gn * dx[u];
              vc[n] = h[u + 1][n] * dy[u];
              if constexpr (GATE) ys[u] = fmaf(c[u][n], h[u + 1][n], ys[u]);
              gb[u] = fmaf(b[u][n], gn, gb[u]);
              gn *= e[u][n];
              const float w = gn * h[u][n];
              da[n0 + n] = fmaf(delta[u], w, da[n0 + n]);
              ga[u] = fmaf(l.a2[n0 + n], w, ga[u]);
            }
            fold_banks<8>(vb, vc, pair[u & 1]);
            if ((u & 1) == 0) fold_banks<4>(pair[0], pair[1], four[u >> 1]);
          }
          // (kept here: sums that only the outputs use are else formed there,
          // from operands kept until then)
#pragma unroll
          for (int u = 0; u < U; ++u) {
            asm volatile("" : "+v"(gb[u]), "+v"(ga[u]));
            if constexpr (GATE) asm volatile("" : "+v"(ys[u]));
          }
          // lane bits: 8 which of db, dc; 4 and 32 the token of the block; the
          // others the state
          float v[N], sum;
#pragma unroll
          for (int n = 0; n < N; ++n) v[n] = fold32(four[0][n], four[1][n]);
#pragma unroll
          for (int n = 0; n < N / 2; ++n) v[n] = fold16(v[n], v[n + N / 2]);
          int n = (lane >> 4) & 1;
          bool own = real;
          if constexpr (N == 8) {
#pragma unroll
            for (int m = 0; m < 2; ++m) v[m] = fold<2>(v[m], v[m + 2]);
            sum = fold<1>(v[0], v[1]);
            n = n * 4 + (lane & 3);
          } else {
            sum = fold<2>(v[0], v[1]);
            sum += lane_of_other<0xb1>(sum);
            n = n * 2 + ((lane >> 1) & 1);
            own = own && (lane & 1) == 0;
          }
          const int at = ((lane >> 2) & 1) + (lane >> 5) * 2;
          if (own && at < left)
            A.part[(((t + at) * A.units + l.unit) * WS + wave % WS) * (2 * NS) +
                   ((lane >> 3) & 1) * NS +
                   n0 + n] = sum;
          __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (WS > 1) {
          __syncthreads();
#pragma unroll
          for (int u = 0; u < U; ++u) {
            meet[wave][u][0][lane] = gb[u];
            meet[wave][u][1][lane] = ga[u];
            if constexpr (GATE) meet[wave][u][2][lane] = ys[u];
          }
          __syncthreads();
        }
        const RowsOut<IO, U> outx(A, A.dx, t, left), outt(A, A.ddt, t, left);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (WS > 1 && u % WS != wave % WS) continue;
          float vb = gb[u], va = ga[u], vy = ys[u];
          if constexpr (WS > 1) {
            vb = va = vy = 0.f;
#pragma unroll
            for (int w = 0; w < WS; ++w) {
              vb += meet[wave - wave % WS + w][u][0][lane];
              va += meet[wave - wave % WS + w][u][1][lane];
              if constexpr (GATE) vy += meet[wave - wave % WS + w][u][2][lane];
            }
          }
          float v = fmaf(x[u], vb, kLn2 * va);
          const float rise = sigmoid<IO>(pre[u] + l.bias);
          v *= A.softplus ? rise : 1.f;
          dd = fmaf(dy[u], x[u], dd);
          dbias += u < left ? v : 0.f;
          outx.store(u, l.row, fmaf(l.d, dy[u], delta[u] * vb));
          outt.store(u, l.row, v);
          if constexpr (GATE)
            RowsOut<IO, U>(A, A.dz, t, left).store(u, l.row, slope[u] * fmaf(l.d, x[u], vy));
        }
      }
    }
    if (!r.cont && A.ds0 != nullptr) store_state<NS, PAD>(A, l, A.ds0 + r.seq * size, g);
  }
  store_state<NS, PAD>(A, l, A.pa + s.at * size, da);
  if (l.live) {
    const int64_t row = static_cast<int64_t>(s.at) * WS + wave % WS;
    A.pd[row * A.D + l.ch] = dd;
    A.pb[row * A.D + l.ch] = dbias;
  }
}

// The shares of the gradient walk added in a fixed order, one launch for all:
// db, dc (the channel blocks' of every token, group and state; a thread each;
// rows in front of the first sequence and behind the last one, of which there
// are no shares, stay as they are), then da, dd, dt_bias (rows of shares;
// sixteen columns a workgroup, its sixteen runs of rows added up in LDS).
struct Finish {
  int64_t tokens;
  int NS, WS;
  int64_t rows;            // segments
  unsigned first[4];       // first workgroup of each part: da, dd, dbias, the end
  void *db, *dc;
  float *da, *dd, *dbias;
};

template <typename IO>
__global__ __launch_bounds__(256) void scan_finish_kernel(Args A, Finish F) {
  if (blockIdx.x < F.first[0]) {
    const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int per = 2 * A.dk;
    const int64_t row = e / per;  // token and group
    if (row >= F.tokens * A.hb) return;
    if (A.cu != nullptr && (row < bound(A, 0) * A.hb || row >= bound(A, A.nseq) * A.hb)) return;
    const int k = static_cast<int>(e - row * per), n = k % A.dk, two = k / A.dk;
    const int unit = F.WS * 2 * F.NS;
    const float* p = A.part + row * A.nb * unit + n / F.NS * (2 * F.NS) + two * F.NS + n % F.NS;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    for (int u = 0; u < A.nb; u += 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (u + i < A.nb) s[i] += p[static_cast<int64_t>(u + i) * unit];
    }
    io<IO>::store(two ? F.dc : F.db, row * A.dk + n, (s[0] + s[1]) + (s[2] + s[3]));
    return;
  }
  const int which = blockIdx.x < F.first[1] ? 0 : blockIdx.x < F.first[2] ? 1 : 2;
  const float* part = which == 0 ? A.pa : which == 1 ? A.pd : A.pb;
  float* out = which == 0 ? F.da : which == 1 ? F.dd : F.dbias;
  const int64_t rows = which == 0 ? F.rows : F.rows * F.WS;
  const int64_t cols = which == 0 ? static_cast<int64_t>(A.D) * A.dk : A.D;
  const int lc = threadIdx.x & 15, run = threadIdx.x >> 4;
  const int64_t c = static_cast<int64_t>(blockIdx.x - F.first[which]) * 16 + lc;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (c < cols) {
    for (int64_t k = run; k < rows; k += 64) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (k + 16 * u < rows) s[u] += part[(k + 16 * u) * cols + c];
    }
  }
  __shared__ float t[16][17];
  t[run][lc] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  if (run != 0 || c >= cols) return;
  float v = t[0][lc];
#pragma unroll
  for (int k = 1; k < 16; ++k) v += t[k][lc];
  out[c] = v;
}

// ------------------------------------------------------------------- step ---

// One token of every sequence: a thread owns V adjacent channels of one head
// and reads and writes each of their states once, sixteen of them (and their
// rates) in flight at a time; memory bounds it.
template <typename IO, int V>
__device__ inline void load_row(const void* p, int64_t at, float* x) {
  if constexpr (V == 1) {
    x[0] = io<IO>::load(p, at);
  } else if constexpr (io<IO>::bytes == 2) {
    typedef __bf16 vec __attribute__((ext_vector_type(V)));
    const vec v = *reinterpret_cast<const vec*>(static_cast<const __bf16*>(p) + at);
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = static_cast<float>(v[e]);
  } else {
    typedef float vec __attribute__((ext_vector_type(V)));
    const vec v = *reinterpret_cast<const vec*>(static_cast<const float*>(p) + at);
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = v[e];
  }
}

template <typename IO, int V>
__global__ __launch_bounds__(256) void scan_step_kernel(Args A, int64_t threads) {
  typedef float vec __attribute__((ext_vector_type(V)));
  constexpr int N = 16;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (id >= threads) return;
  const int row = A.D / V;  // threads of a sequence
  const int64_t q = id / row;
  const int ch = static_cast<int>(id - q * row) * V;
  const int head = ch / A.dv, grp = ch / A.Dg;
  const int state = head * A.dk * A.dv + ch - head * A.dv;
  float* p = A.sf + q * A.D * A.dk + state;
  const float* rate = A.a + state;
  const int64_t bc = (q * A.hb + grp) * A.dk;
  float x[V], z[V], delta[V], dx[V], y[V];
  load_row<IO, V>(A.x, q * A.D + ch, x);
  load_row<IO, V>(A.dt, q * A.D + ch, delta);
  if (A.z != nullptr) load_row<IO, V>(A.z, q * A.D + ch, z);
#pragma unroll
  for (int v = 0; v < V; ++v) y[v] = A.d ? A.d[ch + v] * x[v] : 0.f;
  for (int n0 = 0; n0 < A.dk; n0 += N) {
    vec h[N], a[N];
    float b[N], c[N];
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const int n = min(n0 + i, A.dk - 4);  // (the last ones again, not used)
      load_row<IO, 4>(A.b, bc + n, b + i);
      load_row<IO, 4>(A.c, bc + n, c + i);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        h[i + k] = *reinterpret_cast<const vec*>(p + (n + k) * A.dv);
        a[i + k] = *reinterpret_cast<const vec*>(rate + (n + k) * A.dv);
      }
    }
    if (n0 == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        delta[v] = step_of(A, delta[v], A.bias ? A.bias[ch + v] : 0.f);
        dx[v] = delta[v] * x[v];
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (n0 + i >= A.dk) break;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        h[i][v] = fmaf(decay(delta[v], rate_of(a[i][v])), h[i][v], dx[v] * b[i]);
        y[v] = fmaf(c[i], h[i][v], y[v]);
      }
      *reinterpret_cast<vec*>(p + (n0 + i) * A.dv) = h[i];
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (A.z != nullptr) y[v] *= z[v] * sigmoid<IO>(z[v]);
    store_x<IO>(A.y, A, q, ch + v, y[v]);
  }
}

// ------------------------------------------------------------------- plan ---

struct Plan {
  int ns, ws;       // states a lane, waves for a channel's states
  bool pad;
  int chains;       // sequences (packed: 1)
  int64_t len;      // tokens of a chain
  int units;        // channel blocks
  int S, L;
  int64_t segs;     // chains * S
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

Plan plan_scan(const Scan& p) {
  Plan q;
  q.chains = p.varlen ? 1 : p.B;
  q.len = p.T;
  const int64_t D = static_cast<int64_t>(p.H) * p.dv, Dg = D / p.hb;
  q.units = static_cast<int>(p.hb * ceil_div(Dg, 64));
  q.ns = p.dk <= 4 ? 4 : p.dk <= 8 ? 8 : 16;
  auto split = [&] {
    q.ws = 1;
    while (q.ws * q.ns < p.dk) q.ws *= 2;
  };
  split();
  // Segments: eight waves a SIMD to choose from hide the loads (forward of
  // 16384 packed tokens of 4096 channels: 428 us with four, 419 with six, 402;
  // of 65536 tokens of 2048: 825, 814, 780; backward of 16384 of 4096: 1267,
  // 1289, 1260, but of 8 x 2048 of 1024 376, 411, 388), but not below half the
  // square root of the tokens, where the chaining takes over (4096 tokens of
  // 2048 channels: 86 us from a quarter, 74 from half, 77 from the whole root).
  // Up to 96 tokens stay whole: batches fill the machine by themselves (64
  // sequences of 96 tokens of 128 channels: 26.5 us, in segments of 16 39.2;
  // backward 86 and 89), and a short sequence takes less than three launches
  // (64 tokens of 32 channels 17.3 us, cut 18.3).  One sequence alone would gain
  // from about 80 tokens on (96: 24.4 and 18.5), its backward from 32 on (64:
  // 58 and 31, 96: 82 and 31).
  int64_t L;
  if (p.seg_req < 0) {
    L = q.len;
  } else if (p.seg_req > 0) {
    L = static_cast<int64_t>(std::min(p.seg_req, 1 << 20)) * kScanTile;
  } else {
    const int64_t waves = static_cast<int64_t>(q.chains) * q.units * q.ws;
    const int64_t want = std::max<int64_t>(1, ceil_div(8192, waves));  // segments of a chain
    L = std::max<int64_t>(ceil_div(q.len, want),
                          static_cast<int64_t>(0.5 * std::sqrt(static_cast<double>(q.len))));
    L = std::max<int64_t>(ceil_div(L, kScanTile) * kScanTile, kScanTile);
    if (q.len <= 96) L = q.len;
  }
  if (L >= q.len) L = std::max<int64_t>(q.len, 1);
  q.L = static_cast<int>(L);
  q.S = static_cast<int>(std::max<int64_t>(1, ceil_div(q.len, L)));
  q.segs = static_cast<int64_t>(q.chains) * q.S;
  // Few waves: a channel's states are shared out over more of them, so that
  // a token takes less time.
  while (q.ns > 4 && q.ws < 8 && q.segs * q.units * q.ws < 512) {
    q.ns /= 2;
    split();
  }
  q.pad = p.dk != q.ns * q.ws;
  return q;
}

size_t al256(size_t x) { return (x + 255) & ~size_t(255); }

struct Carve {  // pieces of a workspace, or their total when base is 0
  uintptr_t base;
  size_t used;
  template <typename T>
  T* take(int64_t n) {
    T* p = reinterpret_cast<T*>(base + used);
    used += al256(static_cast<size_t>(n) * sizeof(T));
    return p;
  }
};

size_t carve_fwd(const Scan& p, const Plan& q, char* ws, Args* A) {
  if (q.S == 1) return 0;
  const int64_t D = static_cast<int64_t>(p.H) * p.dv;
  Carve c{reinterpret_cast<uintptr_t>(ws), 0};
  A->cut = c.take<int>(q.segs);
  A->h = c.take<float>(q.segs * D * p.dk);
  A->sum = c.take<float>(q.segs * D);
  return c.used;
}

size_t carve_bwd(const Scan& p, const Plan& q, char* ws, Args* A) {
  const int64_t D = static_cast<int64_t>(p.H) * p.dv, size = D * p.dk;
  const int64_t tokens = static_cast<int64_t>(p.B) * p.T;
  Carve c{reinterpret_cast<uintptr_t>(ws), 0};
  if (q.S > 1) {
    A->cut = c.take<int>(q.segs);
    A->cutr = c.take<int>(q.segs);
    A->h = c.take<float>(q.segs * size);
    A->g = c.take<float>(q.segs * size);
    A->sum = c.take<float>(q.segs * D);
  }
  const int64_t marks = tokens / kScanTile + 1;
  A->mark = c.take<float>(marks * size);
  A->msum = c.take<float>(marks * D);
  A->part = c.take<float>(tokens * q.units * q.ws * 2 * q.ns);
  A->pa = c.take<float>(q.segs * size);
  A->pd = c.take<float>(q.segs * q.ws * D);
  A->pb = c.take<float>(q.segs * q.ws * D);
  return c.used;
}

Args make_args(const Scan& p, const Plan& q, const ScanIn& in) {
  Args A{};
  A.x = in.x;
  A.dt = in.dt;
  A.a = in.a;
  A.b = in.b;
  A.c = in.c;
  A.d = in.d;
  A.bias = in.bias;
  A.z = in.z;
  A.s0 = in.s0;
  A.T = q.len;
  A.D = p.H * p.dv;
  A.Dg = A.D / p.hb;
  A.nb = (A.Dg + 63) / 64;
  A.units = q.units;
  A.ublocks = static_cast<int>(ceil_div(q.units, waves_of(q.ws) / q.ws));
  A.dk = p.dk;
  A.dv = p.dv;
  A.hb = p.hb;
  A.S = q.S;
  A.L = q.L;
  A.nseq = p.nseq;
  A.softplus = p.softplus ? 1 : 0;
  A.cu = p.varlen ? p.cu_seqlens : nullptr;
  return A;
}

template <typename IO, int NS, bool PAD>
void launch_local(const Args& A, const Plan& q, int64_t segs, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(A.ublocks * segs));
  hipLaunchKernelGGL((scan_local_kernel<IO, NS, PAD>), grid, dim3(64 * waves_of(q.ws)), 0, s, A,
                     q.ws);
}

template <typename IO, int NS, int WS, bool PAD, bool GATE>
void launch_out(const Args& A, const Plan& q, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(A.ublocks * q.segs));
  hipLaunchKernelGGL((scan_out_kernel<IO, NS, WS, PAD, GATE>), grid, dim3(64 * waves_of(WS)), 0,
                     s, A);
}

void launch_chain(const Args& A, const Plan& q, int ways, hipStream_t s) {
  const int64_t blocks = ceil_div(static_cast<int64_t>(A.D) * A.dk, 64) * q.chains;
  hipLaunchKernelGGL(scan_chain_kernel, dim3(static_cast<unsigned>(ways * blocks)),
                     dim3(64 * kChainWaves), 0, s, A, blocks);
}

// Calls f<NS, WS, PAD, GATE> of a plan.
template <typename F>
void with_plan(const Plan& q, bool gate, F f) {
  using std::integral_constant;
  auto all = [&](auto ns, auto ws, auto pad) {
    if (gate) f(ns, ws, pad, std::true_type{});
    else f(ns, ws, pad, std::false_type{});
  };
  auto pads = [&](auto ns, auto ws) {
    if (!q.pad) return all(ns, ws, std::false_type{});
    if constexpr (ns * ws > 8) all(ns, ws, std::true_type{});  // (4 and 8 states are whole)
  };
  auto waves = [&](auto ns) {
    if (q.ws == 1) return pads(ns, integral_constant<int, 1>{});
    if (q.ws == 2) return pads(ns, integral_constant<int, 2>{});
    if constexpr (ns < 16) {
      if (q.ws == 8) return pads(ns, integral_constant<int, 8>{});
    }
    pads(ns, integral_constant<int, 4>{});
  };
  if (q.ns == 4) return waves(integral_constant<int, 4>{});
  if (q.ns == 8) return waves(integral_constant<int, 8>{});
  waves(integral_constant<int, 16>{});
}

template <typename IO>
hipError_t scan_fwd(const Plan& q, const Args& A, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (q.S > 1) {
    {
      StageScope scope(GDN_STAGE_FWD_TRANS, s);
      with_plan(q, false, [&](auto ns, auto, auto pad, auto) {
        launch_local<IO, ns, pad>(A, q, static_cast<int64_t>(q.chains) * (q.S - 1), s);
      });
      e = hipGetLastError();
    }
    if (e != hipSuccess) return e;
    {
      StageScope scope(GDN_STAGE_FWD_COMBINE, s);
      launch_chain(A, q, 1, s);
      e = hipGetLastError();
    }
    if (e != hipSuccess) return e;
  }
  StageScope scope(GDN_STAGE_FWD_SCAN, s);
  with_plan(q, A.z != nullptr, [&](auto ns, auto ws, auto pad, auto gate) {
    launch_out<IO, ns, ws, pad, gate>(A, q, s);
  });
  return hipGetLastError();
}

template <typename IO>
hipError_t scan_bwd(const Plan& q, const Args& A, int64_t tokens, const ScanGrad& out,
                    hipStream_t s) {
  const int64_t size = static_cast<int64_t>(A.D) * A.dk;
  hipError_t e;
  {
    StageScope scope(GDN_STAGE_BWD_STATES, s);
    with_plan(q, A.z != nullptr, [&](auto ns, auto, auto pad, auto gate) {
      hipLaunchKernelGGL((scan_marks_kernel<IO, ns, pad, gate>),
                         dim3(static_cast<unsigned>(A.ublocks * q.segs)),
                         dim3(64 * waves_of(q.ws)), 0, s, A, q.ws);
    });
    e = hipGetLastError();
  }
  if (e != hipSuccess) return e;
  if (q.S > 1) {
    StageScope scope(GDN_STAGE_BWD_SCAN, s);
    launch_chain(A, q, 2, s);
    e = hipGetLastError();
  }
  if (e != hipSuccess) return e;
  StageScope scope(GDN_STAGE_BWD_GRAD, s);
  with_plan(q, A.z != nullptr, [&](auto ns, auto ws, auto pad, auto gate) {
    hipLaunchKernelGGL((scan_grad_kernel<IO, ns, ws, pad, gate>),
                       dim3(static_cast<unsigned>(A.ublocks * q.segs)), dim3(64 * waves_of(ws)), 0,
                       s, A);
  });
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  Finish F{tokens, q.ns, q.ws, q.segs, {}, out.db, out.dc, out.da, out.dd, out.dbias};
  F.first[0] = static_cast<unsigned>(ceil_div(tokens * A.hb * 2 * A.dk, 256));
  F.first[1] = F.first[0] + static_cast<unsigned>(ceil_div(size, 16));
  F.first[2] = F.first[1] + (out.dd != nullptr ? static_cast<unsigned>(ceil_div(A.D, 16)) : 0);
  F.first[3] = F.first[2] + (out.dbias != nullptr ? static_cast<unsigned>(ceil_div(A.D, 16)) : 0);
  hipLaunchKernelGGL((scan_finish_kernel<IO>), dim3(F.first[3]), dim3(256), 0, s, A, F);
  return hipGetLastError();
}

}  // namespace

bool scan_fits(const Scan& p) {
  // every launch below 2^32 threads
  const Plan q = plan_scan(p);
  const int64_t most = (int64_t(1) << 32) - 1;
  const int64_t state = ceil_div(static_cast<int64_t>(p.H) * p.dv * p.dk, 64);
  const int64_t rows = static_cast<int64_t>(p.B) * p.T;
  const int64_t unit = ceil_div(q.units, waves_of(q.ws) / q.ws) * 64 * waves_of(q.ws);
  return q.segs <= most / unit && q.chains <= most / (2 * 64 * kChainWaves) / state &&
         rows * p.hb * 2 * p.dk + 16 * (state * 64 + 2 * static_cast<int64_t>(p.H) * p.dv) + 1024 <=
             most;
}

size_t scan_fwd_workspace_bytes(const Scan& p) {
  Args A{};
  return carve_fwd(p, plan_scan(p), nullptr, &A);
}

hipError_t launch_scan_fwd(const Scan& p, const ScanIn& in, void* y, float* s_final, void* ws,
                           hipStream_t s) {
  const Plan q = plan_scan(p);
  Args A = make_args(p, q, in);
  carve_fwd(p, q, static_cast<char*>(ws), &A);
  A.y = y;
  A.sf = s_final;
  return p.io == GDN_BF16 ? scan_fwd<bf16_t>(q, A, s) : scan_fwd<f32_t>(q, A, s);
}

size_t scan_bwd_workspace_bytes(const Scan& p) {
  Args A{};
  return carve_bwd(p, plan_scan(p), nullptr, &A);
}

hipError_t launch_scan_bwd(const Scan& p, const ScanIn& in, const void* dy, const float* ds_final,
                           const ScanGrad& out, void* ws, hipStream_t s) {
  const Plan q = plan_scan(p);
  Args A = make_args(p, q, in);
  carve_bwd(p, q, static_cast<char*>(ws), &A);
  A.dy = dy;
  A.ds = ds_final;
  A.dx = out.dx;
  A.ddt = out.ddt;
  A.dz = out.dz;
  A.ds0 = out.ds0;
  const int64_t tokens = static_cast<int64_t>(p.B) * p.T;
  return p.io == GDN_BF16 ? scan_bwd<bf16_t>(q, A, tokens, out, s)
                          : scan_bwd<f32_t>(q, A, tokens, out, s);
}

hipError_t launch_scan_step(const Scan& p, const ScanIn& in, float* state, void* y,
                            hipStream_t s) {
  Args A = make_args(p, plan_scan(p), in);
  A.y = y;
  A.sf = state;
  // four channels a thread where that leaves threads enough to keep the memory
  // busy, else one
  const int V = p.dv % 4 == 0 && static_cast<int64_t>(A.D) * p.nseq >= (1 << 17) ? 4 : 1;
  const int64_t threads = static_cast<int64_t>(A.D / V) * p.nseq;
  const dim3 grid(static_cast<unsigned>(ceil_div(threads, 256)));
  StageScope scope(GDN_STAGE_DECODE, s);
  auto go = [&](auto io_tag) {
    using IO = decltype(io_tag);
    if (V == 4) hipLaunchKernelGGL((scan_step_kernel<IO, 4>), grid, dim3(256), 0, s, A, threads);
    else hipLaunchKernelGGL((scan_step_kernel<IO, 1>), grid, dim3(256), 0, s, A, threads);
  };
  if (p.io == GDN_BF16) go(bf16_t{});
  else go(f32_t{});
  return hipGetLastError();
}

}  // namespace gdn
