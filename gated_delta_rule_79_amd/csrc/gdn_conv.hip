// Short causal depthwise convolution with a carried history, its backward and
// its single-token step: for every channel
//
//   p_t = bias + sum_{j < W} taps[j] x_{t - j},   y_t = act(p_t)
//
// where inputs in front of a sequence's first are its history s0 (the W - 1
// last inputs, oldest first) or zeros.  Backward, with e_t = dy_t act'(p_t):
//
//   dx_t = sum_j taps[j] e_{t + j} (+ ds_final),  dtaps[j] = sum_t e_t x_{t - j},
//   dbias = sum_t e_t
//
// A thread owns V adjacent channels (one 16-byte piece where the row allows
// it) and walks a run of tokens with the last W - 1 inputs in registers, so
// every row is read once and memory bounds the pass: the forward of 16384
// tokens of 4096 channels in bf16, width 4, 53 us with its inputs in cache, 60
// without (5.1, 4.5 TB/s).  The backward (16384 tokens of 1024 channels: 33 and
// 39 us, 3.1 and 2.6 TB/s) fills neither: its 512 workgroups are two waves a
// SIMD, with which the vector unit is 52 % busy, and more of them leave more
// shares of dtaps and dbias to add (kBwdBlocks).  Runs lie on the grid of
// all tokens; a walk that meets a sequence's end takes up the next one's
// history.

#include <algorithm>

#include "gdn_device.hpp"
#include "gdn_internal.hpp"

namespace gdn {

namespace {

constexpr int kThreads = 256;

struct Args {
  int64_t tokens;     // of all sequences
  int64_t T;          // of a dense sequence
  int ch;             // channels
  int lanes;          // threads of a row: channels / V
  int cblocks;        // workgroups of a row
  int R;              // tokens of a run
  int runs;
  int nseq;
  const int32_t* cu;
  const void *x, *s0, *dy, *ds;
  const float *taps, *bias;
  void *y, *sf, *dx, *ds0;
  float *part;        // [runs][W + 1][channels] shares of dtaps, dbias
  float *dtaps, *dbias;
};

template <typename IO, int V>
__device__ inline void load_v(const void* p, int64_t i, float* x) {
  if constexpr (V * io<IO>::bytes < 4) {
    x[0] = io<IO>::load(p, i);
  } else if constexpr (io<IO>::bytes == 2) {
    typedef __bf16 vec __attribute__((ext_vector_type(V)));
    const vec v = *reinterpret_cast<const vec*>(static_cast<const __bf16*>(p) + i);
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = static_cast<float>(v[e]);
  } else {
    typedef float vec __attribute__((ext_vector_type(V)));
    const vec v = *reinterpret_cast<const vec*>(static_cast<const float*>(p) + i);
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = v[e];
  }
}

template <typename IO, int V>
__device__ inline void store_v(void* p, int64_t i, const float* x) {
  if constexpr (V * io<IO>::bytes < 4) {
    io<IO>::store(p, i, x[0]);
  } else if constexpr (io<IO>::bytes == 2) {
    typedef __bf16 vec __attribute__((ext_vector_type(V)));
    vec v;
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = static_cast<__bf16>(x[e]);
    *reinterpret_cast<vec*>(static_cast<__bf16*>(p) + i) = v;
  } else {
    typedef float vec __attribute__((ext_vector_type(V)));
    vec v;
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = x[e];
    *reinterpret_cast<vec*>(static_cast<float*>(p) + i) = v;
  }
}

// The hardware's exponential and reciprocal for bf16 rows, the library's
// exponential and a division for fp32 ones.  What the former are off by, a few
// 2^-24 (1 + |p|) of the value, is far below the rounding of rows in bf16; in
// the fp32 sums dtaps and dbias it is the size of a term's own rounding (a
// division in full takes ten instructions more, and the forward of 16384
// tokens of 4096 channels 57 us instead of 53).
template <typename IO>
__device__ inline float sigmoid(float x) {
  if constexpr (io<IO>::bytes == 2) return __builtin_amdgcn_rcpf(1.0f + __expf(-x));
  else return 1.0f / (1.0f + expf(-x));
}

template <typename IO, int ACT>
__device__ inline float act(float x) {
  if constexpr (ACT == GDN_ACT_NONE) return x;
  const float s = sigmoid<IO>(x);
  return ACT == GDN_ACT_SILU ? x * s : s;
}
template <typename IO, int ACT>
__device__ inline float act_grad(float x) {
  if constexpr (ACT == GDN_ACT_NONE) return 1.0f;
  const float s = sigmoid<IO>(x);
  return ACT == GDN_ACT_SILU ? s * (1.0f + x * (1.0f - s)) : s * (1.0f - s);
}

// ---------------------------------------------------------------- sequences ---

struct Seq {
  int n;
  int64_t lo, hi;  // its tokens
};

__device__ inline int64_t bound(const Args& A, int n) {
  typedef __attribute__((address_space(4))) const int32_t* ptr;
  const int64_t b = reinterpret_cast<ptr>(reinterpret_cast<uintptr_t>(A.cu))[n];
  return b < 0 ? 0 : b > A.tokens ? A.tokens : b;
}

__device__ inline Seq seq_of(const Args& A, int n) {
  Seq s;
  s.n = n;
  s.lo = A.cu ? bound(A, n) : n * A.T;
  s.hi = A.cu ? bound(A, n + 1) : s.lo + A.T;
  if (s.hi < s.lo) s.hi = s.lo;
  return s;
}

// The sequence of token t, or the first one behind it; n = nseq: none.
__device__ inline Seq seq_at(const Args& A, int64_t t) {
  if (!A.cu) return seq_of(A, static_cast<int>(t / A.T));
  int lo = 0, hi = A.nseq;  // smallest n with cu[n + 1] > t
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (bound(A, m + 1) > t) hi = m;
    else lo = m + 1;
  }
  if (lo == A.nseq) return Seq{lo, A.tokens, A.tokens};
  return seq_of(A, lo);
}

// Input j places in front of token t of a sequence (j < W): a token, its
// history, or zero.
template <typename IO, int W, int V>
__device__ inline void input_at(const Args& A, const Seq& s, int64_t t, int64_t c, float* x) {
  if (t >= s.lo) return load_v<IO, V>(A.x, t * A.ch + c, x);
  const int64_t back = W - 1 + (t - s.lo);  // row of the history
  if (A.s0 != nullptr && back >= 0)
    return load_v<IO, V>(A.s0, (static_cast<int64_t>(s.n) * (W - 1) + back) * A.ch + c, x);
#pragma unroll
  for (int e = 0; e < V; ++e) x[e] = 0.f;
}

template <int W, int V>
struct Weights {
  float tap[W][V], bias[V];
  __device__ inline void load(const Args& A, int64_t c) {
    constexpr int P = V % 4 == 0 ? 4 : 1;  // values of a load
    float all[V * W];
#pragma unroll
    for (int i = 0; i < V * W; i += P) load_v<f32_t, P>(A.taps, c * W + i, all + i);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      bias[e] = 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j) tap[j][e] = all[e * W + j];
    }
    if (A.bias != nullptr) {
#pragma unroll
      for (int i = 0; i < V; i += P) load_v<f32_t, P>(A.bias, c + i, bias + i);
    }
  }
  // p_t from the input of the token and the W - 1 in front of it, x[j] the
  // one j places back
  __device__ inline void sum(const float (*x)[V], float* p) const {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float v = bias[e];
#pragma unroll
      for (int j = 0; j < W; ++j) v = fmaf(tap[j][e], x[j][e], v);
      p[e] = v;
    }
  }
};

// ---------------------------------------------------------------- forward ---

// Runs first, then one workgroup row for each sequence's kept inputs.
template <typename IO, int W, int V, int ACT>
__global__ __launch_bounds__(kThreads) void conv_fwd_kernel(Args A) {
  const int row = blockIdx.x / A.cblocks;
  const int lane = (blockIdx.x - row * A.cblocks) * kThreads + threadIdx.x;
  if (lane >= A.lanes) return;
  const int64_t c = static_cast<int64_t>(lane) * V;
  if (row >= A.runs) {
    const Seq s = seq_of(A, row - A.runs);
    for (int i = 0; i < W - 1; ++i) {
      float x[V];
      input_at<IO, W, V>(A, s, s.hi - (W - 1) + i, c, x);
      store_v<IO, V>(A.sf, (static_cast<int64_t>(s.n) * (W - 1) + i) * A.ch + c, x);
    }
    return;
  }
  Weights<W, V> w;
  w.load(A, c);
  const int64_t from = static_cast<int64_t>(row) * A.R;
  const int64_t end = from + A.R < A.tokens ? from + A.R : A.tokens;
  for (Seq s = seq_at(A, from); s.n < A.nseq && s.lo < end; s = seq_of(A, s.n + 1)) {
    int64_t t = s.lo > from ? s.lo : from;
    const int64_t stop = s.hi < end ? s.hi : end;
    if (t >= stop) {
      if (s.n + 1 >= A.nseq) break;
      continue;
    }
    float x[W][V];
#pragma unroll
    for (int j = 1; j < W; ++j) input_at<IO, W, V>(A, s, t - j, c, x[j - 1]);
    constexpr int U = 4;
    for (; t < stop; t += U) {
      float in[U][V];
#pragma unroll
      for (int u = 0; u < U; ++u)
        load_v<IO, V>(A.x, (t + u < stop ? t + u : stop - 1) * A.ch + c, in[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int j = W - 1; j > 0; --j)
#pragma unroll
          for (int e = 0; e < V; ++e) x[j][e] = x[j - 1][e];
        float p[V];
#pragma unroll
        for (int e = 0; e < V; ++e) x[0][e] = in[u][e];
        w.sum(x, p);
#pragma unroll
        for (int e = 0; e < V; ++e) p[e] = act<IO, ACT>(p[e]);
        if (t + u < stop) store_v<IO, V>(A.y, (t + u) * A.ch + c, p);
      }
    }
    if (s.n + 1 >= A.nseq) break;
  }
}

// One token of every sequence; its history moves up by one row in place.
template <typename IO, int W, int V, int ACT>
__global__ __launch_bounds__(kThreads) void conv_step_kernel(Args A) {
  const int n = blockIdx.x / A.cblocks;
  const int lane = (blockIdx.x - n * A.cblocks) * kThreads + threadIdx.x;
  if (lane >= A.lanes) return;
  const int64_t c = static_cast<int64_t>(lane) * V;
  const int64_t s = static_cast<int64_t>(n) * (W - 1) * A.ch + c;
  float x[W][V], p[V];
  load_v<IO, V>(A.x, static_cast<int64_t>(n) * A.ch + c, x[0]);
#pragma unroll
  for (int j = 1; j < W; ++j) load_v<IO, V>(A.sf, s + static_cast<int64_t>(W - 1 - j) * A.ch, x[j]);
  Weights<W, V> w;
  w.load(A, c);
  w.sum(x, p);
#pragma unroll
  for (int e = 0; e < V; ++e) p[e] = act<IO, ACT>(p[e]);
  store_v<IO, V>(A.y, static_cast<int64_t>(n) * A.ch + c, p);
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
    store_v<IO, V>(A.sf, s + static_cast<int64_t>(W - 2 - j) * A.ch, x[j]);
}

// --------------------------------------------------------------- backward ---

// Runs first (dx and the shares of dtaps, dbias), then one workgroup row for
// each sequence's ds0.  A run also forms the e of the W - 1 tokens behind it.
template <typename IO, int W, int V, int ACT>
__global__ __launch_bounds__(kThreads) void conv_bwd_kernel(Args A) {
  const int row = blockIdx.x / A.cblocks;
  const int lane = (blockIdx.x - row * A.cblocks) * kThreads + threadIdx.x;
  if (lane >= A.lanes) return;
  const int64_t c = static_cast<int64_t>(lane) * V;
  Weights<W, V> w;
  w.load(A, c);
  if (row >= A.runs) {
    // history row i is read by the tokens i - (W - 1) + j, j >= 1
    const Seq s = seq_of(A, row - A.runs);
    float g[W][V];
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) g[i][e] = 0.f;
#pragma unroll
    for (int t = 0; t < W - 1; ++t) {
      if (s.lo + t >= s.hi) break;
      float x[W][V], p[V], dy[V];
#pragma unroll
      for (int j = 0; j < W; ++j) input_at<IO, W, V>(A, s, s.lo + t - j, c, x[j]);
      w.sum(x, p);
      load_v<IO, V>(A.dy, (s.lo + t) * A.ch + c, dy);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float v = dy[e] * act_grad<IO, ACT>(p[e]);
#pragma unroll
        for (int j = t + 1; j < W; ++j) g[W - 1 + t - j][e] = fmaf(w.tap[j][e], v, g[W - 1 + t - j][e]);
      }
    }
    const int64_t size = s.hi - s.lo;
    for (int i = 0; i < W - 1; ++i) {
      float v[V];
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = 0.f;
      if (A.ds != nullptr && i >= size)
        load_v<IO, V>(A.ds, (static_cast<int64_t>(s.n) * (W - 1) + i - size) * A.ch + c, v);
#pragma unroll
      for (int k = 0; k < W - 1; ++k)
        if (k == i)
#pragma unroll
          for (int e = 0; e < V; ++e) v[e] += g[k][e];
      store_v<IO, V>(A.ds0, (static_cast<int64_t>(s.n) * (W - 1) + i) * A.ch + c, v);
    }
    return;
  }
  constexpr int U = 4;
  float dtap[W][V], db[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    db[e] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dtap[j][e] = 0.f;
  }
  const int64_t from = static_cast<int64_t>(row) * A.R;
  const int64_t end = from + A.R < A.tokens ? from + A.R : A.tokens;
  for (Seq s = seq_at(A, from); s.n < A.nseq && s.lo < end; s = seq_of(A, s.n + 1)) {
    const int64_t first = s.lo > from ? s.lo : from;
    const int64_t stop = s.hi < end ? s.hi : end;        // own tokens
    const int64_t past = stop + W - 1 < s.hi ? stop + W - 1 : s.hi;  // with those behind
    if (first < stop) {
      float x[W][V], g[W][V];  // g[j]: what is known of dx of the token j places back
#pragma unroll
      for (int j = 1; j < W; ++j) input_at<IO, W, V>(A, s, first - j, c, x[j - 1]);
#pragma unroll
      for (int j = 0; j < W; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) g[j][e] = 0.f;
      // one turn past the last token for each dx that is still open
      for (int64_t t0 = first; t0 < stop + W - 1; t0 += U) {
        float in[U][V], dy[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t at = (t0 + u < past ? t0 + u : past - 1) * A.ch + c;
          load_v<IO, V>(A.x, at, in[u]);
          load_v<IO, V>(A.dy, at, dy[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t t = t0 + u;
          if (t >= stop + W - 1) break;
          const bool live = t < past;
          float p[V];
#pragma unroll
          for (int j = W - 1; j > 0; --j)
#pragma unroll
            for (int e = 0; e < V; ++e) {
              x[j][e] = x[j - 1][e];
              g[j][e] = g[j - 1][e];
            }
#pragma unroll
          for (int e = 0; e < V; ++e) {
            x[0][e] = in[u][e];
            g[0][e] = 0.f;
          }
          w.sum(x, p);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float v = live ? dy[u][e] * act_grad<IO, ACT>(p[e]) : 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) g[j][e] = fmaf(w.tap[j][e], v, g[j][e]);
            const float own = t < stop ? v : 0.f;
            db[e] += own;
#pragma unroll
            for (int j = 0; j < W; ++j) dtap[j][e] = fmaf(own, x[j][e], dtap[j][e]);
          }
          const int64_t done = t - (W - 1);
          if (done >= first) {
            const int64_t keep = done - (s.hi - (W - 1));
            if (A.ds != nullptr && keep >= 0) {
              float k[V];
              load_v<IO, V>(A.ds, (static_cast<int64_t>(s.n) * (W - 1) + keep) * A.ch + c, k);
#pragma unroll
              for (int e = 0; e < V; ++e) g[W - 1][e] += k[e];
            }
            store_v<IO, V>(A.dx, done * A.ch + c, g[W - 1]);
          }
        }
      }
    }
    if (s.n + 1 >= A.nseq) break;
  }
#pragma unroll
  for (int j = 0; j < W; ++j)
    store_v<f32_t, V>(A.part, (static_cast<int64_t>(row) * (W + 1) + j) * A.ch + c, dtap[j]);
  store_v<f32_t, V>(A.part, (static_cast<int64_t>(row) * (W + 1) + W) * A.ch + c, db);
}

// dtaps, dbias: the runs' shares added in a fixed order.  Sixteen values a
// workgroup, 64 runs of rows added up in LDS.
constexpr int kRuns = 64;
__global__ __launch_bounds__(16 * kRuns) void conv_sum_kernel(Args A, int W) {
  const int lc = threadIdx.x & 15, run = threadIdx.x >> 4;
  const int64_t cols = static_cast<int64_t>(W + 1) * A.ch;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 16 + lc;
  float s[4] = {0.f, 0.f, 0.f, 0.f};  // four rows at a time in flight
  if (col < cols) {
    for (int k = run; k < A.runs; k += 4 * kRuns) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (k + u * kRuns < A.runs) s[u] += A.part[(k + u * kRuns) * cols + col];
    }
  }
  __shared__ float t[kRuns][17];
  t[run][lc] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
#pragma unroll
  for (int n = kRuns / 2; n >= 1; n >>= 1) {
    if (run < n) t[run][lc] += t[run + n][lc];
    __syncthreads();
  }
  if (run != 0 || col >= cols) return;
  const int j = static_cast<int>(col / A.ch), c = static_cast<int>(col - static_cast<int64_t>(j) * A.ch);
  if (j < W) A.dtaps[static_cast<int64_t>(c) * W + j] = t[0][lc];
  else if (A.dbias != nullptr) A.dbias[c] = t[0][lc];
}

// ------------------------------------------------------------------- plan ---

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Channels of a thread: a 16-byte piece of a row, 8 bytes where wide windows
// of it would not fit the registers, one channel where rows are not whole
// pieces.  The backward keeps twice the window: 16384 tokens of 1024 channels
// in bf16 take 33 us with four channels a thread, 45 with eight (of 4096
// channels 121 and 102; widths from 5 on have four either way).
int vec_of(const ShortConv& p, bool bwd) {
  int v = p.io == GDN_BF16 ? 8 : 4;
  if (p.width > 4 || bwd) v = 4;
  return p.ch % v == 0 ? v : 1;
}

Args make_args(const ShortConv& p, int V, int64_t most) {
  Args A{};
  A.tokens = static_cast<int64_t>(p.B) * p.T;
  A.T = p.T;
  A.ch = p.ch;
  A.lanes = p.ch / V;
  A.cblocks = static_cast<int>(ceil_div(A.lanes, kThreads));
  A.nseq = p.nseq;
  A.cu = p.varlen ? p.cu_seqlens : nullptr;
  // runs of 16 tokens, longer ones where there are more than `most` workgroups
  A.R = static_cast<int>(std::max<int64_t>(16, ceil_div(A.tokens * A.cblocks, most)));
  A.runs = static_cast<int>(ceil_div(A.tokens, A.R));
  return A;
}

// (backward of 16384 tokens, inputs in cache / not, us with 256, 512 and 1024
// workgroups: 1024 channels in bf16 42/52, 33/39, 35/38, of width 8 56/64,
// 48/53, 60/68, in fp32 53/63, 44/50, 49/56; 4096 channels in bf16 185/186,
// 121/122, 102/104: shorter runs form more of their neighbours' e and leave
// more shares)
constexpr int64_t kFwdBlocks = 4096, kBwdBlocks = 512;

template <typename F>
void with_act(int act, F f) {
  using std::integral_constant;
  if (act == GDN_ACT_NONE) f(integral_constant<int, GDN_ACT_NONE>{});
  else if (act == GDN_ACT_SILU) f(integral_constant<int, GDN_ACT_SILU>{});
  else f(integral_constant<int, GDN_ACT_SIGMOID>{});
}

// Calls f<W, V> of a width and a piece of V channels (wide windows: 4 or 1).
template <int WIDE, typename F>
void with_width(int W, int V, F f) {
  using std::integral_constant;
  auto v = [&](auto w) {
    if constexpr (w <= 4) {
      if (V == WIDE) f(w, integral_constant<int, WIDE>{});
      else f(w, integral_constant<int, 1>{});
    } else {
      if (V == 4) f(w, integral_constant<int, 4>{});
      else f(w, integral_constant<int, 1>{});
    }
  };
  switch (W) {
    case 1: return v(integral_constant<int, 1>{});
    case 2: return v(integral_constant<int, 2>{});
    case 3: return v(integral_constant<int, 3>{});
    case 4: return v(integral_constant<int, 4>{});
    case 5: return v(integral_constant<int, 5>{});
    case 6: return v(integral_constant<int, 6>{});
    case 7: return v(integral_constant<int, 7>{});
    default: return v(integral_constant<int, 8>{});
  }
}

template <typename IO>
void conv_fwd(const ShortConv& p, const Args& A, int V, bool step, hipStream_t s) {
  constexpr int WIDE = 16 / io<IO>::bytes;
  const int64_t rows = step ? p.nseq : A.runs + (A.sf != nullptr ? p.nseq : 0);
  const dim3 grid(static_cast<unsigned>(rows * A.cblocks));
  with_act(p.act, [&](auto a) {
    with_width<WIDE>(p.width, V, [&](auto w, auto v) {
      if (step)
        hipLaunchKernelGGL((conv_step_kernel<IO, w, v, a>), grid, dim3(kThreads), 0, s, A);
      else
        hipLaunchKernelGGL((conv_fwd_kernel<IO, w, v, a>), grid, dim3(kThreads), 0, s, A);
    });
  });
}

template <typename IO>
void conv_bwd(const ShortConv& p, const Args& A, int V, hipStream_t s) {
  const int64_t rows = A.runs + (A.ds0 != nullptr ? p.nseq : 0);
  const dim3 grid(static_cast<unsigned>(rows * A.cblocks));
  with_act(p.act, [&](auto a) {
    with_width<4>(p.width, V, [&](auto w, auto v) {
      hipLaunchKernelGGL((conv_bwd_kernel<IO, w, v, a>), grid, dim3(kThreads), 0, s, A);
    });
  });
}

}  // namespace

bool short_conv_fits(const ShortConv& p, bool bwd) {
  const Args A = make_args(p, vec_of(p, bwd), bwd ? kBwdBlocks : kFwdBlocks);
  const int64_t rows = static_cast<int64_t>(A.runs) + p.nseq;
  return rows <= ((int64_t(1) << 32) / kThreads - 1) / A.cblocks;
}

hipError_t launch_short_conv_fwd(const ShortConv& p, const void* x, const float* taps,
                                 const float* bias, const void* s0, void* y, void* s_final,
                                 hipStream_t s) {
  const int V = vec_of(p, false);
  Args A = make_args(p, V, kFwdBlocks);
  A.x = x;
  A.taps = taps;
  A.bias = bias;
  A.s0 = s0;
  A.y = y;
  A.sf = p.width > 1 ? s_final : nullptr;
  if (A.runs == 0 && A.sf == nullptr) return hipSuccess;
  StageScope scope(GDN_STAGE_PROLOGUE, s);
  if (p.io == GDN_BF16) conv_fwd<bf16_t>(p, A, V, false, s);
  else conv_fwd<f32_t>(p, A, V, false, s);
  return hipGetLastError();
}

hipError_t launch_short_conv_step(const ShortConv& p, const void* x, const float* taps,
                                  const float* bias, void* state, void* y, hipStream_t s) {
  const int V = vec_of(p, false);
  Args A = make_args(p, V, kFwdBlocks);
  A.x = x;
  A.taps = taps;
  A.bias = bias;
  A.sf = state;
  A.y = y;
  StageScope scope(GDN_STAGE_PROLOGUE, s);
  if (p.io == GDN_BF16) conv_fwd<bf16_t>(p, A, V, true, s);
  else conv_fwd<f32_t>(p, A, V, true, s);
  return hipGetLastError();
}

size_t short_conv_bwd_workspace_bytes(const ShortConv& p) {
  const Args A = make_args(p, vec_of(p, true), kBwdBlocks);
  return static_cast<size_t>(std::max(A.runs, 1)) * (p.width + 1) * p.ch * 4;
}

hipError_t launch_short_conv_bwd(const ShortConv& p, const void* x, const float* taps,
                                 const float* bias, const void* s0, const void* dy,
                                 const void* ds_final, void* dx, float* dtaps, float* dbias,
                                 void* ds0, void* ws, hipStream_t s) {
  const int V = vec_of(p, true);
  Args A = make_args(p, V, kBwdBlocks);
  A.x = x;
  A.taps = taps;
  A.bias = bias;
  A.s0 = s0;
  A.dy = dy;
  A.ds = ds_final;
  A.dx = dx;
  A.dtaps = dtaps;
  A.dbias = dbias;
  A.ds0 = p.width > 1 ? ds0 : nullptr;
  A.part = static_cast<float*>(ws);
  StageScope scope(GDN_STAGE_PROLOGUE, s);
  if (A.runs > 0 || A.ds0 != nullptr) {
    if (p.io == GDN_BF16) conv_bwd<bf16_t>(p, A, V, s);
    else conv_bwd<f32_t>(p, A, V, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 grid(static_cast<unsigned>(ceil_div(static_cast<int64_t>(p.ch) * (p.width + 1), 16)));
  hipLaunchKernelGGL(conv_sum_kernel, grid, dim3(16 * kRuns), 0, s, A, p.width);
  return hipGetLastError();
}

}  // namespace gdn
