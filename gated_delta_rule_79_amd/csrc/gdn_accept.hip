// Acceptance of drafted tokens against the target's probabilities, from given
// uniform numbers.  A sequence has a chain or a tree of up to 64 drafted
// nodes; the walk starts at its root and tries the children of where it
// stands in index order.  With r the target's row there (Z = 1), q the
// draft's:
//
//   child i of token x is accepted when  u_i q(x) Z < r(x);  the walk moves on
//   else  r <- max(r / Z - q, 0),  Z <- sum r  (unless that leaves nothing)
//
// and the next token is the first whose running sum of r exceeds u Z.  Children
// come behind their parents, so the walk tries nodes in ascending order and
// one loop over them ends it.  Everything is 64 bits: u q and the first
// difference are exact, and the sums' order moves a border by 2^-50 of it, so
// the answers are those of any other order but for numbers that close to one.
//
// The rows are what has to be read: one (or two, with a draft's) of V values
// for the next token, one more for every place with a rejection that the walk
// leaves.  What bounds a call is a chain of waits, not their bytes: the nodes,
// the values of their tokens, a row, its sum, and again for every row.  One
// workgroup walks a sequence, with its row in the CU where it fits (256 trees
// of 16 nodes over 32000 fp32 values: 36 to 42 us by the slowest of them, where
// 65 MB at the rate of a copy are 13; a chain of 8: 12 us).  Longer rows, and
// odd ones, are read anew for every sum (256 such trees over 32001 fp32 values:
// 145 us, over 50257: 195; over 128256 values in bf16: 324).  Of a chain of such
// only one node is ever tried at a place, so its end is known from gathered
// values alone: every workgroup finds it by itself and takes a slab of the row,
// a second launch finds the token in the slabs' sums (256 chains of 16 over
// 50257 fp32 values 51 us, one of them 15).

#include <algorithm>

#include "gdn_accept_row.hpp"
#include "gdn_device.hpp"
#include "gdn_internal.hpp"

namespace gdn {

namespace {

constexpr int kMaxNodes = 64;
constexpr int kWalkThreads = 1024;
constexpr int kHeldPer = 32;  // values a thread holds: rows up to 32768 stay in the CU
constexpr int kSlabThreads = 256;
constexpr int kLastPer = 4;  // values a thread takes where a token is looked for

struct Args {
  int n, V, trees;
  int64_t total;      // nodes of a packed batch
  const int32_t *cu, *parent, *tokens;
  const void *p, *q;  // target and draft rows, q null: certain drafts
  const float* u;
  int32_t *accepted, *length, *next;
  int slabs, slab;    // of a chain's row
  double* part;       // [trees][slabs] sums
  int2* head;         // [trees] a chain's accepted nodes, the token that failed
};

// Where a sequence's nodes and rows lie.
struct Tree {
  int64_t node, row;  // first node, first row (of the root)
  int size;
};

__device__ inline Tree tree_at(const Args& A, int m) {
  Tree t;
  if (A.cu == nullptr) {
    t.node = static_cast<int64_t>(m) * A.n;
    t.size = A.n;
  } else {
    const int64_t lo = min(max(static_cast<int64_t>(A.cu[m]), int64_t(0)), A.total);
    const int64_t hi = min(max(static_cast<int64_t>(A.cu[m + 1]), lo), A.total);
    t.node = lo;
    t.size = static_cast<int>(min(hi - lo, int64_t(kMaxNodes)));
  }
  t.row = t.node + m;
  return t;
}

template <typename IO>
using Row = AcceptRow<io<IO>>;

// A wave's sum of the row over [lo, hi); W: values of a load (lo a multiple).
template <typename IO, int W>
__device__ inline double wave_sum(const Row<IO>& r, int lo, int hi) {
  constexpr int U = 4;
  const int lane = threadIdx.x & 63;
  double s[U] = {0.0, 0.0, 0.0, 0.0};
  const bool two = r.two();
  for (int i = lo + lane * W; i < hi; i += 64 * W * U) {
    float p[U][W], q[U][W];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = i + u * 64 * W < hi ? i + u * 64 * W : i;  // (again, and not counted)
      if constexpr (W == 1) {
        p[u][0] = io<IO>::load(r.p, k);
        q[u][0] = two ? io<IO>::load(r.q, k) : 0.f;
      } else {
        typedef typename io<IO>::storage vec __attribute__((ext_vector_type(W)));
        const vec a = *reinterpret_cast<const vec*>(
            static_cast<const typename io<IO>::storage*>(r.p) + k);
        vec b{};
        if (two)
          b = *reinterpret_cast<const vec*>(static_cast<const typename io<IO>::storage*>(r.q) + k);
#pragma unroll
        for (int e = 0; e < W; ++e) {
          if constexpr (io<IO>::bytes == 2) {
            p[u][e] = bf16_bits_to_float(a[e]);
            q[u][e] = bf16_bits_to_float(b[e]);
          } else {
            p[u][e] = a[e];
            q[u][e] = b[e];
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u * 64 * W < hi)
#pragma unroll
        for (int e = 0; e < W; ++e) s[u] += r.less(p[u][e], q[u][e], i + u * 64 * W + e);
  }
  double v = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}

// Scratch of a workgroup of up to 16 waves.
struct Meet {
  double part[16];
  int first, last, token;
  double before;
};

// Sums of the waves' shares of [lo, hi) into meet.part; returns their total.
template <typename IO, int W>
__device__ inline double block_sums(const Row<IO>& r, int lo, int hi, Meet* meet) {
  const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6;
  const int each = ((hi - lo + waves - 1) / waves + W - 1) / W * W;
  const int from = min(lo + wave * each, hi), to = min(from + each, hi);
  const double v = wave_sum<IO, W>(r, from, to);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) meet->part[wave] = v;
  __syncthreads();
  double s = 0.0;
  for (int k = 0; k < waves; ++k) s += meet->part[k];
  return s;
}

// Of the workgroup's values v >= 0 (one a thread, in order): the first thread
// at which the running sum exceeds *target, or the last with a value if none
// does (0 if none has one).  Takes the sum in front of it off *target.
__device__ inline int pick(double v, double* target, Meet* meet) {
  const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  double run = v;  // of the wave's lanes up to this one
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const double o = __shfl_up(run, m, 64);
    if (lane >= m) run += o;
  }
  __syncthreads();
  if (lane == 63) meet->part[wave] = run;
  if (threadIdx.x == 0) meet->first = 0x7fffffff, meet->last = 0;
  __syncthreads();
  double front = run - v;
  for (int k = 0; k < wave && k < waves; ++k) front += meet->part[k];
  const int id = threadIdx.x;
  if (v > 0.0) {
    if (front + v > *target) atomicMin(&meet->first, id);
    atomicMax(&meet->last, id);
  }
  __syncthreads();
  const int at = meet->first != 0x7fffffff ? meet->first : meet->last;
  if (id == at) meet->before = front;
  __syncthreads();
  *target -= meet->before;
  return at;
}

// The token among a thread's values w (kLastPer of them from `at` on, the
// threads' in order) at which the running sum exceeds target; the last one with
// a part of the row if none does.
template <int PER>
__device__ inline int find(const double (&w)[PER], int at, double target, int none, Meet* meet) {
  double sum = 0.0;
#pragma unroll
  for (int e = 0; e < PER; ++e) sum += w[e];
  const int owner = pick(sum, &target, meet);
  if (static_cast<int>(threadIdx.x) == owner) {
    int token = none;
    double run = 0.0;
    for (int e = PER - 1; e >= 0; --e)
      if (w[e] > 0.0 && token == none) token = at + e;  // the last
    bool found = false;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      run += w[e];
      if (!found && w[e] > 0.0 && run > target) token = at + e, found = true;
    }
    meet->token = token;
  }
  __syncthreads();
  return meet->token;
}

// The token of [lo, hi), narrowed to what the threads hold at once.
template <typename IO, int W>
__device__ inline int draw(const Row<IO>& r, int lo, int hi, double target, int none, Meet* meet) {
  const int waves = blockDim.x >> 6;
  while (hi - lo > static_cast<int>(blockDim.x) * kLastPer) {
    block_sums<IO, W>(r, lo, hi, meet);
    const int each = ((hi - lo + waves - 1) / waves + W - 1) / W * W;
    const double v = static_cast<int>(threadIdx.x) < waves ? meet->part[threadIdx.x] : 0.0;
    const int k = pick(v, &target, meet);
    lo = min(lo + k * each, hi);
    hi = min(lo + each, hi);
  }
  double w[kLastPer];
  const int at = lo + threadIdx.x * kLastPer;
  r.take(at, hi, w);
  return find(w, at, target, none, meet);
}

template <typename IO>
__device__ inline const void* row_at(const void* base, int64_t row, int V) {
  return base == nullptr ? nullptr : static_cast<const char*>(base) + row * V * io<IO>::bytes;
}

__device__ inline bool take(float u, float q, double Z, double r) {
  return static_cast<double>(u) * static_cast<double>(q) * Z < r;
}

// ---------------------------------------------- one workgroup a sequence ---

// A sequence's nodes in LDS: every node with the target's and the draft's value of
// its token in its parent's row, gathered at once.
struct Nodes {
  int parent[kMaxNodes], token[kMaxNodes], tried[kMaxNodes];
  float p[kMaxNodes], q[kMaxNodes], u[kMaxNodes + 1];
  double scale[kMaxNodes];

  template <typename IO>
  __device__ inline void load(const Args& A, const Tree& t) {
    const int i = threadIdx.x;
    if (i <= t.size) u[i] = A.u[t.row + i];
    if (i < t.size) {
      const int x = A.tokens[t.node + i], up = A.parent != nullptr ? A.parent[t.node + i] : i - 1;
      const int from = up >= 0 && up < i ? up : -1;
      const bool ok = x >= 0 && x < A.V;
      const int64_t row = t.row + from + 1;
      parent[i] = ok ? from : -2;  // (a token that is none is no one's child)
      token[i] = x;
      p[i] = ok ? io<IO>::load(row_at<IO>(A.p, row, A.V), x) : 0.f;
      q[i] = ok && A.q != nullptr ? io<IO>::load(row_at<IO>(A.q, row, A.V), x) : 1.f;
    }
  }
};

// Where the walk stands.
struct Place {
  int node, length;   // last accepted node, accepted nodes
  int i;              // node that is tried next
  int m;              // rejections here
  double Z;
  __device__ inline void move() {
    node = i++;
    ++length;
    m = 0;
    Z = 1.0;
  }
  // the next child from i on; false: there is none
  __device__ inline bool child(const Nodes& nodes, const Tree& t) {
    while (i < t.size && nodes.parent[i] != node) ++i;
    return i < t.size;
  }
  __device__ inline bool accepts(const Nodes& nodes, bool drawn) const {
    double r = nodes.p[i];
    for (int j = 0; j < m; ++j) {
      const double by = drawn ? static_cast<double>(nodes.q[i])
                              : nodes.token[i] == nodes.tried[j] ? 1.0 : 0.0;
      r = fmax(fma(r, nodes.scale[j], -by), 0.0);
    }
    return take(nodes.u[i], nodes.q[i], Z, r);
  }
  // child i is rejected; sum(k): of what k rejections leave
  template <typename F>
  __device__ inline void reject(Nodes& nodes, F sum) {
    __syncthreads();  // (all have read what is written now)
    if (threadIdx.x == 0) nodes.scale[m] = 1.0 / Z, nodes.tried[m] = nodes.token[i];
    __syncthreads();
    const double left = sum(m + 1);
    if (left > 0.0) Z = left, ++m;  // else nothing would be left: the row stays
    ++i;
  }
};

// Rows of any length, read anew for every sum.
template <typename IO, int W>
__global__ __launch_bounds__(kWalkThreads) void accept_walk_kernel(Args A) {
  __shared__ Meet meet;
  __shared__ Nodes nodes;
  const Tree t = tree_at(A, blockIdx.x);
  nodes.load<IO>(A, t);
  __syncthreads();
  Place at{-1, 0, 0, 0, 1.0};
  Row<IO> r{row_at<IO>(A.p, t.row, A.V), row_at<IO>(A.q, t.row, A.V), 0, nodes.scale, nodes.tried};
  while (at.child(nodes, t)) {
    if (at.accepts(nodes, A.q != nullptr)) {
      at.move();
      r.p = row_at<IO>(A.p, t.row + at.node + 1, A.V);
      r.q = row_at<IO>(A.q, t.row + at.node + 1, A.V);
    } else {
      at.reject(nodes, [&](int k) {
        r.m = k;
        return block_sums<IO, W>(r, 0, A.V, &meet);
      });
    }
  }
  r.m = at.m;
  double target = static_cast<double>(nodes.u[t.size]) * block_sums<IO, W>(r, 0, A.V, &meet);
  const int waves = kWalkThreads / 64, each = ((A.V + waves - 1) / waves + W - 1) / W * W;
  const double v = static_cast<int>(threadIdx.x) < waves ? meet.part[threadIdx.x] : 0.0;
  const int lo = min(pick(v, &target, &meet) * each, A.V);
  const int next = draw<IO, W>(r, lo, min(lo + each, A.V), target, A.V - 1, &meet);
  if (threadIdx.x == 0) {
    A.accepted[blockIdx.x] = at.node;
    A.length[blockIdx.x] = at.length;
    A.next[blockIdx.x] = next;
  }
}

// Rows that fit a CU, the target's in registers and the draft's in LDS: a row
// is read once at most, and one whose first child is accepted not at all.  With
// drawn drafts k rejections leave max(p a - q b, 0), a the product of their 1/Z
// and b the sum of the products behind each (what is negative once stays so),
// as much work for the last one as for the first.  A wave has adjacent tokens,
// so that its sum alone says whether the next token is among them; it then
// looks for it by itself.
template <typename IO, int W>
__global__ __launch_bounds__(kWalkThreads) void accept_held_kernel(Args A) {
  constexpr int C = kHeldPer / W, WAVES = kWalkThreads / 64, SPAN = 64 * W;
  typedef typename io<IO>::storage store;
  struct Piece {  // W values as they are stored
    uint32_t bits[W * sizeof(store) / 4];
    __device__ inline float operator[](int e) const {
      if constexpr (sizeof(store) == 4) return __uint_as_float(bits[e]);
      else return __uint_as_float(e & 1 ? bits[e >> 1] & 0xffff0000u : bits[e >> 1] << 16);
    }
    // Taken for changed here: the 64-bit values of a whole row are else formed
    // once for all sums and kept, more than there are registers.
    __device__ inline void fresh() {
      for (auto& b : bits) asm volatile("" : "+v"(b));
    }
  };
  __shared__ Nodes nodes;
  __shared__ double part[2][WAVES];  // the waves' sums, of every second row in turn
  __shared__ Piece q[C][kWalkThreads];  // (a thread reads its own)
  const Tree t = tree_at(A, blockIdx.x);
  const bool drawn = A.q != nullptr;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  nodes.load<IO>(A, t);
  __syncthreads();
  Place at{-1, 0, 0, 0, 1.0};
  const int count = (A.V + WAVES * SPAN - 1) / (WAVES * SPAN);  // pieces of a wave that are used
  const int first = (wave * count * 64 + lane) * W;             // token
  Piece p[C];
  double scale = 1.0, less = 0.0;  // a, b of the rejections here
  int turn = 0;
  // (through a descriptor: what lies past the row is zero)
  auto load = [&](const void* base, auto&& set) {
    const auto row = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<void*>(row_at<IO>(base, t.row + at.node + 1, A.V)), 0, A.V * io<IO>::bytes,
        0x00027000);
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c < count)
        set(c, __builtin_bit_cast(Piece, __builtin_amdgcn_raw_buffer_load_b128(
                                             row, (first + c * SPAN) * io<IO>::bytes, 0, 0)));
  };
  // piece c of the row behind k rejections
  auto piece = [&](int c, int k, double (&w)[W]) {
    p[c].fresh();
#pragma unroll
    for (int e = 0; e < W; ++e) w[e] = p[c][e] > 0.f ? p[c][e] : 0.f;  // (a NaN counts nothing)
    if (k == 0) return;
    if (drawn) {
      const Piece by = q[c][threadIdx.x];
#pragma unroll
      for (int e = 0; e < W; ++e)
        w[e] = fmax(fma(w[e], scale, -(static_cast<double>(by[e]) * less)), 0.0);
    } else {
      for (int j = 0; j < k; ++j) {
        const double s = nodes.scale[j];
        const int x = nodes.tried[j] - (first + c * SPAN);
#pragma unroll
        for (int e = 0; e < W; ++e) w[e] = fmax(fma(w[e], s, e == x ? -1.0 : 0.0), 0.0);
      }
    }
  };
  // the row's sum behind k rejections, the waves' in part[turn]
  auto total = [&](int k) {
    if (k > 0) {
      scale = 1.0, less = 0.0;
      for (int j = 0; j < k; ++j) {
        scale *= nodes.scale[j];
        less = fma(less, nodes.scale[j], 1.0);
      }
    }
    double s = 0.0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (c >= count) break;
      double w[W];
      piece(c, k, w);
#pragma unroll
      for (int e = 0; e < W; ++e) s += w[e];
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
    turn ^= 1;
    if (lane == 0) part[turn][wave] = s;
    __syncthreads();
    double all = 0.0;
#pragma unroll
    for (int o = 0; o < WAVES; ++o) all += part[turn][o];
    return all;
  };
  double sum;
  bool moved;
  do {
    bool child = at.child(nodes, t);
    while (child && at.accepts(nodes, drawn)) {
      at.move();
      child = at.child(nodes, t);
    }
    load(A.p, [&](int c, Piece v) { p[c] = v; });
    if (child && drawn) load(A.q, [&](int c, Piece v) { q[c][threadIdx.x] = v; });
    sum = 0.0;
    moved = false;
    while (child && !moved) {
      __syncthreads();  // (all have read what is written now)
      if (threadIdx.x == 0) nodes.scale[at.m] = 1.0 / at.Z, nodes.tried[at.m] = nodes.token[at.i];
      __syncthreads();
      sum = total(at.m + 1);
      if (sum > 0.0) at.Z = sum, ++at.m;  // else nothing would be left: the row stays
      ++at.i;
      child = at.child(nodes, t);
      if (child && at.accepts(nodes, drawn)) {
        at.move();
        moved = true;
      }
    }
  } while (moved);
  if (!(sum > 0.0)) sum = total(at.m);  // none tried here, or the last one left nothing
  // the wave that has the token: the first at which the running sum exceeds the
  // target, or the last with a part of the row
  const double target = static_cast<double>(nodes.u[t.size]) * sum;
  int owner = 0;
  double front = 0.0, run = 0.0;
  bool found = false;
#pragma unroll
  for (int o = 0; o < WAVES; ++o) {
    const double v = part[turn][o];
    if (v > 0.0 && !found) {
      owner = o;
      front = run;
      found = run + v > target;
    }
    run += v;
  }
  if (wave != owner) return;
  double own[C], upto[C];  // a lane's part of a piece, and with the lanes in front
#pragma unroll
  for (int c = 0; c < C; ++c) {
    own[c] = 0.0;
    if (c < count) {
      double w[W];
      piece(c, at.m, w);
#pragma unroll
      for (int e = 0; e < W; ++e) own[c] += w[e];
    }
    upto[c] = own[c];
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const double o = __shfl_up(upto[c], m, 64);
      if (lane >= m) upto[c] += o;
    }
  }
  int holder = 0, which = -1;
  double before = 0.0;
  found = false;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const unsigned long long some = __ballot(own[c] > 0.0);
    const unsigned long long over = __ballot(own[c] > 0.0 && front + upto[c] > target);
    if (some != 0 && !found) {
      found = over != 0;
      holder = found ? __ffsll(over) - 1 : 63 - __clzll(some);
      which = c;
      before = front + (upto[c] - own[c]);
    }
    front += __shfl(upto[c], 63, 64);
  }
  int token = A.V - 1;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (c != which) continue;  // (uniform)
    double w[W];
    piece(c, at.m, w);
    bool here = false;
#pragma unroll
    for (int e = 0; e < W; ++e) {
      before += w[e];
      if (w[e] > 0.0 && !here) {
        token = first + c * SPAN + e;
        here = before > target;
      }
    }
  }
  if (lane == holder) {
    A.accepted[blockIdx.x] = at.node;
    A.length[blockIdx.x] = at.length;
    A.next[blockIdx.x] = token;
  }
}

// -------------------------------------------------- chains of longer rows ---

// Length of a chain's accepted part: every lane tries a node against the
// target's row in front of it, the first that fails ends it.  Also whether
// one failed, and so what its place is drawn from.
template <typename IO>
__device__ inline int chain_end(const Args& A, const Tree& t, int* x) {
  const int i = threadIdx.x & 63;
  int token = -1;
  bool ok = false;
  if (i < t.size) {
    token = A.tokens[t.node + i];
    if (token >= 0 && token < A.V) {
      const double p = io<IO>::load(row_at<IO>(A.p, t.row + i, A.V), token);
      const float q =
          A.q != nullptr ? io<IO>::load(row_at<IO>(A.q, t.row + i, A.V), token) : 1.f;
      ok = take(A.u[t.row + i], q, 1.0, p);
    }
  }
  const unsigned long long fails = __ballot(!ok);
  const int end = fails == 0 ? 64 : __ffsll(fails) - 1;  // (lanes past the chain fail)
  *x = __shfl(token, end & 63, 64);
  return min(end, t.size);
}

template <typename IO>
__device__ inline Row<IO> chain_row(const Args& A, const Tree& t, int end, int x, double* scale,
                                    int* tried) {
  // a token that is none was not tried: the row stays
  const bool rejected = end < t.size && x >= 0 && x < A.V;
  if (threadIdx.x == 0) scale[0] = 1.0, tried[0] = x;
  __syncthreads();
  return Row<IO>{row_at<IO>(A.p, t.row + end, A.V), row_at<IO>(A.q, t.row + end, A.V),
                 rejected ? 1 : 0, scale, tried};
}

template <typename IO, int W>
__global__ __launch_bounds__(kSlabThreads) void accept_slab_kernel(Args A) {
  __shared__ Meet meet;
  __shared__ double scale[1];
  __shared__ int tried[1];
  const int m = blockIdx.x / A.slabs, k = blockIdx.x - m * A.slabs;
  const Tree t = tree_at(A, m);
  int x;
  const int end = chain_end<IO>(A, t, &x);
  const Row<IO> r = chain_row<IO>(A, t, end, x, scale, tried);
  const int lo = min(k * A.slab, A.V), hi = min(lo + A.slab, A.V);
  const double sum = block_sums<IO, W>(r, lo, hi, &meet);
  if (threadIdx.x == 0) {
    A.part[static_cast<int64_t>(m) * A.slabs + k] = sum;
    if (k == 0) A.head[m] = int2{end, x};
  }
}

template <typename IO, int W>
__global__ __launch_bounds__(kSlabThreads) void accept_chain_kernel(Args A) {
  __shared__ Meet meet;
  __shared__ double scale[1];
  __shared__ int tried[1];
  const int m = blockIdx.x;
  const Tree t = tree_at(A, m);
  const int2 head = A.head[m];
  const int end = head.x;
  const double part = static_cast<int>(threadIdx.x) < A.slabs
                          ? A.part[static_cast<int64_t>(m) * A.slabs + threadIdx.x] : 0.0;
  const double u = A.u[t.row + t.size];
  Row<IO> r = chain_row<IO>(A, t, end, head.y, scale, tried);
  double sum = part;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 64);
  if ((threadIdx.x & 63) == 0) meet.part[threadIdx.x >> 6] = sum;
  __syncthreads();
  sum = (meet.part[0] + meet.part[1]) + (meet.part[2] + meet.part[3]);
  int lo = 0, hi = A.V;
  double target;
  if (r.m > 0 && !(sum > 0.0)) {  // (uniform) nothing is left: the target's own row
    r.m = 0;
    target = u * block_sums<IO, W>(r, 0, A.V, &meet);
  } else {
    target = u * sum;
    lo = min(pick(part, &target, &meet) * A.slab, A.V);
    hi = min(lo + A.slab, A.V);
  }
  const int next = draw<IO, W>(r, lo, hi, target, A.V - 1, &meet);
  if (threadIdx.x == 0) {
    A.accepted[m] = end - 1;
    A.length[m] = end;
    A.next[m] = next;
  }
}

// Rows that stay in a CU (where they are whole 16-byte pieces too).
bool held(int64_t V) { return V <= kWalkThreads * kHeldPer; }

int values_of_piece(const Accept& p) {
  const int W = p.io == GDN_BF16 ? 8 : 4;
  return p.V % W == 0 ? W : 1;
}

// Slabs of a chain's row: 1024 values, which the second launch's workgroup
// holds at once, more where there are more than 2048 workgroups or 256 slabs.
void plan_slabs(const Accept& p, int* slabs, int* slab) {
  const int64_t V = p.V;
  int64_t each = std::max<int64_t>(1024, (V * p.trees + 2047) / 2048);
  each = (std::max(each, (V + kSlabThreads - 1) / kSlabThreads) + 7) / 8 * 8;
  each = std::min(each, (V + 7) / 8 * 8);
  *slab = static_cast<int>(each);
  *slabs = static_cast<int>((V + each - 1) / each);
}

template <typename IO, int W>
hipError_t accept(const Args& A, hipStream_t s) {
  // (Chains of rows that fit: 1 of 32000 fp32 values 15.5 us in slabs, 13.0
  // held; 256 of them 38 and 20; 2048 of 4096 values 52 and 57.)
  const dim3 grid(A.trees), threads(kWalkThreads);
  if constexpr (W > 1) {
    if (held(A.V)) {
      hipLaunchKernelGGL((accept_held_kernel<IO, W>), grid, threads, 0, s, A);
      return hipGetLastError();
    }
  }
  if (A.parent != nullptr) {
    hipLaunchKernelGGL((accept_walk_kernel<IO, W>), grid, threads, 0, s, A);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((accept_slab_kernel<IO, W>), dim3(A.trees * A.slabs), dim3(kSlabThreads), 0,
                     s, A);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((accept_chain_kernel<IO, W>), dim3(A.trees), dim3(kSlabThreads), 0, s, A);
  return hipGetLastError();
}

}  // namespace

size_t accept_workspace_bytes(const Accept& p) {
  if (p.tree || (values_of_piece(p) > 1 && held(p.V))) return 0;
  int slabs, slab;
  plan_slabs(p, &slabs, &slab);
  return static_cast<size_t>(p.trees) * (slabs * sizeof(double) + sizeof(int2));
}

hipError_t launch_accept(const Accept& p, const int32_t* parent, const int32_t* tokens,
                         const void* target, const void* draft, const float* u,
                         int32_t* accepted, int32_t* length, int32_t* next, void* ws,
                         hipStream_t s) {
  Args A{};
  A.n = p.n;
  A.V = p.V;
  A.trees = p.trees;
  A.total = p.n;
  A.cu = p.cu_seqlens;
  A.parent = parent;
  A.tokens = tokens;
  A.p = target;
  A.q = draft;
  A.u = u;
  A.accepted = accepted;
  A.length = length;
  A.next = next;
  plan_slabs(p, &A.slabs, &A.slab);
  A.part = static_cast<double*>(ws);
  if (ws != nullptr)
    A.head = reinterpret_cast<int2*>(A.part + static_cast<int64_t>(A.trees) * A.slabs);
  StageScope scope(GDN_STAGE_OTHER, s);
  // whole rows of 16-byte pieces, else one value at a time
  const bool whole = values_of_piece(p) > 1;
  if (p.io == GDN_BF16) return whole ? accept<bf16_t, 8>(A, s) : accept<bf16_t, 1>(A, s);
  return whole ? accept<f32_t, 4>(A, s) : accept<f32_t, 1>(A, s);
}

}  // namespace gdn
