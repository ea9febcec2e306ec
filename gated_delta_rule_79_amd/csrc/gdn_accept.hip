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
// for the next token, one more pass for every rejected sibling.  Of a chain
// only one node is ever tried at a place, so its end is known from gathered
// values alone: every workgroup finds it by itself and takes a slab of the
// row, a second launch finds the token in the slabs' sums.  A tree's passes
// depend on each other; one workgroup walks it.

#include <algorithm>

#include "gdn_device.hpp"
#include "gdn_internal.hpp"

namespace gdn {

namespace {

constexpr int kMaxNodes = 64;
constexpr int kWalkThreads = 1024;
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

// The row that is drawn from: the target's, less what was tried there.
template <typename IO>
struct Row {
  const void *p, *q;      // the target's and the draft's row
  int m;                  // rejected children
  const double* scale;    // 1 / Z in front of each rejection
  const int* tried;       // their tokens (certain drafts)

  __device__ inline double less(float pv, float qv, int x) const {
    double w = static_cast<double>(pv);
    for (int j = 0; j < m; ++j) {
      const double d = w * scale[j] - (q != nullptr ? static_cast<double>(qv)
                                                    : x == tried[j] ? 1.0 : 0.0);
      w = d;
      if (!(w > 0.0)) w = 0.0;
    }
    return w > 0.0 ? w : 0.0;  // (a NaN counts nothing)
  }
  __device__ inline double at(int x) const {
    return less(io<IO>::load(p, x), q != nullptr ? io<IO>::load(q, x) : 0.f, x);
  }
};

// A wave's sum of the row over [lo, hi); W: values of a load (lo a multiple).
template <typename IO, int W>
__device__ inline double wave_sum(const Row<IO>& r, int lo, int hi) {
  constexpr int U = 4;
  const int lane = threadIdx.x & 63;
  double s[U] = {0.0, 0.0, 0.0, 0.0};
  const bool two = r.q != nullptr && r.m > 0;
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
  int lo, hi, first, last;
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

// The share of `count` sums whose running sum first exceeds what is left of
// `target`, or the last that is not empty; takes the sums in front off it.
__device__ inline int pick(const double* part, int count, double* target) {
  double before = 0.0, at = 0.0;
  int last = 0;
  for (int k = 0; k < count; ++k) {
    if (part[k] > 0.0) last = k, at = before;
    if (before + part[k] > *target && part[k] > 0.0) break;
    before += part[k];
  }
  *target -= at;
  return last;
}

// The token of [lo, hi) (few enough for the workgroup) at which the running
// sum exceeds target; the last one with a part of the row if none does.
template <typename IO>
__device__ inline int find(const Row<IO>& r, int lo, int hi, double target, int none, Meet* meet) {
  const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  double w[kLastPer], sum = 0.0;
  const int at = lo + threadIdx.x * kLastPer;
#pragma unroll
  for (int e = 0; e < kLastPer; ++e) {
    w[e] = at + e < hi ? r.at(at + e) : 0.0;
    sum += w[e];
  }
  double run = sum;  // of the wave's lanes up to this one
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const double v = __shfl_up(run, m, 64);
    if (lane >= m) run += v;
  }
  __syncthreads();
  if (lane == 63) meet->part[wave] = run;
  if (threadIdx.x == 0) meet->first = 0x7fffffff, meet->last = -1;
  __syncthreads();
  double before = run - sum;
  for (int k = 0; k < wave && k < waves; ++k) before += meet->part[k];
#pragma unroll
  for (int e = 0; e < kLastPer; ++e) {
    before += w[e];
    if (w[e] > 0.0) {
      if (before > target) atomicMin(&meet->first, at + e);
      atomicMax(&meet->last, at + e);
    }
  }
  __syncthreads();
  return meet->first != 0x7fffffff ? meet->first : meet->last >= 0 ? meet->last : none;
}

// Narrows [lo, hi) to what find() takes, then finds the token.
template <typename IO, int W>
__device__ inline int draw(const Row<IO>& r, int lo, int hi, double target, int none, Meet* meet) {
  const int waves = blockDim.x >> 6;
  while (hi - lo > static_cast<int>(blockDim.x) * kLastPer) {
    block_sums<IO, W>(r, lo, hi, meet);
    const int each = ((hi - lo + waves - 1) / waves + W - 1) / W * W;
    const int k = pick(meet->part, waves, &target);
    __syncthreads();
    lo = min(lo + k * each, hi);
    hi = min(lo + each, hi);
  }
  return find(r, lo, hi, target, none, meet);
}

template <typename IO>
__device__ inline const void* row_at(const void* base, int64_t row, int V) {
  return base == nullptr ? nullptr : static_cast<const char*>(base) + row * V * io<IO>::bytes;
}

__device__ inline bool take(float u, float q, double Z, double r) {
  return static_cast<double>(u) * static_cast<double>(q) * Z < r;
}

// ------------------------------------------------------------------- trees ---

template <typename IO, int W>
__global__ __launch_bounds__(kWalkThreads) void accept_walk_kernel(Args A) {
  __shared__ Meet meet;
  __shared__ double scale[kMaxNodes];
  __shared__ int tried[kMaxNodes], parent[kMaxNodes], token[kMaxNodes];
  __shared__ float u[kMaxNodes + 1];
  const Tree t = tree_at(A, blockIdx.x);
  if (threadIdx.x < t.size) {
    parent[threadIdx.x] = A.parent[t.node + threadIdx.x];
    token[threadIdx.x] = A.tokens[t.node + threadIdx.x];
  }
  if (threadIdx.x <= t.size) u[threadIdx.x] = A.u[t.row + threadIdx.x];
  __syncthreads();
  int cur = -1, length = 0;
  double Z = 1.0;
  Row<IO> r{row_at<IO>(A.p, t.row, A.V), row_at<IO>(A.q, t.row, A.V), 0, scale, tried};
  for (int i = 0; i < t.size; ++i) {
    const int from = parent[i], x = token[i];
    const bool here = (from >= 0 && from < i ? from : -1) == cur && x >= 0 && x < A.V;
    if (!here) continue;  // (uniform)
    const float q = r.q != nullptr ? io<IO>::load(r.q, x) : 1.f;
    if (take(u[i], q, Z, r.at(x))) {
      cur = i;
      ++length;
      Z = 1.0;
      r.m = 0;
      r.p = row_at<IO>(A.p, t.row + i + 1, A.V);
      r.q = row_at<IO>(A.q, t.row + i + 1, A.V);
      continue;
    }
    __syncthreads();  // (all have read what is written now)
    if (threadIdx.x == 0) scale[r.m] = 1.0 / Z, tried[r.m] = x;
    __syncthreads();
    ++r.m;
    const double left = block_sums<IO, W>(r, 0, A.V, &meet);
    if (left > 0.0) Z = left;
    else --r.m;  // nothing would be left: the row stays
  }
  // (the sum of a row that was rejected from is known, its shares are not kept)
  const double sum = block_sums<IO, W>(r, 0, A.V, &meet);
  double target = static_cast<double>(u[t.size]) * sum;
  const int waves = kWalkThreads / 64, each = ((A.V + waves - 1) / waves + W - 1) / W * W;
  const int k = pick(meet.part, waves, &target);
  __syncthreads();
  const int lo = min(k * each, A.V);
  const int next = draw<IO, W>(r, lo, min(lo + each, A.V), target, A.V - 1, &meet);
  if (threadIdx.x == 0) {
    A.accepted[blockIdx.x] = cur;
    A.length[blockIdx.x] = length;
    A.next[blockIdx.x] = next;
  }
}

// ------------------------------------------------------------------ chains ---

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
  if (threadIdx.x == 0) A.part[static_cast<int64_t>(m) * A.slabs + k] = sum;
}

template <typename IO, int W>
__global__ __launch_bounds__(kSlabThreads) void accept_chain_kernel(Args A) {
  __shared__ Meet meet;
  __shared__ double scale[1], part[kSlabThreads];
  __shared__ int tried[1];
  const int m = blockIdx.x;
  const Tree t = tree_at(A, m);
  int x;
  const int end = chain_end<IO>(A, t, &x);
  Row<IO> r = chain_row<IO>(A, t, end, x, scale, tried);
  if (threadIdx.x < A.slabs)
    part[threadIdx.x] = A.part[static_cast<int64_t>(m) * A.slabs + threadIdx.x];
  __syncthreads();
  double sum = 0.0;
  for (int k = 0; k < A.slabs; ++k) sum += part[k];
  const double u = A.u[t.row + t.size];
  int lo = 0, hi = A.V;
  double target = 0.0;
  if (r.m > 0 && !(sum > 0.0)) {  // (uniform) nothing is left: the target's own row
    r.m = 0;
    sum = block_sums<IO, W>(r, 0, A.V, &meet);
    target = u * sum;
  } else {
    target = u * sum;
    const int k = pick(part, A.slabs, &target);
    lo = min(k * A.slab, A.V);
    hi = min(lo + A.slab, A.V);
  }
  __syncthreads();
  const int next = draw<IO, W>(r, lo, hi, target, A.V - 1, &meet);
  if (threadIdx.x == 0) {
    A.accepted[m] = end - 1;
    A.length[m] = end;
    A.next[m] = next;
  }
}

// Slabs of a chain's row: at least 2048 values, and no more of them than give
// every CU two workgroups.
void plan_slabs(const Accept& p, int* slabs, int* slab) {
  const int64_t most = std::min<int64_t>(std::max<int64_t>(1, 512 / p.trees), kSlabThreads);
  int64_t each = (p.V + most - 1) / most;
  each = (std::max<int64_t>(each, 2048) + 7) / 8 * 8;
  *slab = static_cast<int>(each);
  *slabs = static_cast<int>((p.V + each - 1) / each);
}

template <typename IO, int W>
hipError_t accept(const Args& A, hipStream_t s) {
  if (A.parent != nullptr) {
    hipLaunchKernelGGL((accept_walk_kernel<IO, W>), dim3(A.trees), dim3(kWalkThreads), 0, s, A);
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
  if (p.tree) return 0;
  int slabs, slab;
  plan_slabs(p, &slabs, &slab);
  return static_cast<size_t>(p.trees) * slabs * sizeof(double);
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
  StageScope scope(GDN_STAGE_OTHER, s);
  // whole rows of 16-byte pieces, else one value at a time
  if (p.io == GDN_BF16)
    return p.V % 8 == 0 ? accept<bf16_t, 8>(A, s) : accept<bf16_t, 1>(A, s);
  return p.V % 4 == 0 ? accept<f32_t, 4>(A, s) : accept<f32_t, 1>(A, s);
}

}  // namespace gdn
