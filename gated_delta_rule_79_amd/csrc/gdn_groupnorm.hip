// Group norm of a causal block's output with an activation or a gate, and
// its backward.  Channels are last: x [tokens, H, d], a group is one token's
// d channels of one head, and no statistic crosses tokens.
//
//   c = x - mean(x) (center; else c = x),  r = 1 / sqrt(mean(c^2) + eps),
//   n = c r w + b,   y = act(n)  or, with a gate z,  y = n act(z)
// Backward:
//   dn = dy act'(n)  or  dy act(z),   dz = dy n act'(z)
//   g = dn w,  dx = r (g - mean(g) [center] - c r mean(g c r))
//   dw = sum dn c r,  db = sum dn   over tokens (and groups when shared)
//
// A row (one group of one token) sits on adjacent lanes, 8 channels each as
// 16-byte pieces (fp32: two); the lanes of a row are a power of two, those
// past d / 8 idle.  The row stays in registers between its statistics and
// its output, so x (z, dy) is read once and y (dx, dz) written once: the
// pass is a stream and HBM bounds it (forward, 65536 gated rows of 128 in
// bf16: 50 MB in 11.5 us, 4.4 TB/s; backward, 262144 of 256: 671 MB in 135
// us, 5.0 TB/s; holding the next row's pieces in registers meanwhile took
// 13.5 us, two rows a turn 15).  All arithmetic is fp32, the variance
// taken around the mean.  A thread keeps its head over its rows (the grid's
// stride is a whole number of tokens), so its weights are loaded once and
// its share of dw, db stays in registers.

#include <algorithm>
#include <numeric>

#include "gdn_device.hpp"
#include "gdn_internal.hpp"

namespace gdn {

namespace {

constexpr int kThreads = 256;

template <typename IO>
__device__ inline void load8(const void* p, int64_t i, float* x) {
  if constexpr (io<IO>::bytes == 2) {
    const bf16x8 v = *reinterpret_cast<const bf16x8*>(static_cast<const char*>(p) + i * 2);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = static_cast<float>(v[e]);
  } else {
    const floatx4* q = reinterpret_cast<const floatx4*>(static_cast<const float*>(p) + i);
    const floatx4 a = q[0], b = q[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = a[e], x[4 + e] = b[e];
  }
}

template <typename IO>
__device__ inline void store8(void* p, int64_t i, const float* x) {
  if constexpr (io<IO>::bytes == 2) {
    bf16x8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = static_cast<__bf16>(x[e]);
    *reinterpret_cast<bf16x8*>(static_cast<char*>(p) + i * 2) = v;
  } else {
    floatx4* q = reinterpret_cast<floatx4*>(static_cast<float*>(p) + i);
    q[0] = floatx4{x[0], x[1], x[2], x[3]};
    q[1] = floatx4{x[4], x[5], x[6], x[7]};
  }
}

// Sum over the LPR adjacent lanes of a row.
template <int LPR>
__device__ inline float row_sum(float x) {
#pragma unroll
  for (int m = 1; m < LPR; m <<= 1) x += __shfl_xor(x, m, 64);
  return x;
}

// The hardware's exponential for bf16 rows (its error, a few 2^-24 times
// |x|, is far below their rounding), the library's for fp32 ones.
template <typename IO>
__device__ inline float sigmoid(float x) {
  return 1.0f / (1.0f + (io<IO>::bytes == 2 ? __expf(-x) : expf(-x)));
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

// Statistics of a row from its pieces: c = x - mean (or x) and r.
template <int LPR>
__device__ inline float normalize(float* x, bool live, int d, bool center, float eps) {
  const float inv = 1.0f / static_cast<float>(d);
  if (center) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s += x[e];
    const float mean = row_sum<LPR>(s) * inv;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = live ? x[e] - mean : 0.f;
  }
  float q = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) q += x[e] * x[e];
  return 1.0f / sqrtf(row_sum<LPR>(q) * inv + eps);
}

struct Args {
  int64_t rows;     // tokens * H
  int64_t stride;   // rows between a thread's rows, a multiple of H
  int H, d;
  int center;
  float eps;
  int wstride;      // d, or 0 when one set of weights serves all groups
  const void *x, *z, *dy;
  const float *w, *b;
  void *y, *dx, *dz;
  int q;            // rows of partial dw, db a block leaves
  float *pw, *pb;   // partial dw, db [blocks * q][d]
};

template <typename IO, int LPR, int ACT, bool GATE, bool BWD>
__global__ __launch_bounds__(kThreads) void group_norm_kernel(Args a) {
  const int piece = threadIdx.x % LPR;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads / LPR) + threadIdx.x / LPR;
  const bool live = piece * 8 < a.d;
  const int h = static_cast<int>(first % a.H);
  float w[8], b[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = 1.f, b[e] = 0.f;
  if (live && a.w != nullptr) load8<f32_t>(a.w, int64_t(h) * a.wstride + piece * 8, w);
  if (live && a.b != nullptr) load8<f32_t>(a.b, int64_t(h) * a.wstride + piece * 8, b);
  float sw[8], sb[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sw[e] = sb[e] = 0.f;

  // every lane of a wave takes the same number of turns: rows past the end
  // are computed on zeros and not stored
  const int64_t wave0 = first - (threadIdx.x & 63) / LPR;
  for (int64_t r0 = wave0; r0 < a.rows; r0 += a.stride) {
    const int64_t row = r0 + (threadIdx.x & 63) / LPR;
    const bool ok = live && row < a.rows;
    const int64_t at = row * a.d + piece * 8;
    float x[8], z[8], dy[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = z[e] = dy[e] = 0.f;
    if (ok) {
      load8<IO>(a.x, at, x);
      if constexpr (GATE) load8<IO>(a.z, at, z);
      if constexpr (BWD) load8<IO>(a.dy, at, dy);
    }
    const float r = normalize<LPR>(x, live, a.d, a.center, a.eps);
    float o[8];
    if constexpr (!BWD) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = x[e] * r * w[e] + b[e];
        o[e] = GATE ? n * act<IO, ACT>(z[e]) : act<IO, ACT>(n);
      }
      if (ok) store8<IO>(a.y, at, o);
    } else {
      float g[8], gz[8], s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xh = x[e] * r, n = xh * w[e] + b[e];
        const float dn = dy[e] * (GATE ? act<IO, ACT>(z[e]) : act_grad<IO, ACT>(n));
        gz[e] = GATE ? dy[e] * n * act_grad<IO, ACT>(z[e]) : 0.f;
        sw[e] += dn * xh;
        sb[e] += dn;
        g[e] = dn * w[e];
        s1 += g[e];
        s2 += g[e] * xh;
        x[e] = xh;
      }
      const float inv = 1.0f / static_cast<float>(a.d);
      const float m1 = a.center ? row_sum<LPR>(s1) * inv : 0.f;
      const float m2 = row_sum<LPR>(s2) * inv;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = r * (g[e] - m1 - x[e] * m2);
      if (ok) {
        store8<IO>(a.dx, at, o);
        if constexpr (GATE) store8<IO>(a.dz, at, gz);
      }
    }
  }
  if constexpr (BWD) {
    // the block's shares of dw, db: rows of the same weights added in order
    constexpr int PER = kThreads / LPR;
    __shared__ float t[kThreads * 8];
    auto leave = [&](float* part, const float* v) {
      if (part == nullptr) return;
      __syncthreads();
      store8<f32_t>(t, threadIdx.x * 8, v);
      __syncthreads();
      for (int o = threadIdx.x; o < a.q * a.d; o += kThreads) {
        const int r = o / a.d, c = o - r * a.d;
        float s = t[r * LPR * 8 + c];
        for (int k = r + a.q; k < PER; k += a.q) s += t[k * LPR * 8 + c];
        part[static_cast<int64_t>(blockIdx.x) * a.q * a.d + o] = s;
      }
    };
    leave(a.pw, sw);
    leave(a.pb, sb);
  }
}

// Sums of the partial dw, db rows of each group (row index mod `period`), in
// a fixed order: out[g, c] = sum_k part[g + k period, c].  Sixteen columns of
// one group a workgroup, 64 runs of rows added up in LDS (16k tokens, H16,
// d 256: 8 us for 17 MB).
constexpr int kRuns = 64;
__global__ __launch_bounds__(16 * kRuns) void group_norm_sum_kernel(const float* pw,
                                                                    const float* pb, int64_t rows,
                                                                    int period, int d, float* ow,
                                                                    float* ob) {
  const float* part = blockIdx.z == 0 ? pw : pb;
  float* out = blockIdx.z == 0 ? ow : ob;
  if (part == nullptr) return;
  const int lc = threadIdx.x & 15, run = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + lc, g = blockIdx.y;
  float s[4] = {0.f, 0.f, 0.f, 0.f};  // four rows at a time in flight
  const int64_t step = static_cast<int64_t>(kRuns) * period;
  for (int64_t k = g + static_cast<int64_t>(run) * period; k < rows; k += 4 * step) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (k + u * step < rows) s[u] += part[(k + u * step) * d + c];
  }
  __shared__ float t[kRuns][17];
  t[run][lc] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
#pragma unroll
  for (int n = kRuns / 2; n >= 1; n >>= 1) {
    if (run < n) t[run][lc] += t[run + n][lc];
    __syncthreads();
  }
  if (run == 0) out[static_cast<int64_t>(g) * d + c] = t[0][lc];
}

int lanes_per_row(int d) {
  int l = 2;
  while (l * 8 < d) l *= 2;
  return l;  // 2 .. 32
}

// Blocks of the pass: enough to fill the machine, and a whole number of
// tokens' rows per turn of the grid.
int64_t norm_blocks(const GroupNorm& p, int64_t most) {
  const int per = kThreads / lanes_per_row(p.d);  // rows per block
  const int64_t rows = p.tokens * p.H;
  const int64_t unit = p.H / std::gcd(p.H, per);  // blocks in a whole number of tokens
  const int64_t want = std::min<int64_t>((rows + per - 1) / per, most);
  return std::max<int64_t>(1, (want + unit - 1) / unit) * unit;
}

// Rows of partial dw, db a block leaves: one when all groups share their
// weights, one for each head where its rows are whole tokens, else all.
int partial_rows(const GroupNorm& p) {
  const int per = kThreads / lanes_per_row(p.d);
  return p.shared ? 1 : per % p.H == 0 ? p.H : per;
}

// (eight and four blocks a CU: the forward measured slower at 1024 and 4096)
constexpr int64_t kFwdBlocks = 2048, kBwdBlocks = 1024;

template <typename IO, int LPR, int ACT, bool BWD>
void launch_act(const Args& a, int64_t blocks, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(blocks));
  if (a.z != nullptr)
    hipLaunchKernelGGL((group_norm_kernel<IO, LPR, ACT, true, BWD>), grid, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((group_norm_kernel<IO, LPR, ACT, false, BWD>), grid, dim3(kThreads), 0, s,
                       a);
}

template <typename IO, int LPR, bool BWD>
void launch_lpr(const GroupNorm& p, const Args& a, int64_t blocks, hipStream_t s) {
  switch (p.act) {
    case GDN_ACT_NONE: return launch_act<IO, LPR, GDN_ACT_NONE, BWD>(a, blocks, s);
    case GDN_ACT_SILU: return launch_act<IO, LPR, GDN_ACT_SILU, BWD>(a, blocks, s);
    default: return launch_act<IO, LPR, GDN_ACT_SIGMOID, BWD>(a, blocks, s);
  }
}

template <typename IO, bool BWD>
void launch_io(const GroupNorm& p, const Args& a, int64_t blocks, hipStream_t s) {
  switch (lanes_per_row(p.d)) {
    case 2: return launch_lpr<IO, 2, BWD>(p, a, blocks, s);
    case 4: return launch_lpr<IO, 4, BWD>(p, a, blocks, s);
    case 8: return launch_lpr<IO, 8, BWD>(p, a, blocks, s);
    case 16: return launch_lpr<IO, 16, BWD>(p, a, blocks, s);
    default: return launch_lpr<IO, 32, BWD>(p, a, blocks, s);
  }
}

Args make_args(const GroupNorm& p, int64_t blocks, const void* x, const void* z, const float* w,
               const float* b) {
  Args a{};
  a.rows = p.tokens * p.H;
  a.stride = blocks * (kThreads / lanes_per_row(p.d));
  a.H = p.H;
  a.d = p.d;
  a.center = p.center ? 1 : 0;
  a.eps = p.eps;
  a.wstride = p.shared ? 0 : p.d;
  a.q = partial_rows(p);
  a.x = x;
  a.z = z;
  a.w = w;
  a.b = b;
  return a;
}

}  // namespace

hipError_t launch_group_norm_fwd(const GroupNorm& p, const void* x, const void* z, const float* w,
                                 const float* b, void* y, hipStream_t s) {
  if (p.tokens == 0) return hipSuccess;
  const int64_t blocks = norm_blocks(p, kFwdBlocks);
  Args a = make_args(p, blocks, x, z, w, b);
  a.y = y;
  StageScope scope(GDN_STAGE_OTHER, s);
  if (p.io == GDN_BF16)
    launch_io<bf16_t, false>(p, a, blocks, s);
  else
    launch_io<f32_t, false>(p, a, blocks, s);
  return hipGetLastError();
}

// Partial dw and db (for weights of each group: a shared set needs less).
size_t group_norm_bwd_workspace_bytes(const GroupNorm& p) {
  return 2 * static_cast<size_t>(norm_blocks(p, kBwdBlocks) * partial_rows(p)) * p.d * 4;
}

hipError_t launch_group_norm_bwd(const GroupNorm& p, const void* x, const void* z, const float* w,
                                 const float* b, const void* dy, void* dx, void* dz, float* dw,
                                 float* db, void* ws, hipStream_t s) {
  const int64_t blocks = norm_blocks(p, kBwdBlocks);
  Args a = make_args(p, blocks, x, z, w, b);
  a.dy = dy;
  a.dx = dx;
  a.dz = dz;
  if (dw != nullptr) a.pw = static_cast<float*>(ws);
  const int64_t rows = blocks * a.q;
  if (db != nullptr) a.pb = static_cast<float*>(ws) + rows * p.d;
  StageScope scope(GDN_STAGE_OTHER, s);
  if (p.io == GDN_BF16)
    launch_io<bf16_t, true>(p, a, blocks, s);
  else
    launch_io<f32_t, true>(p, a, blocks, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || (dw == nullptr && db == nullptr)) return e;
  const int period = p.shared ? 1 : p.H;
  hipLaunchKernelGGL(group_norm_sum_kernel, dim3(p.d / 16, period, 2), dim3(16 * kRuns), 0, s,
                     a.pw, a.pb, rows, period, p.d, dw, db);
  return hipGetLastError();
}

}  // namespace gdn
