// Linear attention with a constant decay per head: chunked forward,
// backward and the single-token step.
//
//   S_t = a S_{t-1} + k_t v_t^T   (S: [dk, dv] fp32, a = exp(log_decay[h])),
//   o_t = S_t^T q_t
//
// Backward, with dS_t the gradient reaching S_t:
//   dS_t = q_t do_t^T + a dS_{t+1},  dq_t = S_t do_t,  dk_t = dS_t v_t,
//   dv_t = dS_t^T k_t,  dS0 = a dS_1  (dS_T takes ds_final).
// Each of o, dq, dk, dv is the same walk on other operands:
//
//   M_t = a M_{t-1} + y_t z_t^T,   out_t = M_t^T x_t
//   o : (x, y, z) = (q, k, v),  M = S               in token order
//   dq: (do, v, k),             M = S^T             in token order
//   dk: (v, do, q),             M = dS^T            from the last token back
//   dv: (k, q, do),             M = dS              from the last token back
//
// so one kernel serves all four (REV: rows taken from the end; the entering
// state then reaches the first walked token undecayed, and the state handed
// on is multiplied by a once more).
//
// Chunk form over C tokens (i, j: rows in walk order, off = 1, REV: 0):
//   out_i = a^{i+off} M_in^T x_i + sum_{j<=i} a^{i-j} (x_i . y_j) z_j
//   M_out = a^len M_in + sum_j a^{len-off-j} y_j z_j^T
// Every power of a has a non-negative exponent, so no factor overflows for
// a <= 1 and a = 0 (log_decay = -inf) is exact; a^0 is 1.

#include <algorithm>
#include <type_traits>

#include "gdn_chunk_common.hpp"

namespace gdn {

namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;

// Tokens per chunk: the LDS tiles of x, y (up to 256 wide) and z fit one
// workgroup in either type.
template <typename IO> constexpr int walk_chunk() { return opstore<IO>::bytes == 2 ? 64 : 32; }

// ------------------------------------------------------------- segments ---
// A walk is cut into segments of `span` tokens (a multiple of the chunk,
// counted from each sequence's first token); one workgroup walks one segment
// of one head and column slab.  Segment slots of packed sequences are found
// from cu_seqlens by every wave for itself (lengths clamped into [0, T], so
// malformed bounds cannot send a kernel out of range).

struct Cut {
  const int32_t* cu;  // device [nseq + 1], or nullptr: dense
  int nseq, T;
  int span;           // tokens per segment
  int per_seq;        // dense: segments per sequence (>= 1)
};

struct Segment {
  int seq;       // < 0: unused slot
  int j, n;      // index among the sequence's n segments
  int64_t tok0;  // first token
  int len;       // tokens, 0 .. span
};

__device__ inline void seq_range(const Cut& c, int seq, int* st, int* en) {
  *st = min(max(c.cu[seq], 0), c.T);
  *en = min(max(c.cu[seq + 1], *st), c.T);
}

__device__ inline int seg_count(int len, int span) {
  return max(1, len / span + (len % span != 0));
}

// First segment slot of each of 64 sequences from `base` on (exclusive scan
// over the lanes), given the running total before them.
__device__ inline int lane_slots(const Cut& c, int base, int lane, int* cnt) {
  int n = 0;
  if (base + lane < c.nseq) {
    int st, en;
    seq_range(c, base + lane, &st, &en);
    n = seg_count(en - st, c.span);
  }
  *cnt = n;
  int incl = n;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(incl, d, 64);
    if (lane >= d) incl += up;
  }
  return incl - n;
}

__device__ inline Segment find_segment(const Cut& c, int slot) {
  Segment s;
  if (c.cu == nullptr) {
    s.seq = slot / c.per_seq;
    s.j = slot - s.seq * c.per_seq;
    s.n = c.per_seq;
    s.tok0 = static_cast<int64_t>(s.seq) * c.T + static_cast<int64_t>(s.j) * c.span;
    s.len = min(c.span, c.T - s.j * c.span);
    return s;
  }
  const int lane = threadIdx.x & 63;
  int before = 0;
  s.seq = -1;
  for (int base = 0; base < c.nseq; base += 64) {
    int cnt;
    const int first = before + lane_slots(c, base, lane, &cnt);
    const uint64_t hit = __ballot(slot >= first && slot < first + cnt);
    if (hit != 0) {
      const int l = __ffsll(static_cast<unsigned long long>(hit)) - 1;
      s.seq = base + l;
      s.j = slot - __shfl(first, l, 64);
      s.n = __shfl(cnt, l, 64);
      break;
    }
    before = __shfl(first + cnt, 63, 64);
  }
  s.seq = __builtin_amdgcn_readfirstlane(s.seq);
  if (s.seq < 0) return s;
  s.j = __builtin_amdgcn_readfirstlane(s.j);
  s.n = __builtin_amdgcn_readfirstlane(s.n);
  int st, en;
  seq_range(c, s.seq, &st, &en);
  s.tok0 = st + static_cast<int64_t>(s.j) * c.span;
  s.len = min(c.span, en - st - s.j * c.span);
  return s;
}

// a^n for a whole n >= 0, in 64 bits: a walk multiplies thousands of these.
__device__ inline double decay_pow(double log_a, int n) { return n == 0 ? 1.0 : exp(log_a * n); }

// ------------------------------------------------------- LDS tile reads ---
// Operand fragments from row-major LDS tiles.  `p` is a lane's own base; all
// further offsets are constants, which the reads take as immediates.

// 8 consecutive elements.
template <typename IO>
__device__ inline opvec<IO> lds_run8(const char* p) {
  if constexpr (opstore<IO>::bytes == 2) {
    return *reinterpret_cast<const bf16x8*>(p);
  } else {
    const floatx4 x = *reinterpret_cast<const floatx4*>(p);
    const floatx4 y = *reinterpret_cast<const floatx4*>(p + 16);
    return floatx8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
  }
}

// Elements 0..3 and 16..19 (the permuted K order, perm_k).
template <typename IO>
__device__ inline opvec<IO> lds_perm8(const char* p) {
  if constexpr (opstore<IO>::bytes == 2) {
    return join44(*reinterpret_cast<const uint2*>(p), *reinterpret_cast<const uint2*>(p + 32));
  } else {
    const floatx4 x = *reinterpret_cast<const floatx4*>(p);
    const floatx4 y = *reinterpret_cast<const floatx4*>(p + 64);
    return floatx8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
  }
}

// One column over the rows of a 32-row block in the permuted order (rows
// STRIDE elements apart).  16-bit tiles use the transposing LDS read:
// sixteen lanes name the 8-byte pieces of four rows of 16 columns, and lane
// i receives column i of the four rows.  col_base: a lane's base for it.
template <typename IO, int STRIDE>
__device__ inline const char* col_base(const char* t, int lane) {
  const int g = lane >> 4;
  if constexpr (opstore<IO>::bytes == 2)
    return t + ((4 * g + ((lane & 15) >> 2)) * STRIDE + 4 * (lane & 3)) * 2;
  else
    return t + (4 * g * STRIDE + (lane & 15)) * 4;
}
template <typename IO, int STRIDE>
__device__ inline opvec<IO> lds_col8(const char* p) {
  if constexpr (opstore<IO>::bytes == 2) {
    using v4 = short __attribute__((ext_vector_type(4)));
    using lds_v4 = __attribute__((address_space(3))) v4;
    const v4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4*)(p));
    const v4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4*)(p + 16 * STRIDE * 2));
    return join44(__builtin_bit_cast(uint2, a), __builtin_bit_cast(uint2, b));
  } else {
    const float* f = reinterpret_cast<const float*>(p);
    floatx8 r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = f[(e < 4 ? e : 12 + e) * STRIDE];
    return r;
  }
}

// x = parts[0] + parts[1] + parts[2] in the operand type: bf16 operands
// leave 2^-9, 2^-18, 2^-27 of x behind; fp32 operands are x itself.
template <typename IO> struct Parts;
template <> struct Parts<f32_t> {
  static constexpr int n = 1;
  floatx8 p[1];
  __device__ inline void set(int e, float x) { p[0][e] = x; }
};
template <> struct Parts<bf16_t> {
  static constexpr int n = 3;
  bf16x8 p[3];
  __device__ inline void set(int e, float x) {
    const __bf16 hi = (__bf16)x;
    const float r = x - (float)hi;
    const __bf16 mid = (__bf16)r;
    p[0][e] = hi;
    p[1][e] = mid;
    p[2][e] = (__bf16)(r - (float)mid);
  }
};

// ----------------------------------------------------------------- walk ---

struct Walk {
  Cut cut;
  const void *x, *y, *z;  // [tokens, hx, R], [tokens, hy, R], [tokens, hz, N]
  int hx, hy, hz;         // heads of each; head h of H reads h / (H / hx) ...
  int H, R, N;
  const float* log_decay;  // [H] or nullptr (a = 1)
  void* out;               // [tokens, H, N]
  int out_f32;             // 1: out is fp32 whatever the operands are
  // state in front of each (segment slot, head) in walk order: [dk, dv]
  // matrices, nullptr = zeros; `turned`: M is that matrix transposed
  const float* enter;
  int turned;
  // state behind the walk: of each (sequence, head), by its last segment in
  // walk order (OUT); of each (slot, head) but those (not OUT)
  float* behind;
};

// Tiles of a workgroup: R up to 32 NKB, slabs of NP columns.  A wave owns 16
// columns; with narrow slabs SETS groups of W waves share the output rows (OUT)
// or the state's rows.
template <typename IO, int NKB, int NP, bool OUT>
struct WalkTiles {
  static constexpr int C = walk_chunk<IO>();
  static constexpr int ob = opstore<IO>::bytes;
  static constexpr int RP = 32 * NKB, NR = 2 * NKB, NI = C / 16, NKC = C / 32;
  static constexpr int W = NP / 16;  // waves that cover the slab
  static constexpr int SETS = std::min(kWaves / W, OUT ? NI : NR);
  static constexpr int IPS = OUT ? NI / SETS : 0;   // output row tiles of a wave
  static constexpr int RPS = OUT ? NR : NR / SETS;  // state row tiles of a wave
  // LDS: row strides (elements) that spread 16 rows read 16 bytes at a time
  // (x) or by transposing reads (y, z: 32 bytes of a row) over the banks
  static constexpr int sx = RP + 16 / ob, sy = RP + (ob == 2 ? 16 : 4),
                       sz = NP + (ob == 2 ? 16 : 4);
  static constexpr int off_y = OUT ? C * sx * ob : 0, off_z = off_y + C * sy * ob,
                       off_p = off_z + C * sz * ob, off_d = off_p + (OUT ? C * C * ob : 0),
                       off_w = off_d + (C + 4) * 4, bytes = off_w + (C + 4) * 8;
  // 16-byte pieces of a row, rows per turn of the workgroup, turns
  static constexpr int px = RP * ob / 16, pz = NP * ob / 16;
  static constexpr int stepx = kThreads / px, stepz = kThreads / pz;
  static constexpr int nx = (C + stepx - 1) / stepx, nz = (C + stepz - 1) / stepz;
};

// One segment of one head and column slab.  The state sits in accumulator
// registers.  Per chunk: rows of x, y, z arrive in LDS from registers that
// were loaded during the previous chunk; x y^T on the matrix cores, decayed
// and rounded once into operand fragments in LDS; out^T = M^T x^T (from the
// state's registers, re-packed as an operand), scaled in fp32, plus
// z^T (x y^T)^T; the state update between the two.
// The update's weights go onto z in fp32, and the product is split into
// bf16 parts, so the carried state keeps the fp32 accuracy of its storage.
template <typename IO, int NKB, int NP, bool OUT, bool REV>
__global__ __launch_bounds__(kThreads) void linattn_walk_kernel(Walk a) {
  using L = WalkTiles<IO, NKB, NP, OUT>;
  constexpr int C = L::C, NI = L::NI, NKC = L::NKC, ob = L::ob, off = REV ? 0 : 1;
  __shared__ __align__(16) char lds[L::bytes];
  char* const tx = lds;
  char* const ty = lds + L::off_y;
  char* const tz = lds + L::off_z;
  char* const tp = lds + L::off_p;
  float* const dec = reinterpret_cast<float*>(lds + L::off_d);    // a^0 .. a^C
  double* const dec64 = reinterpret_cast<double*>(lds + L::off_w);

  const int nslab = (a.N + NP - 1) / NP;
  const int id = xcd_swizzle(blockIdx.x, gridDim.x);
  const int slab = id % nslab;
  const int h = (id / nslab) % a.H;
  const int slot = id / (nslab * a.H);
  const Segment seg = find_segment(a.cut, slot);
  if (seg.seq < 0) return;
  const bool last = REV ? seg.j == 0 : seg.j == seg.n - 1;  // in walk order
  if (!OUT && last) return;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, l16 = lane & 15;

  const double log_a = a.log_decay == nullptr ? 0.0 : static_cast<double>(a.log_decay[h]);
  for (int n = tid; n <= C; n += kThreads) {
    const double d = decay_pow(log_a, n);
    dec[n] = static_cast<float>(d);
    dec64[n] = d;
  }

  // this wave's columns and set; state rows r0 .., output row tiles set, set + SETS ..
  const int n0 = slab * NP;
  const int set = L::SETS == 1 ? 0 : wave / L::W, col = (wave % L::W) * 16;  // column in the slab
  const bool active = set < L::SETS && n0 + col < a.N;
  const int r0 = OUT ? 0 : set * L::RPS * 16;

  // the state in front
  floatx4 S[L::RPS];
  const float* ent = a.enter == nullptr
                         ? nullptr
                         : a.enter + (static_cast<int64_t>(slot) * a.H + h) * a.R * a.N;
#pragma unroll
  for (int rt = 0; rt < L::RPS; ++rt) {
    S[rt] = floatx4{0.f, 0.f, 0.f, 0.f};
    const int r = rt * 16 + 4 * g, n = n0 + col + l16;
    if (OUT && ent != nullptr && active && r < a.R) {
      if (a.turned) {
        S[rt] = *reinterpret_cast<const floatx4*>(ent + n * a.R + r);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) S[rt][e] = ent[(r + e) * a.N + n];
      }
    }
  }

  // Rows of the next chunk, loaded ahead into registers as 16-byte pieces.
  // Row r of the walk is token t0 + r, backwards t0 + len - 1 - r: counted
  // from the row that would be a full chunk's last, so that a lane's offsets
  // do not depend on the chunk.  Rows past len and columns past the width
  // read zeros from no memory.
  using PX = std::integral_constant<int, L::px>;
  using PZ = std::integral_constant<int, L::pz>;
  using NX = std::integral_constant<int, L::nx>;
  using NZ = std::integral_constant<int, L::nz>;
  const int nch = (seg.len + C - 1) / C;
  uint4 rx[OUT ? L::nx : 1], ry[L::nx], rz[L::nz];
  auto chunk_of = [&](int c, int64_t* t0, int* len) __attribute__((always_inline)) {
    const int w = REV ? nch - 1 - c : c;
    *t0 = seg.tok0 + static_cast<int64_t>(w) * C;
    *len = min(C, seg.len - w * C);
  };
  auto load_rows = [&](const void* base, int heads, int width, int col0, auto per_row, auto turns,
                       int64_t t0, int len, uint4* r) __attribute__((always_inline)) {
    constexpr int PR = decltype(per_row)::value, NT = decltype(turns)::value;
    constexpr int step = kThreads / PR;
    const uint32_t stride = static_cast<uint32_t>(heads) * width * ob;
    const int64_t row0 = REV ? t0 + len - C : t0;
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(
        static_cast<const char*>(base) +
            (row0 * heads + h / (a.H / heads)) * static_cast<int64_t>(width) * ob + col0 * ob,
        kOob);
    const int row = tid / PR, c16 = (tid % PR) * 16;
    const bool in = c16 < (width - col0) * ob;
    // one offset a lane, the turns' rows in the scalar offset
    const uint32_t at =
        static_cast<uint32_t>(REV ? C - 1 - row - (NT - 1) * step : row) * stride + c16;
#pragma unroll
    for (int u = 0; u < NT; ++u)
      r[u] = __builtin_bit_cast(
          uint4, __builtin_amdgcn_raw_buffer_load_b128(
                     rs, in && row + u * step < len ? at : kOob,
                     (REV ? NT - 1 - u : u) * step * stride, 0));
  };
  auto load_chunk = [&](int c) __attribute__((always_inline)) {
    int64_t t0;
    int len;
    chunk_of(c, &t0, &len);
    if constexpr (OUT) load_rows(a.x, a.hx, a.R, 0, PX(), NX(), t0, len, rx);
    load_rows(a.y, a.hy, a.R, 0, PX(), NX(), t0, len, ry);
    load_rows(a.z, a.hz, a.N, n0, PZ(), NZ(), t0, len, rz);
  };
  auto put_rows = [&](char* t, auto stride, auto per_row, auto turns, const uint4* r)
      __attribute__((always_inline)) {
    constexpr int ST = decltype(stride)::value, PR = decltype(per_row)::value,
                  NT = decltype(turns)::value, step = kThreads / PR;
    const int row = tid / PR;
    char* p = t + row * ST * ob + (tid % PR) * 16;
    if (C % step == 0 || row < C) {
#pragma unroll
      for (int u = 0; u < NT; ++u) *reinterpret_cast<uint4*>(p + u * step * ST * ob) = r[u];
    }
  };

  // lane bases of the operand reads and of the stores
  const char* const x_run = tx + (l16 * L::sx + 8 * g) * ob;
  const char* const x_perm = tx + ((set * 16 + l16) * L::sx + 4 * g) * ob;
  const char* const y_run = ty + (l16 * L::sy + 8 * g) * ob;
  const char* const y_col = col_base<IO, L::sy>(ty, lane) + r0 * ob;
  const char* const z_col = col_base<IO, L::sz>(tz, lane) + col * ob;
  const char* const p_run = tp + (set * NKC * 64 + lane) * 8 * ob;
  const int os = a.out_f32 ? 4 : ob;  // bytes per output element
  const uint32_t ostride = static_cast<uint32_t>(a.H) * a.N * os;
  const uint32_t o_lane = (REV ? 15 - l16 : l16) * ostride + (n0 + col + 4 * g) * os;

  if (nch > 0) load_chunk(0);

  for (int c = 0; c < nch; ++c) {
    int64_t t0;
    int len;
    chunk_of(c, &t0, &len);
    __syncthreads();  // the previous chunk's tiles have been read
    if constexpr (OUT)
      put_rows(tx, std::integral_constant<int, L::sx>(), PX(), NX(), rx);
    put_rows(ty, std::integral_constant<int, L::sy>(), PX(), NX(), ry);
    put_rows(tz, std::integral_constant<int, L::sz>(), PZ(), NZ(), rz);
    __syncthreads();
    if (c + 1 < nch) load_chunk(c + 1);

    if constexpr (OUT) {
      // x y^T tiles with i >= j, transposed (column i, rows j): a fragment
      // block takes two stacked j tiles; above the diagonal zeros
      for (int job = wave; job < NI * (NI + 2) / 2; job += kWaves) {
        int it = 0, first = 0;
#pragma unroll
        for (int i = 1; i < NI; ++i)
          if (job >= first + 2 * ((it >> 1) + 1)) first += 2 * ((it >> 1) + 1), it = i;
        const int jt = job - first;
        floatx4 acc = {0.f, 0.f, 0.f, 0.f};
        if (jt <= it) {
          const char* const yp = y_run + jt * 16 * L::sy * ob;
          const char* const xp = x_run + it * 16 * L::sx * ob;
#pragma unroll
          for (int kb = 0; kb < NKB; ++kb)
            acc = mma32(lds_run8<IO>(yp + kb * 32 * ob), lds_run8<IO>(xp + kb * 32 * ob), acc);
        }
        const int d = (it - jt) * 16 + l16 - 4 * g;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = d - e >= 0 ? acc[e] * dec[max(0, d - e)] : 0.f;
        *reinterpret_cast<typename acc4<IO>::type*>(
            tp + (((it * NKC + (jt >> 1)) * 64 + lane) * 8 + (jt & 1) * 4) * ob) =
            from_f4<IO>(acc);
      }
    }

    opvec<IO> zf[NKC];
    floatx4 acc[OUT ? L::IPS : 1];
    if (active) {
#pragma unroll
      for (int kb = 0; kb < NKC; ++kb)
        zf[kb] = lds_col8<IO, L::sz>(z_col + kb * 32 * L::sz * ob);
      if constexpr (OUT) {
        // M^T x^T, the state rounded once to the operand type
#pragma unroll
        for (int it = 0; it < L::IPS; ++it) acc[it] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) {
          const opvec<IO> m = pack2<IO>(S[2 * kb], S[2 * kb + 1]);
#pragma unroll
          for (int it = 0; it < L::IPS; ++it) {
            const opvec<IO> xf =
                lds_perm8<IO>(x_perm + (it * L::SETS * 16 * L::sx + kb * 32) * ob);
            acc[it] = mma32(m, xf, acc[it]);
          }
        }
#pragma unroll
        for (int it = 0; it < L::IPS; ++it) acc[it] *= dec[(set + it * L::SETS) * 16 + l16 + off];
      }
      // the state behind the chunk, where another chunk or the caller wants it
      if (!OUT || c + 1 < nch || (last && a.behind != nullptr)) {
        const double dl = dec64[len];
        const float dh = static_cast<float>(dl), dr = static_cast<float>(dl - dh);
#pragma unroll
        for (int rt = 0; rt < L::RPS; ++rt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            S[rt][e] = __builtin_fmaf(S[rt][e], dh, S[rt][e] * dr);
#pragma unroll
        for (int kb = 0; kb < NKC; ++kb) {
          Parts<IO> wz;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            wz.set(e, (float)zf[kb][e] * dec[max(0, len - off - (kb * 32 + perm_k(g, e)))]);
#pragma unroll
          for (int rt = 0; rt < L::RPS; ++rt) {
            const opvec<IO> yf =
                lds_col8<IO, L::sy>(y_col + (kb * 32 * L::sy + rt * 16) * ob);
#pragma unroll
            for (int u = 0; u < Parts<IO>::n; ++u) S[rt] = mma32(yf, wz.p[u], S[rt]);
            // a state of over 128 rows leaves no registers for reads far ahead
            if constexpr (NKB > 4)
              if (rt % 4 == 3) __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
    }

    if constexpr (OUT) {
      __syncthreads();  // x y^T is in LDS
      if (active) {
        // uniform base of the chunk's rows (backwards: of a full chunk's)
        char* const orow = static_cast<char*>(a.out) +
                           ((REV ? t0 + len - C : t0) * a.H + h) * static_cast<int64_t>(a.N) * os;
#pragma unroll
        for (int u = 0; u < L::IPS; ++u) {
          const int it = set + u * L::SETS;
#pragma unroll
          for (int kb = 0; kb < NKC; ++kb) {
            if (kb > it / 2) continue;
            const opvec<IO> pf = lds_run8<IO>(p_run + (u * L::SETS * NKC + kb) * 512 * ob);
            acc[u] = mma32(zf[kb], pf, acc[u]);
          }
          char* const orow_it =
              orow + static_cast<int64_t>((REV ? C / 16 - 1 - it : it) * 16) * ostride;
          if (it * 16 + l16 < len) {
            char* const p = orow_it + o_lane;
            if (ob == 4 || a.out_f32)
              *reinterpret_cast<floatx4*>(p) = acc[u];
            else
              *reinterpret_cast<typename acc4<IO>::type*>(p) = from_f4<IO>(acc[u]);
          }
        }
      }
    }
  }

  float* bh = a.behind;
  if (bh != nullptr && active && (OUT ? last && set == 0 : true)) {
    const int64_t at = OUT ? static_cast<int64_t>(seg.seq) * a.H + h
                           : static_cast<int64_t>(slot) * a.H + h;
    bh += at * a.R * a.N;
#pragma unroll
    for (int rt = 0; rt < L::RPS; ++rt) {
      const int r = r0 + rt * 16 + 4 * g, n = n0 + col + l16;
      if (r >= a.R) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) bh[(r + e) * a.N + n] = S[rt][e];
    }
  }
}

// -------------------------------------------------------------- combine ---
// The state in front of every segment, in place: buf[slot, h] holds each
// segment's own contribution (all but the last in walk order) and becomes
// the state entering it,  E' = a^len E + own.  A thread carries four state
// elements through the sequence's segments; loads run ahead of the chain.
template <bool REV>
__global__ __launch_bounds__(256) void linattn_combine_kernel(Cut cut, int H, int elems,
                                                              const float* log_decay,
                                                              const float* init, float* buf) {
  const int nblk = (elems / 4 + 255) / 256;
  const int blk = blockIdx.x % nblk;
  const int h = (blockIdx.x / nblk) % H;
  const int seq = blockIdx.x / (nblk * H);
  int first, n, len;
  if (cut.cu == nullptr) {
    n = cut.per_seq;
    first = seq * n;
    len = cut.T;
  } else {
    const int lane = threadIdx.x & 63;
    int before = 0, f = 0, cnt = 0;
    for (int base = 0; base <= seq; base += 64) {
      f = before + lane_slots(cut, base, lane, &cnt);
      before = __shfl(f + cnt, 63, 64);
    }
    first = __shfl(f, seq & 63, 64);
    n = __shfl(cnt, seq & 63, 64);
    int st, en;
    seq_range(cut, seq, &st, &en);
    len = en - st;
  }
  const int e4 = blk * 256 + threadIdx.x;
  if (e4 >= elems / 4) return;
  const double log_a = log_decay == nullptr ? 0.0 : static_cast<double>(log_decay[h]);
  const double ds = decay_pow(log_a, cut.span);
  const double dt = decay_pow(log_a, len - (n - 1) * cut.span);  // the last segment's

  floatx4 E = {0.f, 0.f, 0.f, 0.f};
  if (init != nullptr)
    E = *reinterpret_cast<const floatx4*>(init + (static_cast<int64_t>(seq) * H + h) * elems +
                                          4 * e4);
  auto at = [&](int w) {  // w: index in walk order
    const int j = REV ? n - 1 - w : w;
    return reinterpret_cast<floatx4*>(
        buf + (static_cast<int64_t>(first + j) * H + h) * elems + 4 * e4);
  };
  constexpr int kAhead = 8;
  for (int w0 = 0; w0 < n; w0 += kAhead) {
    floatx4 own[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (w0 + u < n - 1) own[u] = *at(w0 + u);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (w0 + u >= n) break;
      *at(w0 + u) = E;
      const double d = REV && w0 + u == 0 ? dt : ds;
      if (w0 + u < n - 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          E[e] = static_cast<float>(d * static_cast<double>(E[e]) + static_cast<double>(own[u][e]));
      }
    }
  }
}

// ---------------------------------------------------------- shared heads ---
// Gradient of a q or k head: the sum over the v heads that read it, in head
// order, from the fp32 rows of each (part: [tokens, H, d] -> out
// [tokens, Hq, d]).  Tokens behind the last sequence are left alone.
template <typename IO>
__global__ __launch_bounds__(256) void linattn_share_kernel(const float* part, void* out,
                                                            int64_t tokens, int Hq, int grp,
                                                            int d, const int32_t* cu, int nseq) {
  if (cu != nullptr) tokens = min(tokens, static_cast<int64_t>(max(cu[nseq], 0)));
  const int p4 = d / 4;
  const int64_t total = tokens * Hq * p4;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t row = i / p4;  // token * Hq + head
    const int c = static_cast<int>(i - row * p4) * 4;
    floatx4 s = *reinterpret_cast<const floatx4*>(part + row * grp * d + c);
    for (int j = 1; j < grp; ++j)
      s += *reinterpret_cast<const floatx4*>(part + (row * grp + j) * d + c);
    *reinterpret_cast<typename acc4<IO>::type*>(static_cast<char*>(out) +
                                                (row * d + c) * opstore<IO>::bytes) =
        from_f4<IO>(s);
  }
}

// --------------------------------------------------------------- decode ---
// M <- a M + k v^T, o = M^T q: every state element read once and written
// once in 16-byte pieces; a workgroup takes one (sequence, head) and 64
// columns, a thread DK / 16 rows of 4 columns.  No step waits for another
// before the store, so only the reading and writing of the state bounds it.
template <int DK, typename IO>
__global__ __launch_bounds__(256) void linattn_decode_kernel(
    int H, int grp, int dv, const void* __restrict__ q, const void* __restrict__ k,
    const void* __restrict__ v, const float* __restrict__ log_decay, float* __restrict__ state,
    void* __restrict__ o) {
  constexpr int RPT = DK / 16;
  const int nslab = (dv + 63) / 64;
  const int nh = blockIdx.x / nslab;  // sequence * H + head
  const int slab = blockIdx.x - nh * nslab;
  const int n = nh / H, h = nh - n * H;
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
  const int col = slab * 64 + cg * 4;
  const bool active = col < dv;
  float* M = state + static_cast<int64_t>(nh) * DK * dv + col;
  floatx4 m[RPT];
#pragma unroll
  for (int j = 0; j < RPT; ++j)
    m[j] = active ? __builtin_nontemporal_load(
                        reinterpret_cast<const floatx4*>(M + (rg + 16 * j) * dv))
                  : floatx4{0.f, 0.f, 0.f, 0.f};
  const int64_t qo = (static_cast<int64_t>(n) * (H / grp) + h / grp) * DK;
  const int64_t vo = static_cast<int64_t>(nh) * dv + col;
  const float a =
      log_decay == nullptr ? 1.0f : static_cast<float>(exp(static_cast<double>(log_decay[h])));
  floatx4 vv = {0.f, 0.f, 0.f, 0.f}, w = vv;
  if (active) {
#pragma unroll
    for (int c = 0; c < 4; ++c) vv[c] = io<IO>::load(v, vo + c);
  }
#pragma unroll
  for (int j = 0; j < RPT; ++j) {
    const int r = rg + 16 * j;
    const float kr = io<IO>::load(k, qo + r), qr = io<IO>::load(q, qo + r);
#pragma unroll
    for (int c = 0; c < 4; ++c) m[j][c] = __builtin_fmaf(a, m[j][c], kr * vv[c]);
    w += m[j] * qr;
    if (active)
      __builtin_nontemporal_store(m[j], reinterpret_cast<floatx4*>(M + r * dv));
  }
  // over the 16 row groups: 4 in the wave, then the 4 waves through LDS
#pragma unroll
  for (int c = 0; c < 4; ++c) w[c] = wave_sum_xor(w[c], 48);
  __shared__ floatx4 sw[4][16];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if (lane < 16) sw[wave][lane] = w;
  __syncthreads();
  if (threadIdx.x < 16 && active) {
    w = sw[0][cg] + sw[1][cg] + sw[2][cg] + sw[3][cg];
    *reinterpret_cast<typename acc4<IO>::type*>(static_cast<char*>(o) +
                                                vo * opstore<IO>::bytes) = from_f4<IO>(w);
  }
}

// ------------------------------------------------------------- launches ---

size_t al256(size_t x) { return (x + 255) & ~size_t(255); }

// Segments of a walk, from sizes alone.
struct Plan {
  int span;        // tokens per segment
  int per_seq;     // dense: segments per sequence
  int64_t slots;   // segment slots (an upper bound when packed)
  bool split;
};

Plan plan_walk(const LinAttn& p) {
  const int C = p.io == GDN_BF16 ? 64 : 32;
  Plan r;
  const int64_t nch = (static_cast<int64_t>(p.T) + C - 1) / C;  // of one dense sequence, or all
  const int64_t slabs = (p.dv + 127) / 128;
  int64_t L = nch;  // chunks per segment
  if (p.seg_req > 0) {
    L = std::min<int64_t>(nch, p.seg_req);
  } else if (p.seg_req == 0) {
    // workgroups when nothing is split: one chain of chunks each
    const int64_t total = nch * (p.varlen ? 1 : p.nseq) * p.H * slabs;
    const int64_t fill = (total + 255) / 256;
    L = std::max<int64_t>(fill, 2);
    if (!p.varlen && static_cast<int64_t>(p.nseq) * p.H * slabs >= 256) L = nch;
    L = std::min(L, nch);
  }
  L = std::max<int64_t>(L, 1);
  r.split = L < nch;
  r.span = static_cast<int>(std::min<int64_t>(r.split ? L * C : int64_t(1) << 30, 1 << 30));
  r.per_seq = r.split ? static_cast<int>((nch + L - 1) / L) : 1;
  if (p.varlen)
    r.slots = r.split ? p.T / r.span + p.nseq : p.nseq;
  else
    r.slots = static_cast<int64_t>(p.nseq) * r.per_seq;
  return r;
}

Cut make_cut(const LinAttn& p, const Plan& pl) {
  return Cut{p.varlen ? p.cu_seqlens : nullptr, p.nseq, p.T, pl.span, pl.per_seq};
}

template <typename IO, int NKB, int NP, bool OUT, bool REV>
void launch_walk_t(const Walk& w, int64_t slots, hipStream_t s) {
  const int64_t nslab = (w.N + NP - 1) / NP;
  hipLaunchKernelGGL((linattn_walk_kernel<IO, NKB, NP, OUT, REV>),
                     dim3(static_cast<unsigned>(slots * w.H * nslab)), dim3(kThreads), 0, s, w);
}

template <typename IO, int NKB, bool OUT, bool REV>
void launch_walk_n(const Walk& w, int64_t slots, hipStream_t s) {
  if (w.N <= 32) return launch_walk_t<IO, NKB, 32, OUT, REV>(w, slots, s);
  if (w.N <= 64) return launch_walk_t<IO, NKB, 64, OUT, REV>(w, slots, s);
  launch_walk_t<IO, NKB, 128, OUT, REV>(w, slots, s);
}

template <typename IO, bool OUT, bool REV>
void launch_walk_io(const Walk& w, int64_t slots, hipStream_t s) {
  if (w.R > 128) {
    if constexpr (OUT) return launch_walk_n<IO, 8, OUT, REV>(w, slots, s);
  }
  if (w.R > 64) return launch_walk_n<IO, 4, OUT, REV>(w, slots, s);
  if (w.R > 32) return launch_walk_n<IO, 2, OUT, REV>(w, slots, s);
  launch_walk_n<IO, 1, OUT, REV>(w, slots, s);
}

hipError_t launch_walk(const LinAttn& p, const Walk& w, int64_t slots, bool out, bool rev,
                       int stage, hipStream_t s) {
  StageScope scope(stage, s);
  if (p.io == GDN_BF16) {
    if (out)
      rev ? launch_walk_io<bf16_t, true, true>(w, slots, s)
          : launch_walk_io<bf16_t, true, false>(w, slots, s);
    else
      rev ? launch_walk_io<bf16_t, false, true>(w, slots, s)
          : launch_walk_io<bf16_t, false, false>(w, slots, s);
  } else {
    if (out)
      rev ? launch_walk_io<f32_t, true, true>(w, slots, s)
          : launch_walk_io<f32_t, true, false>(w, slots, s);
    else
      rev ? launch_walk_io<f32_t, false, true>(w, slots, s)
          : launch_walk_io<f32_t, false, false>(w, slots, s);
  }
  return hipGetLastError();
}

hipError_t launch_combine(const LinAttn& p, const Cut& cut, bool rev, const float* la,
                          const float* init, float* buf, hipStream_t s) {
  StageScope scope(GDN_STAGE_FWD_COMBINE, s);
  const int elems = p.dk * p.dv;
  const int64_t grid = static_cast<int64_t>(p.nseq) * p.H * ((elems / 4 + 255) / 256);
  if (rev)
    hipLaunchKernelGGL(linattn_combine_kernel<true>, dim3(static_cast<unsigned>(grid)), dim3(256),
                       0, s, cut, p.H, elems, la, init, buf);
  else
    hipLaunchKernelGGL(linattn_combine_kernel<false>, dim3(static_cast<unsigned>(grid)),
                       dim3(256), 0, s, cut, p.H, elems, la, init, buf);
  return hipGetLastError();
}

// States in front of every segment into `buf`: own contributions, chained.
hipError_t enter_states(const LinAttn& p, const Plan& pl, bool rev, const void* y, const void* z,
                        int hy, int hz, const float* la, const float* init, float* buf,
                        hipStream_t s) {
  Walk w{};
  w.cut = make_cut(p, pl);
  w.y = y;
  w.z = z;
  w.hx = p.H;
  w.hy = hy;
  w.hz = hz;
  w.H = p.H;
  w.R = p.dk;
  w.N = p.dv;
  w.log_decay = la;
  w.behind = buf;
  hipError_t e = launch_walk(p, w, pl.slots, false, rev, GDN_STAGE_FWD_TRANS, s);
  if (e != hipSuccess) return e;
  return launch_combine(p, w.cut, rev, la, init, buf, s);
}

size_t state_bytes(const LinAttn& p, const Plan& pl) {
  return pl.split ? al256(static_cast<size_t>(pl.slots) * p.H * p.dk * p.dv * 4) : 0;
}

size_t part_bytes(const LinAttn& p) {
  return p.hq == p.H ? 0 : al256(static_cast<size_t>(p.B) * p.T * p.H * p.dk * 4);
}

template <int DK>
void launch_decode_dk(const LinAttn& p, const void* q, const void* k, const void* v,
                      const float* la, float* state, void* o, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(p.B) * p.H * ((p.dv + 63) / 64)));
  if (p.io == GDN_BF16)
    hipLaunchKernelGGL((linattn_decode_kernel<DK, bf16_t>), grid, dim3(256), 0, s, p.H,
                       p.H / p.hq, p.dv, q, k, v, la, state, o);
  else
    hipLaunchKernelGGL((linattn_decode_kernel<DK, f32_t>), grid, dim3(256), 0, s, p.H,
                       p.H / p.hq, p.dv, q, k, v, la, state, o);
}

}  // namespace

bool linattn_grid_ok(const LinAttn& p) {
  const Plan pl = plan_walk(p);
  const int64_t most = (int64_t(1) << 31) - 1;
  const int64_t blocks = (static_cast<int64_t>(p.dk) * p.dv / 4 + 255) / 256;
  return pl.slots * p.H * 2 <= most && static_cast<int64_t>(p.nseq) * p.H * blocks <= most;
}

size_t linattn_fwd_workspace_bytes(const LinAttn& p) { return state_bytes(p, plan_walk(p)); }

hipError_t launch_linattn_fwd(const LinAttn& p, const void* q, const void* k, const void* v,
                              const float* la, const float* s0, void* o, float* s_final,
                              void* ws, hipStream_t s) {
  const Plan pl = plan_walk(p);
  Walk w{};
  w.cut = make_cut(p, pl);
  w.enter = s0;
  if (pl.split) {
    float* buf = static_cast<float*>(ws);
    const hipError_t e = enter_states(p, pl, false, k, v, p.hq, p.H, la, s0, buf, s);
    if (e != hipSuccess) return e;
    w.enter = buf;
  }
  w.x = q;
  w.y = k;
  w.z = v;
  w.hx = w.hy = p.hq;
  w.hz = w.H = p.H;
  w.R = p.dk;
  w.N = p.dv;
  w.log_decay = la;
  w.out = o;
  w.behind = s_final;
  return launch_walk(p, w, pl.slots, true, false, GDN_STAGE_FWD_SCAN, s);
}

size_t linattn_bwd_workspace_bytes(const LinAttn& p) {
  return 2 * state_bytes(p, plan_walk(p)) + 2 * part_bytes(p);
}

hipError_t launch_linattn_bwd(const LinAttn& p, const void* q, const void* k, const void* v,
                              const float* la, const float* s0, const void* d_o,
                              const float* ds_final, void* dq, void* dk, void* dv, float* ds0,
                              void* ws, hipStream_t s) {
  const Plan pl = plan_walk(p);
  const float *front = s0, *back = ds_final;
  char* at = static_cast<char*>(ws);
  hipError_t e;
  if (pl.split) {
    float* bf = reinterpret_cast<float*>(at);
    at += state_bytes(p, pl);
    float* bb = reinterpret_cast<float*>(at);
    at += state_bytes(p, pl);
    e = enter_states(p, pl, false, k, v, p.hq, p.H, la, s0, bf, s);
    if (e != hipSuccess) return e;
    e = enter_states(p, pl, true, q, d_o, p.hq, p.H, la, ds_final, bb, s);
    if (e != hipSuccess) return e;
    front = bf;
    back = bb;
  }
  const bool shared = p.hq != p.H;
  float* part_q = reinterpret_cast<float*>(at);
  float* part_k = reinterpret_cast<float*>(at + part_bytes(p));

  Walk w{};
  w.cut = make_cut(p, pl);
  w.H = p.H;
  w.log_decay = la;
  w.out_f32 = shared ? 1 : 0;
  w.turned = 1;
  w.R = p.dv;
  w.N = p.dk;
  w.hx = w.hy = p.H;
  w.hz = p.hq;
  // dq
  w.x = d_o;
  w.y = v;
  w.z = k;
  w.enter = front;
  w.out = shared ? static_cast<void*>(part_q) : dq;
  e = launch_walk(p, w, pl.slots, true, false, GDN_STAGE_BWD_GRAD, s);
  if (e != hipSuccess) return e;
  // dk
  w.x = v;
  w.y = d_o;
  w.z = q;
  w.enter = back;
  w.out = shared ? static_cast<void*>(part_k) : dk;
  e = launch_walk(p, w, pl.slots, true, true, GDN_STAGE_BWD_GRAD, s);
  if (e != hipSuccess) return e;
  // dv
  w.turned = 0;
  w.out_f32 = 0;
  w.R = p.dk;
  w.N = p.dv;
  w.hx = w.hy = p.hq;
  w.hz = p.H;
  w.x = k;
  w.y = q;
  w.z = d_o;
  w.out = dv;
  w.behind = ds0;
  e = launch_walk(p, w, pl.slots, true, true, GDN_STAGE_BWD_GRAD, s);
  if (e != hipSuccess) return e;
  if (!shared) return hipSuccess;
  const int64_t tok = static_cast<int64_t>(p.B) * p.T;
  const int64_t pieces = tok * p.hq * (p.dk / 4);
  if (pieces == 0) return hipSuccess;
  StageScope scope(GDN_STAGE_OTHER, s);
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>((pieces + 255) / 256, 4096)));
  for (int u = 0; u < 2; ++u) {
    const float* part = u == 0 ? part_q : part_k;
    void* out = u == 0 ? dq : dk;
    const int32_t* cu = p.varlen ? p.cu_seqlens : nullptr;
    if (p.io == GDN_BF16)
      hipLaunchKernelGGL(linattn_share_kernel<bf16_t>, grid, dim3(256), 0, s, part, out, tok,
                         p.hq, p.H / p.hq, p.dk, cu, p.nseq);
    else
      hipLaunchKernelGGL(linattn_share_kernel<f32_t>, grid, dim3(256), 0, s, part, out, tok, p.hq,
                         p.H / p.hq, p.dk, cu, p.nseq);
  }
  return hipGetLastError();
}

hipError_t launch_linattn_decode(const LinAttn& p, const void* q, const void* k, const void* v,
                                 const float* la, float* state, void* o, hipStream_t s) {
  StageScope scope(GDN_STAGE_DECODE, s);
  switch (p.dk) {
    case 16: launch_decode_dk<16>(p, q, k, v, la, state, o, s); break;
    case 32: launch_decode_dk<32>(p, q, k, v, la, state, o, s); break;
    case 64: launch_decode_dk<64>(p, q, k, v, la, state, o, s); break;
    default: launch_decode_dk<128>(p, q, k, v, la, state, o, s); break;
  }
  return hipGetLastError();
}

}  // namespace gdn
