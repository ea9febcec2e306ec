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
// so one kernel serves all four (rev: rows taken from the end; the entering
// state then reaches the first walked token undecayed, and the state handed
// on is multiplied by a once more).
//
// Chunk form over C tokens (i, j: rows in walk order, off = 1, rev: 0):
//   out_i = a^{i+off} M_in^T x_i + sum_{j<=i} a^{i-j} (x_i . y_j) z_j
//   M_out = a^len M_in + sum_j a^{len-off-j} y_j z_j^T
// Every power of a has a non-negative exponent, so no factor overflows for
// a <= 1 and a = 0 (log_decay = -inf) is exact; a^0 is 1.
//
// A long sequence with few heads is cut into segments: one launch walks the
// segments' own states (no outputs), one chains them, one walks the outputs
// from the chained states (plan_walk).  The whole needs 4 dk dv flops a token
// and head for 4 rows of bytes (bf16 128 x 128: 64 flops a byte), so memory
// bounds large calls: 65k packed tokens of 16 heads take 414 us for 1.09 GB
// that must move (2.6 TB/s; 1.7 GB with k and v read twice and the states,
// 4.2 TB/s).  Small ones are bound by the chain: a workgroup's chunk has
// three barriers and takes 3.1 to 4.7 us alone on its CU.

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "gdn_chunk_common.hpp"

namespace gdn {

namespace {

// Tokens per chunk: the LDS tiles of x, y (up to 256 wide) and z fit one
// workgroup in either type.
template <typename IO> constexpr int walk_chunk() { return opstore<IO>::bytes == 2 ? 64 : 32; }

// ------------------------------------------------------------- segments ---
// A walk is cut into segments of `span` tokens (a multiple of the chunk,
// counted from each sequence's first token); one workgroup walks one segment
// of one head and column slab.  Of a packed batch only sequences longer than
// `span` are cut: their segments take the first `slots` slots, found from
// cu_seqlens by every wave for itself, and slot slots + i is sequence i where
// it is walked whole (lengths clamped into [0, T], so malformed bounds cannot
// send a kernel out of range).

struct Cut {
  const int32_t* cu;  // device [nseq + 1], or nullptr: dense
  int nseq, T;
  int span;           // tokens per segment
  int per_seq;        // dense: segments per sequence (>= 1)
  int64_t slots;      // segment slots there is room for (packed: of cut sequences)
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

// Segments of a packed sequence that is cut, 0 for one that is not.
__device__ inline int cut_count(int len, int span) {
  return len <= span ? 0 : len / span + (len % span != 0);
}

// Cut sequences' slots of 64 sequences from `base` on in front of each
// (exclusive scan over the lanes).  Bounds that overlap could add up to more
// slots than there are: 64 counts of at most 2^25 + 1 and a total held at
// `slots` (< 2^29) stay below 2^32.
__device__ inline uint32_t lane_slots(const Cut& c, int base, int lane, uint32_t* cnt) {
  uint32_t n = 0;
  if (base + lane < c.nseq) {
    int st, en;
    seq_range(c, base + lane, &st, &en);
    n = cut_count(en - st, c.span);
  }
  *cnt = n;
  uint32_t incl = n;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t up = __shfl_up(incl, d, 64);
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
  int st, en;
  if (slot >= c.slots) {
    s.seq = slot - static_cast<int>(c.slots);
    seq_range(c, s.seq, &st, &en);
    s.j = 0;
    s.n = 1;
    s.tok0 = st;
    s.len = en - st;
    if (s.len > c.span) s.seq = -1;
    return s;
  }
  const int lane = threadIdx.x & 63;
  uint32_t before = 0, cnt;
  s.seq = -1;
  for (int base = 0; base < c.nseq; base += 64) {
    const uint32_t first = before + lane_slots(c, base, lane, &cnt);
    const uint32_t at = static_cast<uint32_t>(slot);
    const uint64_t hit = __ballot(at >= first && at < first + cnt);
    if (hit != 0) {
      const int l = __ffsll(static_cast<unsigned long long>(hit)) - 1;
      s.seq = base + l;
      s.j = slot - __shfl(first, l, 64);
      s.n = __shfl(cnt, l, 64);
      break;
    }
    before = min(__shfl(first + cnt, 63, 64), static_cast<uint32_t>(c.slots));
  }
  s.seq = __builtin_amdgcn_readfirstlane(s.seq);
  if (s.seq < 0) return s;
  s.j = __builtin_amdgcn_readfirstlane(s.j);
  s.n = __builtin_amdgcn_readfirstlane(s.n);
  seq_range(c, s.seq, &st, &en);
  s.tok0 = st + static_cast<int64_t>(s.j) * c.span;
  s.len = min(c.span, en - st - s.j * c.span);
  return s;
}

// a^n for a whole n >= 0, in 64 bits: a walk multiplies thousands of these.
__device__ inline double decay_pow(double log_a, int n) { return n == 0 ? 1.0 : exp(log_a * n); }

// a^n in 32 bits: the exponent is reduced in 64, so that the hardware's
// exponential (one unit in the last place) sees a fraction of [0, 1).
__device__ inline float decay_pow32(double log_a, int n) {
  const double x = log_a * n * 1.4426950408889634;
  const double w = floor(x);
  const float r = ldexpf(__builtin_amdgcn_exp2f(static_cast<float>(x - w)),
                         static_cast<int>(fmin(fmax(w, -1000.0), 1000.0)));
  return n == 0 ? 1.0f : x < -1000.0 ? 0.0f : r;
}

// A uniform element of a read-only array by a scalar load.
__device__ inline float ld_scalar(const float* p, int i) {
  return ((const __attribute__((address_space(4))) float*)(p))[i];
}

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
// Column i of the 16 is element GAP (i / 4) + i % 4 from the base; rows
// 4 g .. 4 g + 3 (and 16 further down) start SKEW g elements in.
template <typename IO, int STRIDE, int GAP, int SKEW>
__device__ inline const char* col_base(const char* t, int lane) {
  const int g = lane >> 4, l16 = lane & 15;
  if constexpr (opstore<IO>::bytes == 2)
    return t + ((4 * g + (l16 >> 2)) * STRIDE + SKEW * g + GAP * (lane & 3)) * 2;
  else
    return t + (4 * g * STRIDE + GAP * (l16 >> 2) + (l16 & 3)) * 4;
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

// A column of 8 weighted values as operand parts.  bf16: N parts after
// SKIP earlier ones.  Each keeps 8 bits rounded to nearest, so one leaves at
// most 2^-8 of the value, two 2^-17 (the rest's sign carries the ninth bit),
// and three hold the 24 bits of an fp32 one (a product whose rest is formed
// by a fused multiply-add may keep bits behind those: 1e-9 of a state, which
// its fp32 sums do not hold).  fp32 operands are the value itself.
template <typename IO> struct Parts;
template <> struct Parts<f32_t> {
  static constexpr int most = 1;
  floatx8 p[1];
  template <int N, int SKIP> __device__ inline void set(const floatx8& z, const float* w) {
#pragma unroll
    for (int e = 0; e < 8; ++e) p[0][e] = z[e] * w[e];
  }
};
template <> struct Parts<bf16_t> {
  static constexpr int most = 3;
  bf16x8 p[3];
  template <int N, int SKIP> __device__ inline void set(const bf16x8& z, const float* w) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    u32x4 out[N];
    const u32x4 in = __builtin_bit_cast(u32x4, z);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a = __uint_as_float(in[e] << 16) * w[2 * e];
      float b = __uint_as_float(in[e] & 0xffff0000u) * w[2 * e + 1];
      auto round = [&]() __attribute__((always_inline)) {
        return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
      };
      auto rest = [&](uint32_t r) __attribute__((always_inline)) {
        a -= __uint_as_float(r << 16);
        b -= __uint_as_float(r & 0xffff0000u);
      };
#pragma unroll
      for (int u = 0; u < SKIP; ++u) rest(round());
#pragma unroll
      for (int u = 0; u < N; ++u) {
        out[u][e] = round();
        if (u + 1 < N) rest(out[u][e]);
      }
    }
#pragma unroll
    for (int u = 0; u < N; ++u) p[u] = __builtin_bit_cast(bf16x8, out[u]);
  }
};

// What a rounding of two stacked tiles left behind, rounded in turn.
__device__ inline bf16x8 pack2_rest(const floatx4& lo, const floatx4& hi, const bf16x8& r) {
  const u32x4 u = __builtin_bit_cast(u32x4, r);
  floatx4 a, b;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    a[2 * e] = lo[2 * e] - __uint_as_float(u[e] << 16);
    a[2 * e + 1] = lo[2 * e + 1] - __uint_as_float(u[e] & 0xffff0000u);
    b[2 * e] = hi[2 * e] - __uint_as_float(u[2 + e] << 16);
    b[2 * e + 1] = hi[2 * e + 1] - __uint_as_float(u[2 + e] & 0xffff0000u);
  }
  return pack2<bf16_t>(a, b);
}

// ----------------------------------------------------------------- walk ---

struct Walk {
  Cut cut;
  int rev;                // from the last token back
  const void *x, *y, *z;  // [tokens, hx, R], [tokens, hy, R], [tokens, hz, N]
  int hx, hy, hz;         // heads of each; head h of H reads h / (H / hx) ...
  int H, R, N;
  const float* log_decay;  // [H] or nullptr (a = 1)
  void* out;               // [tokens, H, N]
  int out_f32;             // 1: out is fp32 whatever the operands are
  // state in front in walk order, [dk, dv] matrices: of each (sequence, head)
  // (nullptr = zeros), taken where a segment is the whole sequence, and of
  // each (segment slot, head); `turned`: M is that matrix transposed
  const float *init, *enter;
  int turned;
  // enter (OUT) and behind (not OUT) in register order instead: per 32 columns
  // (16 where N <= 64) and 16 rows, two tiles (one) of 64 lanes' four rows
  int image;
  // state behind the walk: of each (sequence, head), where a segment is the
  // whole sequence (OUT; nullptr = not wanted); of each (slot, head), the last
  // ones in walk order only if `ends` (not OUT)
  float* behind;
  int ends;
};

// Tiles of a workgroup: R up to 32 NKB, slabs of NP columns (launch_walk_n).
// A wave owns CT 16-column tiles; with narrow slabs SETS groups of W waves
// share the output rows (OUT) or the state's rows.
template <typename IO, int NKB, int NP, bool OUT>
struct WalkTiles {
  static constexpr int C = walk_chunk<IO>();
  static constexpr int ob = opstore<IO>::bytes;
  static constexpr int RP = 32 * NKB, NR = 2 * NKB, NI = C / 16, NKC = C / 32;
  // two column tiles a wave halve the operand reads; a state of over 128
  // rows leaves no registers for them and takes eight waves instead of four
  static constexpr int CT = NP > 64 && NKB <= 4 ? 2 : 1;
  static constexpr int waves = NP > 64 && NKB > 4 ? 8 : 4, threads = 64 * waves;
  static constexpr int W = NP / (16 * CT);
  static constexpr int SETS = std::min(waves / W, OUT ? NI : NR);
  static constexpr int IPS = OUT ? NI / SETS : 0;   // output row tiles of a wave
  static constexpr int RPS = OUT ? NR : NR / SETS;  // state row tiles of a wave
  // LDS: row strides (elements) that spread 16 rows read 16 bytes at a time
  // (x) or by transposing reads (y, z: 32 bytes of a row) over the banks
  static constexpr int sx = RP + 16 / ob, sy = RP + (ob == 2 ? 16 : 4),
                       sz = NP + (ob == 2 ? 16 : 4);
  // (the small tables lie in front: a read's immediate reaches 64 KB)
  static constexpr int off_d = 0, off_w = off_d + (32 + C + 4) * 4, off_x = off_w + C * 4,
                       off_y = off_x + (OUT ? C * sx * ob : 0), off_z = off_y + C * sy * ob,
                       off_p = off_z + C * sz * ob, bytes = off_p + (OUT ? C * C * 4 : 0);
  // y rows shift by 8 bytes every four rows (in the row's padding): 16 rows
  // read 8 bytes at a time then meet all banks, as the transposing reads do
  static constexpr int skew = ob == 2 ? 4 : 0;
  // 16-byte pieces of a row, rows per turn of the workgroup, turns
  static constexpr int px = RP * ob / 16, pz = NP * ob / 16;
  static constexpr int nx = (C * px + threads - 1) / threads,
                       nz = (C * pz + threads - 1) / threads;
};

// One segment of one head and column slab.  The state sits in accumulator
// registers.  Per chunk: rows of x, y, z arrive in LDS from registers that
// were loaded during the previous chunk; x y^T on the matrix cores, decayed
// and split into operand fragments in LDS; out^T = M^T x^T (from the
// state's registers, re-packed as an operand), scaled in fp32, plus
// z^T (x y^T)^T, stored at once; the state update last, while the stores
// drain.
// Alone on a CU a workgroup (four waves, one a SIMD) waits most of a chunk
// (matrix cores 17 % busy); two share it where there is work for them (32 %,
// 65k tokens), which memory then bounds: 267 us for 1.1 GB.  (With one part of
// the state's copy 256; eight waves instead of four took 315 then, one copy of
// the code for both directions 283.)
// The update's weights go onto z in fp32, and the product is split into
// bf16 parts, so the carried state keeps the fp32 accuracy of its storage.
// Operand reads run one step ahead of the products that take them
// (scheduling barriers hold them there).
// One launch takes up to three walks of the same tiles (a backward's), so
// that short ones share the machine.
struct Walks {
  Walk w[3];
  int n;
};

template <typename IO, int NKB, int NP, bool OUT, bool rev>
__device__ __forceinline__ void walk_segment(const Walk& a, int slab, int h, int slot, char* lds) {
  using L = WalkTiles<IO, NKB, NP, OUT>;
  constexpr int C = L::C, NI = L::NI, NKC = L::NKC, CT = L::CT, ob = L::ob, off = rev ? 0 : 1;
  constexpr int kThreads = L::threads;
  char* const tx = lds + L::off_x;
  char* const ty = lds + L::off_y;
  char* const tz = lds + L::off_z;
  char* const tp = lds + L::off_p;
  float* const dec = reinterpret_cast<float*>(lds + L::off_d) + 32;  // a^0 .. a^C, 0 below
  float* const wgt = reinterpret_cast<float*>(lds + L::off_w);       // update weights of rows

  const Segment seg = find_segment(a.cut, slot);
  if (seg.seq < 0) return;
  const bool last = rev ? seg.j == 0 : seg.j == seg.n - 1;  // in walk order
  if (!OUT && last && !a.ends) return;
  // (lane 0's, as everything here is the wave's: the state's descriptor is then
  // known to be one for all lanes)
  const bool whole = __builtin_amdgcn_readfirstlane(seg.n) == 1;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, l16 = lane & 15;

  // this wave's columns and set; state rows r0 .., output row tiles set, set + SETS ..
  const int n0 = slab * NP;
  // (two tiles interleave by fours, so that a lane's outputs are 8 adjacent columns)
  const int set = L::SETS == 1 ? 0 : wave / L::W, col = (wave % L::W) * CT * 16;
  const int n_lane = n0 + col + (CT == 2 ? 8 * (l16 >> 2) + (l16 & 3) : l16);
  const bool active = set < L::SETS && n0 + col < a.N;
  const int r0 = OUT ? 0 : set * L::RPS * 16;

  // this lane's place in a state in register order, bytes between row tiles
  // (a wave of one column tile finds its columns among the interleaved two)
  const bool wide = a.N > 64;
  const uint32_t image_elems = (wide ? (a.N + 31) / 32 * 32 : a.N) * a.R;
  const uint32_t image_step = wide ? 2048 : 1024;
  auto image_place = [&](int ln) __attribute__((always_inline)) {
    if (CT == 2 || !wide) return static_cast<uint32_t>((n0 + col) * a.R * 4 + ln * 16);
    const int n = n0 + col + (ln & 15), c = n & 31;
    return static_cast<uint32_t>((n >> 5) * a.R * 128 + ((c >> 2) & 1) * 1024 +
                                 ((ln & 48) + (c >> 3) * 4 + (c & 3)) * 16);
  };

  // Rows of the next chunk, loaded ahead into registers as 16-byte pieces.
  // Row r of the walk is token t0 + r, backwards t0 + len - 1 - r.  Tokens are
  // loaded in order, backwards from the one that would be a full chunk's
  // first, so that a lane's offsets do not depend on the chunk, and turned
  // round on their way into LDS.  Rows past len and columns past the width
  // read zeros from no memory.
  using PX = std::integral_constant<int, L::px>;
  using PZ = std::integral_constant<int, L::pz>;
  using NX = std::integral_constant<int, L::nx>;
  using NZ = std::integral_constant<int, L::nz>;
  const int nch = (seg.len + C - 1) / C;
  uint4 rx[OUT ? L::nx : 1], ry[L::nx], rz[L::nz];
  auto chunk_of = [&](int c, int64_t* t0, int* len) __attribute__((always_inline)) {
    const int w = rev ? nch - 1 - c : c;
    *t0 = seg.tok0 + static_cast<int64_t>(w) * C;
    *len = min(C, seg.len - w * C);
  };
  // a thread's row among the `step` rows of a turn, as a token
  auto turned_row = [&](int row, int step) __attribute__((always_inline)) {
    return rev ? std::min(step, C) - 1 - row : row;
  };
  // calls put(register, turn in LDS) for a thread's pieces
  auto each_turn = [&](auto turns, auto put) __attribute__((always_inline)) {
    constexpr int NT = decltype(turns)::value;
    if (rev) {
#pragma unroll
      for (int u = 0; u < NT; ++u) put(u, NT - 1 - u);
    } else {
#pragma unroll
      for (int u = 0; u < NT; ++u) put(u, u);
    }
  };
  auto load_rows = [&](const void* base, int heads, int width, int col0, auto per_row, auto turns,
                       int64_t t0, int len, uint4* r) __attribute__((always_inline)) {
    constexpr int PR = decltype(per_row)::value, NT = decltype(turns)::value;
    constexpr int step = kThreads / PR;
    const uint32_t stride = static_cast<uint32_t>(heads) * width * ob;
    const int64_t row0 = rev ? t0 + len - C : t0;
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(
        static_cast<const char*>(base) +
            (row0 * heads + h / (a.H / heads)) * static_cast<int64_t>(width) * ob + col0 * ob,
        kOob);
    const int row = turned_row(tid / PR, step), c16 = (tid % PR) * 16;
    const bool in = c16 < (width - col0) * ob;
    // one offset a lane, the turns' rows in the scalar offset
    const uint32_t at = static_cast<uint32_t>(row) * stride + c16;
    const uint32_t from = row - (rev ? C - len : 0);
#pragma unroll
    for (int u = 0; u < NT; ++u)
      r[u] = __builtin_bit_cast(
          uint4, __builtin_amdgcn_raw_buffer_load_b128(
                     rs, in && from + u * step < static_cast<uint32_t>(len) ? at : kOob,
                     u * step * stride, 0));
  };
  // bit 0 of `which`: x, 1: y, 2: z
  auto load_chunk = [&](int c, auto which) __attribute__((always_inline)) {
    constexpr int w = decltype(which)::value;
    int64_t t0;
    int len;
    chunk_of(c, &t0, &len);
    if constexpr (OUT && (w & 1) != 0) load_rows(a.x, a.hx, a.R, 0, PX(), NX(), t0, len, rx);
    if constexpr ((w & 2) != 0) load_rows(a.y, a.hy, a.R, 0, PX(), NX(), t0, len, ry);
    if constexpr ((w & 4) != 0) load_rows(a.z, a.hz, a.N, n0, PZ(), NZ(), t0, len, rz);
  };
  auto put_rows = [&](char* t, auto stride, auto per_row, auto turns, const uint4* r)
      __attribute__((always_inline)) {
    constexpr int ST = decltype(stride)::value, PR = decltype(per_row)::value,
                  NT = decltype(turns)::value, step = kThreads / PR;
    const int row = tid / PR;
    char* p = t + row * ST * ob + (tid % PR) * 16;
    if (C % step == 0 || row < C)
      each_turn(turns, [&](int u, int t) __attribute__((always_inline)) {
        *reinterpret_cast<uint4*>(p + t * step * ST * ob) = r[u];
      });
  };
  // x rows with the columns of each 32-block in the permuted K order, so that
  // a fragment that matches the state's registers is one 16-byte read
  auto put_x = [&]() __attribute__((always_inline)) {
    constexpr int step = kThreads / L::px;
    const int row = tid / L::px, q = tid % L::px;
    char* p = tx + row * L::sx * ob;
    if (C % step == 0 || row < C) {
      if constexpr (ob == 2) {
        p += (q / 4 * 32 + 16 * (q & 1) + 4 * ((q >> 1) & 1)) * 2;
        each_turn(NX(), [&](int u, int t) __attribute__((always_inline)) {
          *reinterpret_cast<uint2*>(p + t * step * L::sx * 2) = make_uint2(rx[u].x, rx[u].y);
          *reinterpret_cast<uint2*>(p + t * step * L::sx * 2 + 16) = make_uint2(rx[u].z, rx[u].w);
        });
      } else {
        p += (q / 8 * 32 + 8 * (q & 3) + 4 * ((q >> 2) & 1)) * 4;
        each_turn(NX(), [&](int u, int t) __attribute__((always_inline)) {
          *reinterpret_cast<uint4*>(p + t * step * L::sx * 4) = rx[u];
        });
      }
    }
  };
  auto put_y = [&]() __attribute__((always_inline)) {
    if constexpr (L::skew == 0) {
      put_rows(ty, std::integral_constant<int, L::sy>(), PX(), NX(), ry);
    } else {
      constexpr int step = kThreads / L::px;
      // a thread's rows share their shift, or (8 apart) take two in turn
      static_assert(L::nx == 1 || step % 16 == 0 || step == 8, "");
      constexpr int odd = step == 8 ? 2 * L::skew : 0;
      const int row = tid / L::px;
      char* p = ty + (row * L::sy + L::skew * ((row >> 2) & 3)) * 2 + (tid % L::px) * 16;
      if (C % step == 0 || row < C) {
        each_turn(NX(), [&](int u, int t) __attribute__((always_inline)) {
          char* const q = p + (t * step * L::sy + (t & 1) * odd) * 2;
          *reinterpret_cast<uint2*>(q) = make_uint2(ry[u].x, ry[u].y);
          *reinterpret_cast<uint2*>(q + 8) = make_uint2(ry[u].z, ry[u].w);
        });
      }
    }
  };
  if (nch > 0) load_chunk(0, std::integral_constant<int, 7>());

  // The state in front, all loads in flight at once (rows and columns past
  // the state's, and a state that is not there, read zeros from no memory).
  floatx4 S[L::RPS][CT];
  if constexpr (OUT) {
    const float* const enter = whole ? a.init : a.enter;
    const bool image = !whole && a.image;
    const uint32_t elems = image ? image_elems : a.R * a.N;
    const int place = __builtin_amdgcn_readfirstlane(whole ? seg.seq : slot);
    const int64_t at = (static_cast<int64_t>(place) * a.H + h) * elems;
    const __amdgpu_buffer_rsrc_t rs =
        make_rsrc(enter + (enter == nullptr ? 0 : at), enter == nullptr ? 0 : elems * 4);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const int n = n_lane + 4 * ct;
      const bool there = active && enter != nullptr, in = there && n < a.N;
      if (image) {
        const uint32_t at = there ? image_place(lane) + ct * 1024 : kOob;
#pragma unroll
        for (int rt = 0; rt < L::RPS; ++rt)
          S[rt][ct] = __builtin_bit_cast(
              floatx4, __builtin_amdgcn_raw_buffer_load_b128(rs, rt * 16 < a.R ? at : kOob,
                                                             rt * image_step, 0));
      } else if (a.turned) {
        const uint32_t at = in ? (n * a.R + 4 * g) * 4 : kOob;
#pragma unroll
        for (int rt = 0; rt < L::RPS; ++rt)
          S[rt][ct] = __builtin_bit_cast(
              floatx4, __builtin_amdgcn_raw_buffer_load_b128(rs, rt * 16 < a.R ? at : kOob,
                                                             rt * 64, 0));
      } else {
        const uint32_t at = in ? (4 * g * a.N + n) * 4 : kOob;
#pragma unroll
        for (int rt = 0; rt < L::RPS; ++rt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            S[rt][ct][e] = __uint_as_float(
                __builtin_amdgcn_raw_buffer_load_b32(rs, rt * 16 < a.R ? at : kOob,
                                                     (rt * 16 + e) * a.N * 4, 0));
      }
    }
  } else {
#pragma unroll
    for (int rt = 0; rt < L::RPS; ++rt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) S[rt][ct] = floatx4{0.f, 0.f, 0.f, 0.f};
  }

  // powers of the decay, while the loads are on their way
  const double log_a =
      a.log_decay == nullptr ? 0.0 : static_cast<double>(ld_scalar(a.log_decay, h));
  for (int n = tid; n <= C + 32; n += kThreads)
    dec[n - 32] = n < 32 ? 0.f : decay_pow32(log_a, n - 32);
  // A chunk's decay of the state, full chunks' and the segment's last one's:
  // M a^n as M + M (a^n - 1) near 1, so that thousands of chunks keep it.
  auto fade_of = [&](int n, float* mul, float* add) __attribute__((always_inline)) {
    const double d = decay_pow(log_a, n);
    const bool slow = d >= 0.5;
    *mul = __uint_as_float(__builtin_amdgcn_readfirstlane(
        __float_as_uint(static_cast<float>(slow ? d - 1.0 : d))));
    *add = __uint_as_float(__builtin_amdgcn_readfirstlane(slow ? 0x3f800000u : 0u));
  };
  float mul_full, add_full, mul_tail, add_tail;
  fade_of(C, &mul_full, &add_full);
  fade_of(seg.len % C, &mul_tail, &add_tail);

  // lane bases of the operand reads and of the stores
  const char* const x_run = tx + (l16 * L::sx + 8 * g) * ob;
  const char* const x_out = x_run + set * 16 * L::sx * ob;
  const char* const y_perm = ty + (l16 * L::sy + L::skew * (l16 >> 2) + 4 * g) * ob;
  const char* const y_col = col_base<IO, L::sy, 4, L::skew>(ty, lane) + r0 * ob;
  const char* const z_col = col_base<IO, L::sz, 4 * CT, 0>(tz, lane) + col * ob;
  const float* const d_lane = dec + (l16 - 4 * g);
  const char* const p_run = tp + (set * NKC * 64 + lane) * 8 * ob;
  const int os = a.out_f32 ? 4 : ob;  // bytes per output element
  const uint32_t ostride = static_cast<uint32_t>(a.H) * a.N * os;
  const uint32_t o_lane = (rev ? 15 - l16 : l16) * ostride + (n0 + col + 4 * CT * g) * os;

  // Two stacked tiles of x y^T, transposed (column i, rows j): row tiles
  // 2 jp and 2 jp + 1 of y against tile `it` of x, one operand fragment.
  auto pair = [&](int it, int jp) __attribute__((always_inline)) {
    floatx4 p0 = {0.f, 0.f, 0.f, 0.f}, p1 = p0;
    const char* const xp = x_run + it * 16 * L::sx * ob;
    const char* const yp = y_perm + jp * 32 * L::sy * ob;
#pragma unroll
    for (int kb = 0; kb < NKB; ++kb) {
      const opvec<IO> xf = lds_run8<IO>(xp + kb * 32 * ob);
      p0 = mma32(lds_perm8<IO>(yp + kb * 32 * ob), xf, p0);
      p1 = mma32(lds_perm8<IO>(yp + (16 * L::sy + kb * 32) * ob), xf, p1);
    }
    // decays a^(i - j), zero above the diagonal (the table's lower end)
    const float* const d = d_lane + (it * 16 - jp * 32);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      p0[e] *= d[-e];
      p1[e] *= d[-16 - e];
    }
    // In two parts: the first alone would add an output's half step again,
    // which short sequences, all x y^T, show as 1.6 times the error of one
    // rounding; the second costs 1 % (65k tokens) to 4 % (B8 T2048 backward).
    const opvec<IO> r = pack2<IO>(p0, p1);
    char* const at = tp + ((it * NKC + jp) * 64 + lane) * 8 * ob;
    *reinterpret_cast<opvec<IO>*>(at) = r;
    if constexpr (ob == 2)
      *reinterpret_cast<opvec<IO>*>(at + C * C * ob) = pack2_rest(p0, p1, r);
  };

  // M <- a^n M + sum_j y_j (w_j z_j)^T, the weighted rows in their first
  // FIRST operand parts (pass 0), or M += the parts left (pass 1)
  constexpr int FIRST = OUT ? std::min(2, Parts<IO>::most) : Parts<IO>::most;
  auto update = [&](int n, auto which) __attribute__((always_inline)) {
    constexpr int pass = decltype(which)::value;
    constexpr int NPART = pass == 0 ? FIRST : Parts<IO>::most - FIRST;
    const float mul = n == C ? mul_full : mul_tail, add = n == C ? add_full : add_tail;
    auto fade = [&](int rt) __attribute__((always_inline)) {
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          S[rt][ct][e] = __builtin_fmaf(S[rt][ct][e], mul, add * S[rt][ct][e]);
    };
    constexpr int GR = OUT ? std::min(2, L::RPS) : 1;  // state row tiles a step
    constexpr int PER = L::RPS / GR;                   // steps a 32-row block
    opvec<IO> yf[2][GR], zf[CT];
    auto read_z = [&](int kb) __attribute__((always_inline)) {
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
        zf[ct] = lds_col8<IO, L::sz>(z_col + (kb * 32 * L::sz + ct * 4) * ob);
    };
    auto read_y = [&](int step) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < GR; ++u)
        yf[step & 1][u] = lds_col8<IO, L::sy>(
            y_col + (step / PER * 32 * L::sy + ((step % PER) * GR + u) * 16) * ob);
    };
    read_z(0);
    read_y(0);
    if constexpr (pass == 0) {
#pragma unroll
      for (int u = 0; u < GR; ++u) fade(u);
    }
    Parts<IO> wz[CT];
#pragma unroll
    for (int step = 0; step < NKC * PER; ++step) {
      const int kb = step / PER, rt = (step % PER) * GR;
      if (step + 1 < NKC * PER) read_y(step + 1);
      if (rt == 0) {
        float w[8];
        const floatx4 lo = *reinterpret_cast<const floatx4*>(wgt + kb * 32 + 4 * g);
        const floatx4 hi = *reinterpret_cast<const floatx4*>(wgt + kb * 32 + 16 + 4 * g);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = lo[e], w[4 + e] = hi[e];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) wz[ct].template set<NPART, pass * FIRST>(zf[ct], w);
        if (kb + 1 < NKC) read_z(kb + 1);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < NPART; ++u)
#pragma unroll
        for (int v = 0; v < GR; ++v)
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) {
            if constexpr (ob == 2)
              S[rt + v][ct] = mma32(yf[step & 1][v], wz[ct].p[u], S[rt + v][ct]);
            else  // (a step adds four rows only: summed apart, the chunk rounds
                  // the state once, a third of the error after thousands of
                  // tokens for 0 to 2 % of the time)
              S[rt + v][ct] +=
                  mma32(yf[step & 1][v], wz[ct].p[u], floatx4{0.f, 0.f, 0.f, 0.f});
          }
      // the next rows' decay, between the products
      if (pass == 0 && kb == 0 && step + 1 < PER) {
#pragma unroll
        for (int u = 0; u < GR; ++u) fade(rt + GR + u);
      }
    }
  };

  int wlen = -1;  // chunk length that wgt is for
  for (int c = 0; c < nch; ++c) {
    int64_t t0;
    int len;
    chunk_of(c, &t0, &len);
    floatx4 acc[OUT ? L::IPS : 1][CT];
    // the chunk's output rows, from acc
    auto store_out = [&]() __attribute__((always_inline)) {
      // uniform base of the chunk's rows (backwards: of a full chunk's)
      using global = __attribute__((address_space(1))) char;
      global* const orow = (global*)(a.out) +
                         ((rev ? t0 + len - C : t0) * a.H + h) * static_cast<int64_t>(a.N) * os;
      global* p = orow + static_cast<int64_t>((rev ? NI - 1 - set : set) * 16) * ostride;
      const int64_t next = static_cast<int64_t>(rev ? -16 * L::SETS : 16 * L::SETS) * ostride;
#pragma unroll
      for (int u = 0; u < L::IPS; ++u, p += next) {
        const int it = set + u * L::SETS;
        if (it * 16 + l16 < len && n0 + col + 4 * CT * g < a.N) {
          if (ob == 4 || a.out_f32) {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
              *(__attribute__((address_space(1))) floatx4*)(p + o_lane + ct * 16) = acc[u][ct];
          } else if constexpr (CT == 2) {
            *(__attribute__((address_space(1))) opvec<IO>*)(p + o_lane) =
                pack2<IO>(acc[u][0], acc[u][1]);
          } else {
            *(__attribute__((address_space(1))) typename acc4<IO>::type*)(p + o_lane) =
                from_f4<IO>(acc[u][0]);
          }
        }
      }
    };

    __syncthreads();  // the previous chunk's tiles have been read
    if constexpr (OUT) put_x();
    put_y();
    put_rows(tz, std::integral_constant<int, L::sz>(), PZ(), NZ(), rz);
    if (len != wlen) {
      wlen = len;
      if (tid < C) wgt[tid] = tid < len ? dec[len - off - tid] : 0.f;
    }
    __syncthreads();
    // the next chunk's rows, in two goes: a burst would stall the waves behind
    // the memory pipe
    if (c + 1 < nch) load_chunk(c + 1, std::integral_constant<int, OUT ? 1 : 6>());

    if constexpr (OUT) {
      if constexpr (NI == 2) {
        if (wave < 2) pair(wave, 0);
      } else if constexpr (L::waves == 4) {
        pair(wave < 2 ? 3 : 4 - wave, wave == 1 ? 1 : 0);
        if (wave >= 2) pair(wave == 2 ? 0 : 2, wave - 2);
      } else {
        if (wave < 6) pair(wave < 2 ? wave : wave < 4 ? 2 : 3, wave < 2 ? 0 : wave & 1);
      }
      if (c + 1 < nch) load_chunk(c + 1, std::integral_constant<int, 6>());
    }

    if (active) {
      if constexpr (OUT) {
        // M^T x^T, the copy of the state in two operand parts (2^-17 left):
        // with one, its rounding takes the outputs' error from one rounding of
        // their own to 1.4, in every call that enters with a state or runs on
        // past a chunk.  The second part costs 3 % (65k tokens: 409 us, 420)
        // to 10 % (B8 T2048 H8 backward: 130 us, 142).
        opvec<IO> xf[2][L::IPS];
        auto read_x = [&](int kb) __attribute__((always_inline)) {
#pragma unroll
          for (int it = 0; it < L::IPS; ++it)
            xf[kb & 1][it] = lds_run8<IO>(x_out + (it * L::SETS * 16 * L::sx + kb * 32) * ob);
        };
        read_x(0);
#pragma unroll
        for (int it = 0; it < L::IPS; ++it)
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) acc[it][ct] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) {
          if (kb + 1 < NKB) read_x(kb + 1);
          __builtin_amdgcn_sched_barrier(0);
          opvec<IO> m[CT];
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) m[ct] = pack2<IO>(S[2 * kb][ct], S[2 * kb + 1][ct]);
#pragma unroll
          for (int it = 0; it < L::IPS; ++it)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
              acc[it][ct] = mma32(m[ct], xf[kb & 1][it], acc[it][ct]);
          if constexpr (ob == 2) {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
              m[ct] = pack2_rest(S[2 * kb][ct], S[2 * kb + 1][ct], m[ct]);
#pragma unroll
            for (int it = 0; it < L::IPS; ++it)
#pragma unroll
              for (int ct = 0; ct < CT; ++ct)
                acc[it][ct] = mma32(m[ct], xf[kb & 1][it], acc[it][ct]);
          }
        }
#pragma unroll
        for (int it = 0; it < L::IPS; ++it) {
          const float s = dec[(set + it * L::SETS) * 16 + l16 + off];
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) acc[it][ct] *= s;
        }
      }
    }

    if constexpr (OUT) {
      opvec<IO> zf[NKC][CT];
#pragma unroll
      for (int kb = 0; kb < NKC; ++kb)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
          zf[kb][ct] = lds_col8<IO, L::sz>(z_col + (kb * 32 * L::sz + ct * 4) * ob);
      __syncthreads();  // x y^T is in LDS
      if (active) {
#pragma unroll
        for (int u = 0; u < L::IPS; ++u) {
          const int it = set + u * L::SETS;
#pragma unroll
          for (int kb = 0; kb < NKC; ++kb) {
            if (kb > it / 2) continue;
            const opvec<IO> pf = lds_run8<IO>(p_run + (u * L::SETS * NKC + kb) * 512 * ob);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) acc[u][ct] = mma32(zf[kb][ct], pf, acc[u][ct]);
            if constexpr (ob == 2) {
              const opvec<IO> pr =
                  lds_run8<IO>(p_run + (u * L::SETS * NKC + kb) * 512 * ob + C * C * ob);
#pragma unroll
              for (int ct = 0; ct < CT; ++ct) acc[u][ct] = mma32(zf[kb][ct], pr, acc[u][ct]);
            }
          }
        }
        store_out();
      }
    }
    if (active) {
      // The state behind the chunk, where another chunk or the caller wants
      // it.  One that only multiplies bf16 rows keeps 2^-17 of each term with
      // two parts; what a caller gets takes a second pass with the third
      // (another workgroup's: three at once).  A fourth changed nothing but
      // bits below fp32 and cost 4 to 6 % (B32 T1024 H16, uncut: forward 172
      // us, 162; backward 425, 409).
      const bool handed = OUT && whole && a.behind != nullptr;
      if (!OUT || handed || c + 1 < nch) update(len, std::integral_constant<int, 0>());
      if constexpr (FIRST < Parts<IO>::most)
        if (handed) update(len, std::integral_constant<int, 1>());
    }
  }

  // (the lane's place is worked out again: kept, it costs the loop registers)
  int again = lane;
  asm volatile("" : "+v"(again));
  float* bh = a.behind;
  if (bh != nullptr && active && (OUT ? whole && set == 0 : true)) {
    const int64_t at = OUT ? static_cast<int64_t>(seg.seq) * a.H + h
                           : static_cast<int64_t>(slot) * a.H + h;
    bh += at * (!OUT && a.image ? image_elems : a.R * a.N);
#pragma unroll
    for (int rt = 0; rt < L::RPS; ++rt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        if (!OUT && a.image) {
          if (r0 + rt * 16 < a.R)
            *reinterpret_cast<floatx4*>(reinterpret_cast<char*>(bh) + image_place(again) +
                                        (r0 / 16 + rt) * image_step + ct * 1024) = S[rt][ct];
          continue;
        }
        const int l = again & 15, r = r0 + rt * 16 + 4 * (again >> 4),
                  n = n0 + col + (CT == 2 ? 8 * (l >> 2) + (l & 3) + 4 * ct : l);
        if (r >= a.R || n >= a.N) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) bh[(r + e) * a.N + n] = S[rt][ct][e];
      }
  }
}

// BOTH: walks in either direction; else all forward (the reverse copy's
// scalar registers cost a forward 8 %).
template <typename IO, int NKB, int NP, bool OUT, bool BOTH>
__global__ __launch_bounds__((WalkTiles<IO, NKB, NP, OUT>::threads), OUT ? 2 : 3)
void linattn_walk_kernel(Walks walks) {
  __shared__ __align__(16) char lds[WalkTiles<IO, NKB, NP, OUT>::bytes];
  // Consecutive workgroups go round the 8 XCDs.  Items (segment, head) follow
  // each other that way, so that unused slots and short segments fall on all
  // of them alike; the slabs and walks of one item, which read the same rows,
  // are 8 workgroups apart and so share an L2.
  const int parts = (walks.w[0].N + NP - 1) / NP * walks.n;
  const int full = gridDim.x / (8 * parts) * 8;  // items in whole groups of 8
  const int id = blockIdx.x;
  int part = (id >> 3) % parts, item = (id / (8 * parts)) * 8 + (id & 7);
  if (id >= full * parts) {
    part = (id - full * parts) % parts;
    item = full + (id - full * parts) / parts;
  }
  const int slab = part / walks.n;
  // (held in scalar registers: read again inside the loop, the arguments
  // would make every wait for LDS wait for scalar memory too)
  Walk a = walks.w[part - slab * walks.n];
  asm volatile("" : "+s"(a.x), "+s"(a.y), "+s"(a.z), "+s"(a.out), "+s"(a.hx), "+s"(a.hy),
               "+s"(a.hz), "+s"(a.H), "+s"(a.R), "+s"(a.N), "+s"(a.out_f32));
  const int h = item % a.H, slot = item / a.H;
  if constexpr (BOTH) {
    if (a.rev) return walk_segment<IO, NKB, NP, OUT, true>(a, slab, h, slot, lds);
  }
  walk_segment<IO, NKB, NP, OUT, false>(a, slab, h, slot, lds);
}

// -------------------------------------------------------------- combine ---
// The state in front of every segment of the sequences that are cut, in
// place: buf[slot, h] holds each segment's own contribution (the last one's
// in walk order only with `fin`, which takes the state behind it) and becomes
// the state entering it,
// E' = a^len E + own.  A thread carries four state elements through the
// sequence's segments; sixteen loads run ahead of the chain.  Memory bounds
// it (16k tokens in 4 sequences, dk 128 dv 256, both directions: 140 MB in 32
// us, 4.4 TB/s), in short calls the launch (T4096 H16: 33 MB in 8 us).
// image: buf holds the states in register order (Walk::image, with CT column
// tiles a block); init is a [dk, dv] matrix.
struct Combine {  // one of up to two directions of a launch
  int rev;
  const float* init;
  float* buf;
  float* fin;  // [sequences, H, dk, dv] or nullptr
};
struct Combines {
  Combine c[2];
  int n;
};

__global__ __launch_bounds__(256) void linattn_combine_kernel(Cut cut, int H, int R, int N,
                                                              int image, const float* log_decay,
                                                              Combines two) {
  const Combine& dir = two.c[blockIdx.x % two.n];
  const int id = blockIdx.x / two.n;
  const bool rev = dir.rev != 0;
  const float* init = dir.init;
  float* buf = dir.buf;
  float* fin = dir.fin;
  const int CT = N > 64 ? 2 : 1;
  const int elems = image ? (N + 16 * CT - 1) / (16 * CT) * 16 * CT * R : R * N;
  const int nblk = (elems / 4 + 255) / 256;
  const int blk = id % nblk;
  const int h = (id / nblk) % H;
  int seq = id / (nblk * H);  // packed: the how manyeth of the cut sequences
  int first, n, len;
  if (cut.cu == nullptr) {
    n = cut.per_seq;
    first = seq * n;
    len = cut.T;
  } else {
    const int lane = threadIdx.x & 63;
    const uint32_t slots = static_cast<uint32_t>(cut.slots);
    uint32_t before = 0, f = 0, cnt = 0;
    int rank = seq, l = -1, base = 0;  // rank: cut sequences still to pass
    for (; base < cut.nseq; base += 64) {
      f = before + lane_slots(cut, base, lane, &cnt);
      const uint64_t is_cut = __ballot(cnt > 0);
      const int upto = __popcll(is_cut & ((uint64_t(1) << lane) - 1));
      const uint64_t hit = __ballot(cnt > 0 && upto == rank);
      if (hit != 0) {
        l = __ffsll(static_cast<unsigned long long>(hit)) - 1;
        break;
      }
      rank -= __popcll(is_cut);
      before = min(__shfl(f + cnt, 63, 64), slots);
    }
    if (l < 0) return;  // fewer are cut than there is room for
    seq = __builtin_amdgcn_readfirstlane(base + l);
    f = min(__shfl(f, l, 64), slots);
    // (bounds that overlap need more slots than there are: none beyond them)
    first = static_cast<int>(f);
    n = static_cast<int>(min(__shfl(cnt, l, 64), slots - f));
    int st, en;
    seq_range(cut, seq, &st, &en);
    len = en - st;
  }
  const int e4 = blk * 256 + threadIdx.x;
  if (e4 >= elems / 4) return;
  auto at = [&](int w) {  // w: index in walk order
    const int j = rev ? n - 1 - w : w;
    return reinterpret_cast<floatx4*>(
        buf + (static_cast<int64_t>(first + j) * H + h) * elems + 4 * e4);
  };
  constexpr int kAhead = 16;
  floatx4 own[kAhead];
  auto load = [&](int w0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (w0 + u < n - (fin == nullptr)) own[u] = *at(w0 + u);
  };
  load(0);

  // where the thread's four elements are in a [dk, dv] matrix: image: four
  // rows of one column (past the last one: nowhere)
  int place = 4 * e4, apart = 1;
  if (image) {
    const int lane = e4 & 63, tile = e4 >> 6, l16 = lane & 15;
    const int ct = tile % CT, rt = tile / CT % (R / 16), cb = tile / (CT * (R / 16));
    const int col = cb * 16 * CT + (CT == 2 ? 8 * (l16 >> 2) + (l16 & 3) + 4 * ct : l16);
    place = col < N ? (rt * 16 + 4 * (lane >> 4)) * N + col : -1;
    apart = N;
  }
  const int64_t state = (static_cast<int64_t>(seq) * H + h) * R * N;
  floatx4 E = {0.f, 0.f, 0.f, 0.f};
  if (init != nullptr && place >= 0) {
#pragma unroll
    for (int e = 0; e < 4; ++e) E[e] = init[state + place + e * apart];
  }
  const double log_a = log_decay == nullptr ? 0.0 : static_cast<double>(ld_scalar(log_decay, h));
  const double ds = decay_pow(log_a, cut.span);
  const double dt = decay_pow(log_a, len - (n - 1) * cut.span);  // the short last segment's
  for (int w0 = 0; w0 < n; w0 += kAhead) {
    if (w0 > 0) load(w0);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (w0 + u >= n) break;
      *at(w0 + u) = E;
      const double d = w0 + u == (rev ? 0 : n - 1) ? dt : ds;
      if (w0 + u < n - (fin == nullptr)) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          E[e] = static_cast<float>(d * static_cast<double>(E[e]) + static_cast<double>(own[u][e]));
      }
    }
  }
  if (fin != nullptr && place >= 0) {
#pragma unroll
    for (int e = 0; e < 4; ++e) fin[state + place + e * apart] = E[e];
  }
}

// ---------------------------------------------------------- shared heads ---
// Gradients of q and k heads: the sum over the v heads that read it, in head
// order, from the fp32 rows of each (part and part + apart: [tokens, H, d] ->
// out0 and out1: [tokens, Hq, d]).  Tokens behind the last sequence are left
// alone.  A stream: 16k tokens of 16 heads over 8, d 128, 335 MB in 64 us
// (5.2 TB/s).  Atomics into one fp32 row would save the pass but add in an
// order that changes.
template <typename IO>
__global__ __launch_bounds__(256) void linattn_share_kernel(const float* part, int64_t apart,
                                                            void* out0, void* out1,
                                                            int64_t tokens, int Hq, int grp, int d,
                                                            const int32_t* cu, int nseq) {
  void* const out = blockIdx.y == 0 ? out0 : out1;
  part += blockIdx.y * apart;
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
// once in 16-byte pieces, so that memory bounds it (3 flops per 8 bytes); a
// workgroup takes one (sequence, head) and 64 columns, a thread DK / 16 rows
// of 4 columns.  Four loads of a thread are in flight (N256 H32 of 128 x 128,
// 1.08 GB: 189 us, 5.7 TB/s; all eight 193, with the stores between them
// 197, one 185 but 47.3 against 46.7 at N64), and the stores wait for the
// workgroup's loads, since memory turns round less often.
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
  const bool active = slab * 64 + cg * 4 < dv;
  const int col = active ? slab * 64 + cg * 4 : 0;  // (idle lanes read what others do)
  float* M = state + static_cast<int64_t>(nh) * DK * dv + col;
  const int64_t qo = (static_cast<int64_t>(n) * (H / grp) + h / grp) * DK + rg;
  const int64_t vo = static_cast<int64_t>(nh) * dv + col;
  float kr[RPT], qr[RPT];
#pragma unroll
  for (int j = 0; j < RPT; ++j) {
    kr[j] = io<IO>::load(k, qo + 16 * j);
    qr[j] = io<IO>::load(q, qo + 16 * j);
  }
  floatx4 vv;
#pragma unroll
  for (int c = 0; c < 4; ++c) vv[c] = io<IO>::load(v, vo + c);
  floatx4 m[RPT];
#pragma unroll
  for (int j = 0; j < RPT; ++j) {
    m[j] = __builtin_nontemporal_load(reinterpret_cast<const floatx4*>(M + (rg + 16 * j) * dv));
    if (j % 4 == 3 && j + 1 < RPT) {
      __builtin_amdgcn_s_waitcnt(0x0f70);  // loads: none left
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  const float a =
      log_decay == nullptr ? 1.0f : static_cast<float>(exp(static_cast<double>(log_decay[h])));
  floatx4 w = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < RPT; ++j) {
#pragma unroll
    for (int c = 0; c < 4; ++c) m[j][c] = __builtin_fmaf(a, m[j][c], kr[j] * vv[c]);
    w += m[j] * qr[j];
  }
  // over the 16 row groups: 4 in the wave, then the 4 waves through LDS
#pragma unroll
  for (int c = 0; c < 4; ++c) w[c] = wave_sum_xor(w[c], 48);
  __shared__ floatx4 sw[4][16];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if (lane < 16) sw[wave][lane] = w;
  __syncthreads();
  if (!active) return;
#pragma unroll
  for (int j = 0; j < RPT; ++j)
    __builtin_nontemporal_store(m[j], reinterpret_cast<floatx4*>(M + (rg + 16 * j) * dv));
  if (threadIdx.x < 16) {
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
  int64_t slots;   // segment slots; packed: an upper bound, of the cut sequences
  int64_t cuts;    // sequences that are cut (packed: an upper bound)
  int64_t walks;   // slots of an output launch: the cut sequences' and the whole ones
  bool split;
};

// Tiles of a walk, as launch_walk_io and launch_walk_n pick them.
int tiles_of(int R, int N) {
  return (R > 128 ? 8 : R > 64 ? 4 : R > 32 ? 2 : 1) * 1024 +
         (N <= 32 ? 0 : N <= 64 ? 1 : 1 + (N + 127) / 128);
}

// dv's walk joins dq's and dk's where its tiles are theirs
bool walks_join(const LinAttn& p) { return tiles_of(p.dv, p.dk) == tiles_of(p.dk, p.dv); }

Plan plan_walk(const LinAttn& p, bool bwd) {
  const int C = p.io == GDN_BF16 ? 64 : 32;
  Plan r;
  const int64_t nch = (static_cast<int64_t>(p.T) + C - 1) / C;  // of one dense sequence, or all
  const int64_t slabs = (p.dv + 127) / 128, heads = static_cast<int64_t>(p.nseq) * p.H;
  const int64_t chains = heads * slabs;
  const int64_t units = p.varlen ? nch * (chains / p.nseq) : nch * chains;  // chunks to walk
  int64_t L = nch;  // chunks per segment
  if (p.seg_req > 0) {
    L = std::min<int64_t>(nch, p.seg_req);
  } else if (p.seg_req == 0 && nch > 6) {
    // (six chunks or fewer are walked faster than two more launches take)
    // Workgroups of an output launch that is not cut.
    const int64_t whole =
        !bwd ? chains : walks_join(p) ? 3 * chains : std::min(2 * heads, chains);
    if (p.varlen) {
      // The longest of n sequences is likely to have about ln n + 0.58 times
      // the mean's tokens (bounds drawn at random).  A longer one may be there
      // all the same, a prompt among single tokens, so a batch of any size has
      // a length that it is cut at; what is shorter costs nothing but the two
      // launches.
      const double apart = std::log(static_cast<double>(p.nseq)) + 0.58;
      const bool few = nch * apart <= 6.0 * p.nseq;  // six chunks or fewer, most likely
      if (few && nch <= 12) {
        // (7 sequences of 64 tokens at 16 heads: 16 us, cut 27)
        L = nch;
      } else if (whole >= 256 * apart) {
        // Whole sequences fill the machine, and most likely the longest ends
        // before the others do; one that would take as long as all work
        // together (a CU of its own walks a chunk in half the time) is cut.
        // 65k tokens of 16 heads in 256: not cut 389 us, L 64 400, 8 529; in
        // 1024: 617, 667, 951; backward in 32: 880, L 192 875, 16 976.
        const int64_t share = int64_t(256) * p.nseq;
        L = std::max<int64_t>(6, (nch * whole + share - 1) / share);
      } else if (chains > 256 || few) {
        // An even share of two workgroups a CU (65k tokens of 16 heads in 64:
        // L 32 446 us, 12 476, not cut 826; 16k of 2 heads in 256: 6 55, 4 60).
        L = std::max<int64_t>(6, (units + 511) / 512);
      } else {
        // Segments for two workgroups a CU (512): each chain ends in a segment
        // that is half full on average (65k tokens of 16 heads in 7 sequences:
        // 36 chunks 445 us, 24: 433, 48: 468, 12: 453, 96: 783; backward of
        // 16k in 16: 11 chunks 290, 24: 301, 4: 320).
        const int64_t room = 512 - chains / 2;
        L = (units + room - 1) / room;
      }
    } else {
      // Where workgroups that are not cut take most CUs, two more passes over
      // the tokens cost more than the idle ones (dk 128 dv 128 backward, us
      // not cut / cut, 198 of them: T1024 73 / 98, T2048 141 / 158, T8192 550
      // / 562; 192: T1024 73 / 81, T2048 142 / 140, T4096 280 / 245).
      if (whole < (nch <= 32 ? 192 : 200)) {
        // One workgroup a CU while walks are short, since every further segment
        // costs four passes over its state (T4096 H16: 4 chunks 43 us, 2: 51);
        // two where they are long.
        const int64_t target = units < 48 * 256 ? 256 : 512;
        const int64_t per_seq = std::max<int64_t>(1, target / chains);
        L = (nch + per_seq - 1) / per_seq;
      }
    }
    // The states are chained a segment after another: at least
    // sqrt(chunks / 8) chunks each (T16384 H2: 2 chunks 70 us, 6: 47;
    // T65536 H1: 4: 126, 12: 85).
    while (8 * L * L < (p.varlen ? nch / p.nseq : nch)) ++L;
    L = std::min(L, nch);
  }
  L = std::max<int64_t>(L, 1);
  r.split = L < nch;
  r.span = static_cast<int>(std::min<int64_t>(r.split ? L * C : int64_t(1) << 30, 1 << 30));
  r.per_seq = r.split ? static_cast<int>((nch + L - 1) / L) : 1;
  if (p.varlen) {
    // a sequence that is cut has more than `span` tokens, and one segment
    // more than whole spans
    r.cuts = r.split ? std::min<int64_t>(p.nseq, p.T / (static_cast<int64_t>(r.span) + 1)) : 0;
    r.slots = r.split ? p.T / r.span + r.cuts : 0;
    r.walks = r.slots + p.nseq;
  } else {
    r.cuts = p.nseq;
    r.slots = r.walks = static_cast<int64_t>(p.nseq) * r.per_seq;
  }
  return r;
}

Cut make_cut(const LinAttn& p, const Plan& pl) {
  return Cut{p.varlen ? p.cu_seqlens : nullptr, p.nseq, p.T, pl.span, pl.per_seq, pl.slots};
}

template <typename IO, int NKB, int NP, bool OUT, bool BOTH>
void launch_walk_t(const Walks& w, int64_t slots, hipStream_t s) {
  const int64_t nslab = (w.w[0].N + NP - 1) / NP;
  hipLaunchKernelGGL((linattn_walk_kernel<IO, NKB, NP, OUT, BOTH>),
                     dim3(static_cast<unsigned>(slots * w.w[0].H * nslab * w.n)),
                     dim3(WalkTiles<IO, NKB, NP, OUT>::threads), 0, s, w);
}

template <typename IO, int NKB, bool OUT, bool BOTH>
void launch_walk_n(const Walks& w, int64_t slots, hipStream_t s) {
  const int N = w.w[0].N;
  // A workgroup's chunk takes less time the fewer columns it has (dk 128: 4.7
  // us for 128, 3.3 for 64, 3.1 for 32), so slabs are as narrow as leave every
  // workgroup a CU of its own (T256 H16: 128 columns 25.3 us, 64: 18.2, 32:
  // 17.0).  Past that the x and y rows that all slabs read, and their x y^T,
  // cost more (B8 T2048 H8 backward, not cut, 192 workgroups of 128 columns:
  // 142 us, 64: 139, 32: 216; 96 of them: 141, 108, 121).
  auto fits = [&](int np) {
    return slots * w.w[0].H * ((N + np - 1) / np) * w.n <= 256;
  };
  if (N <= 32 || fits(32)) return launch_walk_t<IO, NKB, 32, OUT, BOTH>(w, slots, s);
  if (N <= 64 || fits(64)) return launch_walk_t<IO, NKB, 64, OUT, BOTH>(w, slots, s);
  launch_walk_t<IO, NKB, 128, OUT, BOTH>(w, slots, s);
}

template <typename IO, bool OUT, bool BOTH>
void launch_walk_io(const Walks& w, int64_t slots, hipStream_t s) {
  const int R = w.w[0].R;
  if constexpr (OUT && BOTH)  // (a forward alone contracts over dk <= 128)
    if (R > 128) return launch_walk_n<IO, 8, OUT, BOTH>(w, slots, s);
  if (R > 64) return launch_walk_n<IO, 4, OUT, BOTH>(w, slots, s);
  if (R > 32) return launch_walk_n<IO, 2, OUT, BOTH>(w, slots, s);
  launch_walk_n<IO, 1, OUT, BOTH>(w, slots, s);
}

template <typename IO>
void launch_walk_dir(const Walks& w, int64_t slots, bool out, hipStream_t s) {
  const bool both = w.n > 1 || w.w[0].rev;
  if (out)
    both ? launch_walk_io<IO, true, true>(w, slots, s)
         : launch_walk_io<IO, true, false>(w, slots, s);
  else
    both ? launch_walk_io<IO, false, true>(w, slots, s)
         : launch_walk_io<IO, false, false>(w, slots, s);
}

// Walks of the same tiles together.
hipError_t launch_walks(const LinAttn& p, const Walks& w, int64_t slots, bool out, int stage,
                        hipStream_t s) {
  StageScope scope(stage, s);
  if (p.io == GDN_BF16)
    launch_walk_dir<bf16_t>(w, slots, out, s);
  else
    launch_walk_dir<f32_t>(w, slots, out, s);
  return hipGetLastError();
}

// Elements of a state in register order: whole column blocks.
int image_elems(const LinAttn& p) { return p.dk * (p.dv > 64 ? (p.dv + 31) / 32 * 32 : p.dv); }

// One direction of the states in front of every segment.
struct Front {
  bool rev;
  const void *y, *z;
  int hy, hz;
  const float* init;
  float *buf, *fin;
};

// States in front of every segment into the buffers, and behind the last ones
// where wanted: own contributions, chained; one or two directions.
hipError_t enter_states(const LinAttn& p, const Plan& pl, const Front* f, int n, bool image,
                        const float* la, hipStream_t s) {
  Walks w{};
  Combines c{};
  w.n = c.n = n;
  for (int i = 0; i < n; ++i) {
    Walk& a = w.w[i];
    a.cut = make_cut(p, pl);
    a.rev = f[i].rev ? 1 : 0;
    a.y = f[i].y;
    a.z = f[i].z;
    a.hx = a.H = p.H;
    a.hy = f[i].hy;
    a.hz = f[i].hz;
    a.R = p.dk;
    a.N = p.dv;
    a.log_decay = la;
    a.behind = f[i].buf;
    a.ends = f[i].fin != nullptr ? 1 : 0;
    a.image = image ? 1 : 0;
    c.c[i] = Combine{a.rev, f[i].init, f[i].buf, f[i].fin};
  }
  const hipError_t e = launch_walks(p, w, pl.slots, false, GDN_STAGE_FWD_TRANS, s);
  if (e != hipSuccess) return e;
  StageScope scope(GDN_STAGE_FWD_COMBINE, s);
  const int elems = image ? image_elems(p) : p.dk * p.dv;
  const int64_t grid = pl.cuts * p.H * ((elems / 4 + 255) / 256) * n;
  hipLaunchKernelGGL(linattn_combine_kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0, s,
                     w.w[0].cut, p.H, p.dk, p.dv, image ? 1 : 0, la, c);
  return hipGetLastError();
}

size_t state_bytes(const LinAttn& p, const Plan& pl) {
  return pl.split ? al256(static_cast<size_t>(pl.slots) * p.H * image_elems(p) * 4) : 0;
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

// A launch takes fewer than 2^32 threads (HIP's limit).
bool linattn_fits(const LinAttn& p, bool bwd) {
  const Plan pl = plan_walk(p, bwd);
  const int64_t most = (int64_t(1) << 32) - 1;
  // n walks over `slots` slots with N columns and R state rows (narrower slabs
  // are taken where there are few workgroups only)
  auto walks = [&](int64_t slots, int R, int N, int n) {
    return slots * p.H * ((N + 127) / 128) * n * (R > 128 && N > 64 ? 512 : 256);
  };
  const int64_t blocks = (static_cast<int64_t>(image_elems(p)) / 4 + 255) / 256;
  const int both = bwd ? 2 : 1;
  if (pl.split && std::max(walks(pl.slots, p.dk, p.dv, both),
                           pl.cuts * p.H * blocks * both * 256) > most)
    return false;
  if (!bwd) return walks(pl.walks, p.dk, p.dv, 1) <= most;
  return std::max(walks(pl.walks, p.dv, p.dk, walks_join(p) ? 3 : 2),
                  walks(pl.walks, p.dk, p.dv, 1)) <= most;
}

bool linattn_step_fits(const LinAttn& p) {
  return static_cast<int64_t>(p.B) * p.H * ((p.dv + 63) / 64) * 256 <= (int64_t(1) << 32) - 1;
}

size_t linattn_fwd_workspace_bytes(const LinAttn& p) { return state_bytes(p, plan_walk(p, false)); }

hipError_t launch_linattn_fwd(const LinAttn& p, const void* q, const void* k, const void* v,
                              const float* la, const float* s0, void* o, float* s_final,
                              void* ws, hipStream_t s) {
  const Plan pl = plan_walk(p, false);
  Walks one{};
  one.n = 1;
  Walk& w = one.w[0];
  w.cut = make_cut(p, pl);
  w.init = s0;
  if (pl.split) {
    float* buf = static_cast<float*>(ws);
    const Front f{false, k, v, p.hq, p.H, s0, buf, s_final};
    const hipError_t e = enter_states(p, pl, &f, 1, true, la, s);
    if (e != hipSuccess) return e;
    w.enter = buf;
    w.image = 1;
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
  return launch_walks(p, one, pl.walks, true, GDN_STAGE_FWD_SCAN, s);
}

size_t linattn_bwd_workspace_bytes(const LinAttn& p) {
  return 2 * state_bytes(p, plan_walk(p, true)) + 2 * part_bytes(p);
}

hipError_t launch_linattn_bwd(const LinAttn& p, const void* q, const void* k, const void* v,
                              const float* la, const float* s0, const void* d_o,
                              const float* ds_final, void* dq, void* dk, void* dv, float* ds0,
                              void* ws, hipStream_t s) {
  const Plan pl = plan_walk(p, true);
  const float *front = nullptr, *back = nullptr;  // of every segment
  char* at = static_cast<char*>(ws);
  hipError_t e;
  if (pl.split) {
    float* bf = reinterpret_cast<float*>(at);
    at += state_bytes(p, pl);
    float* bb = reinterpret_cast<float*>(at);
    at += state_bytes(p, pl);
    const Front f[2] = {{false, k, v, p.hq, p.H, s0, bf, nullptr},
                        {true, q, d_o, p.hq, p.H, ds_final, bb, ds0}};
    e = enter_states(p, pl, f, 2, false, la, s);
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
  Walks all{};
  Walk& dq_ = all.w[0] = w;
  dq_.x = d_o;
  dq_.y = v;
  dq_.z = k;
  dq_.init = s0;
  dq_.enter = front;
  dq_.out = shared ? static_cast<void*>(part_q) : dq;
  w.rev = 1;
  w.init = ds_final;
  w.enter = back;
  Walk& dk_ = all.w[1] = w;
  dk_.x = v;
  dk_.y = d_o;
  dk_.z = q;
  dk_.out = shared ? static_cast<void*>(part_k) : dk;
  Walk& dv_ = all.w[2] = w;
  dv_.turned = 0;
  dv_.out_f32 = 0;
  dv_.R = p.dk;
  dv_.N = p.dv;
  dv_.hx = dv_.hy = p.hq;
  dv_.hz = p.H;
  dv_.x = k;
  dv_.y = q;
  dv_.z = d_o;
  dv_.out = dv;
  dv_.behind = ds0;
  all.n = walks_join(p) ? 3 : 2;
  e = launch_walks(p, all, pl.walks, true, GDN_STAGE_BWD_GRAD, s);
  if (e != hipSuccess) return e;
  if (all.n == 2) {
    Walks one{};
    one.n = 1;
    one.w[0] = dv_;
    e = launch_walks(p, one, pl.walks, true, GDN_STAGE_BWD_GRAD, s);
    if (e != hipSuccess) return e;
  }
  if (!shared) return hipSuccess;
  const int64_t tok = static_cast<int64_t>(p.B) * p.T;
  const int64_t pieces = tok * p.hq * (p.dk / 4);
  if (pieces == 0) return hipSuccess;
  StageScope scope(GDN_STAGE_OTHER, s);
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>((pieces + 255) / 256, 4096)), 2);
  const int32_t* cu = p.varlen ? p.cu_seqlens : nullptr;
  if (p.io == GDN_BF16)
    hipLaunchKernelGGL(linattn_share_kernel<bf16_t>, grid, dim3(256), 0, s, part_q,
                       part_k - part_q, dq, dk, tok, p.hq, p.H / p.hq, p.dk, cu, p.nseq);
  else
    hipLaunchKernelGGL(linattn_share_kernel<f32_t>, grid, dim3(256), 0, s, part_q,
                       part_k - part_q, dq, dk, tok, p.hq, p.H / p.hq, p.dk, cu, p.nseq);
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
