// kda_ssm.cuh -- the selective state space scan: a recurrence with one
// diagonal state per channel, for packed sequences, for training and for
// single tokens.
//
// Per channel c with N states, group g = c / (C / G), and a step d_t > 0:
//   d_t = dt_t + dt_bias, or log(1 + exp(dt_t + dt_bias))
//   h_t[n] = exp(d_t A[n]) h_{t-1}[n] + d_t u_t B_t[g, n]
//   y_t = sum_n C_t[g, n] h_t[n] + D u_t,   out_t = y_t or y_t z_t sigmoid(z_t)
//
// Each (channel, state) has a decay of its own, so there is no matrix product in
// it: an exponential, five multiplications and additions and the token's share of
// the loads per state. Its floor is the exponentials': the special-function unit
// does 16 a clock on an SM, 119 us for 8192 tokens x 4096 channels x 16 states,
// whose bytes take 41 us; with the softplus's and the gate's four more a channel,
// on the 128 SMs that 128 blocks use, 172 us. Measured there (bf16, gate): 282 us
// for one sequence (one warp of states a scheduler, which waits for its own results
// and for tiles: the unit is at 58 %), 240 us for eight of 1024 tokens, their
// gradients 1031 us, one token of 256 requests 25 us the kernel. fp32, with decays
// by polynomial: 562, 422 and 1628 us.
#pragma once

#include <type_traits>

#include "kda_io.cuh"

namespace kda {
namespace ssm {

constexpr int NTHREADS = 128;  // consumers of the forward scan; the other kernels' blocks
constexpr int KT = 8;          // tokens between kept states, for the gradients
constexpr int STAGES = 3;      // tiles of steps, B and C in flight
constexpr int YSLOTS = 2;      // tiles of outputs in flight

// Threads that share a channel's N states, four each.
inline int threads_per_channel(int N) { return N <= 16 ? 4 : N <= 32 ? 8 : N <= 64 ? 16 : 32; }
// Channels of a block of the forward scan and of its gradients.
inline int scan_channels(int N) { return 128 / threads_per_channel(N); }
inline int bwd_channels(int N) { return (N <= 32 ? 256 : 128) / threads_per_channel(N); }
// Blocks that an SM holds: of the scan, by registers; of the gradients, by
// registers (up to 32 states) and shared memory (above).
inline int scan_resident(int N) { return N <= 32 ? 2 : 1; }
inline int bwd_resident(int N) { return N <= 16 || (N > 32 && N <= 64) ? 2 : 1; }

struct Params {
  const void* u;
  const void* dt;
  const void* z;            // or null
  const void* b;
  const void* c;
  const float* A;           // [C, N]
  const float* D;           // [C] or null
  const float* dt_bias;     // [C] or null
  const int32_t* cu;
  const float* init;        // [NS, C, N] or null
  void* out;
  float* fin;               // [NS, C, N] or null
  float* ck;                // states before every KT tokens of a sequence, or null
  float* carry;             // time split: [ranges, C, N] each range's last state, else null
  float* sum_d;             // and [ranges, C] the sum of that piece's steps
  // the reverse pass of a time-split gradient
  const void* dout;
  const float* dfin;        // [NS, C, N] or null: zeros
  float* back;              // [ranges, C, N] the states' gradient before each range's first piece
  int64_t dout_st;
  int64_t T;
  int64_t run;              // time split: tokens per range, else 0 (a range is a sequence)
  int64_t u_st, dt_st, z_st, o_st, b_st, b_sg, c_st, c_sg;  // element strides over tokens and groups
  int NS, C, N, G;          // sequences, channels, states, groups
  int blocks_per_group;     // channel blocks of a group
  int softplus;
  int wide;                 // bits 0..5: rows of u, dt, z, B, C, out can be moved in pieces (u, dt, z, out: 2; B, C: S)
};

// log2(e) less its nearest fp32: the second part of a constant in two parts (the
// argument reduction of Cody and Waite)
constexpr float kLog2eRest = static_cast<float>(1.4426950408889634074 - static_cast<double>(kLog2e));
constexpr float kLn2 = 0.69314718055994530942f;

// The step: log(1 + exp(r)) = max(r, 0) + log1p(e) with e = exp(-|r|) in (0, 1],
// and log1p(e) = 2 atanh(s) with s = e / (2 + e) <= 1/3. atanh(s) / s as a
// polynomial in w = s^2 <= 1/9, of degree 6: its series to w^5 / 11 with the
// rest's size at w = 1/9 in the last term (below 2^-26 off).
// EXACT (fp32 inputs): exp's argument in two parts; as one its rounding costs
// |r| 2^-24 of the step, which 16-bit inputs do not show.
template <bool EXACT>
__device__ __forceinline__ float step_of(float r, int softplus) {
  if (!softplus) return r;
  float m = -fabsf(r);
  if (EXACT && m < -200.f) m = -200.f;  // e is 0 there; an infinity would make `rest` NaN
  const float x = m * kLog2e;
  float e = exp2_approx(x);
  if (EXACT) {
    const float rest = fmaf(m, kLog2e, -x) + m * kLog2eRest;
    e = fmaf(e * kLn2, rest, e);
  }
  const float s = __fdividef(e, 2.f + e), w = s * s;
  float t = fmaf(w, 1.f / 12, 1.f / 11);
  t = fmaf(w, t, 1.f / 9);
  t = fmaf(w, t, 1.f / 7);
  t = fmaf(w, t, 1.f / 5);
  t = fmaf(w, t, 1.f / 3);
  t = fmaf(w, t, 1.f);
  return fmaf(2.f * s, t, fmaxf(r, 0.f));
}

// step_of a pair
template <bool EXACT>
__device__ __forceinline__ float2 pstep(float2 r, int softplus) {
  if (!softplus) return r;
  float2 m = make_float2(-fabsf(r.x), -fabsf(r.y));
  if (EXACT) {
    if (m.x < -200.f) m.x = -200.f;
    if (m.y < -200.f) m.y = -200.f;
  }
  const float2 x = __fmul2_rn(m, pair_of(kLog2e));
  float2 e = pexp2(x);
  if (EXACT) {
    const float2 rest = __ffma2_rn(m, pair_of(kLog2eRest), __ffma2_rn(m, pair_of(kLog2e), make_float2(-x.x, -x.y)));
    e = __ffma2_rn(__fmul2_rn(e, pair_of(kLn2)), rest, e);
  }
  const float2 s = __fmul2_rn(e, prcp(__fadd2_rn(pair_of(2.f), e))), w = __fmul2_rn(s, s);
  float2 t = __ffma2_rn(w, pair_of(1.f / 12), pair_of(1.f / 11));
  t = __ffma2_rn(w, t, pair_of(1.f / 9));
  t = __ffma2_rn(w, t, pair_of(1.f / 7));
  t = __ffma2_rn(w, t, pair_of(1.f / 5));
  t = __ffma2_rn(w, t, pair_of(1.f / 3));
  t = __ffma2_rn(w, t, pair_of(1.f));
  return __ffma2_rn(__fadd2_rn(s, s), t, make_float2(fmaxf(r.x, 0.f), fmaxf(r.y, 0.f)));
}

// 2^x on the multiply-add pipe: x = n + f with n the nearest whole number (Cody
// and Waite), 2^f by a polynomial of degree 6 fitted by reweighted least squares
// (Lawson) for the least largest relative error on [-1/2, 1/2], 2e-9, n added to
// the exponent. In fp32 it is at most 8e-8 off, 3e-8 in the mean square, and
// without bias (1e-9 on average).
__device__ __forceinline__ float exp2_poly(float x) {
  const float c = x < -126.f ? -126.f : x > 128.f ? 128.f : x;  // NaN passes
  const float shifted = c + 12582912.f, f = c - (shifted - 12582912.f);  // 1.5 * 2^23: n in the low bits
  float t = fmaf(f, 1.5353362e-4f, 1.3398875e-3f);
  t = fmaf(f, t, 9.6184369e-3f);
  t = fmaf(f, t, 5.5503324e-2f);
  t = fmaf(f, t, 2.4022648e-1f);
  t = fmaf(f, t, 6.9314718e-1f);
  t = fmaf(f, t, 1.f);
  const float y = __int_as_float(__float_as_int(t) + (__float_as_int(shifted) << 23));
  return x == x ? y : x;
}

// h 2^x, the decay of a whole range of tokens, in two halves: with rates above 0
// 2^x alone can overflow where the product does not, and nothing stays nothing.
__device__ __forceinline__ float decayed(float h, float x) {
  const float e = exp2_poly(0.5f * x);
  return h == 0.f ? 0.f : h * e * e;
}

// The decay 2^(d a) of a token for two states. ex2.approx is low by 2e-8 on
// average (measured, 5e-9 to 3e-8 for exponents between -1 and 0), which a state
// that lasts n tokens takes n times; 1.5e-8 on the exponent, which the
// multiply-add brings for nothing, halves that. EXACT (fp32 tensors): without
// it, by the polynomial.
template <bool EXACT>
__device__ __forceinline__ float2 pdecay(float2 d, float2 a) {
  if constexpr (EXACT) {
    const float2 x = __fmul2_rn(d, a);
    return make_float2(exp2_poly(x.x), exp2_poly(x.y));
  } else {
    return pexp2(__ffma2_rn(d, a, pair_of(1.5e-8f)));
  }
}

template <bool EXACT>
__device__ __forceinline__ float decay(float d, float a) {
  return EXACT ? exp2_poly(d * a) : exp2_approx(fmaf(d, a, 1.5e-8f));
}

// S values at p as pairs (S = 1: the second half is 0)
template <int S>
__device__ __forceinline__ void load_pairs(float2 (&x)[(S + 1) / 2], const float* p) {
  if constexpr (S == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = make_float2(v.x, v.y);
    x[1] = make_float2(v.z, v.w);
  } else if constexpr (S == 2) {
    x[0] = *reinterpret_cast<const float2*>(p);
  } else {
    x[0] = make_float2(*p, 0.f);
  }
}

// The kept states of all sequences are numbered from start / KT + seq on:
// distinct, and at most T / KT + NS of them.
__device__ __forceinline__ int64_t first_kept(int64_t start, int seq) { return start / KT + seq; }

// A range's pieces of sequences, in order: f(seq, start, end, lo, hi) for the
// tokens [lo, hi) of the sequence [start, end). A range is a sequence, or, with
// the time split, `run` tokens of the packed batch (a multiple of BORDER), its
// borders moved up to the next multiple of BORDER tokens of the sequence that they
// cut. `which`: all pieces, the one that goes on in the next range, or the one
// that began in an earlier range.
constexpr int BORDER = 16;
enum { ALL_PIECES, GOES_ON, CAME_IN };
__device__ __forceinline__ int64_t border(int64_t r, int64_t start) {
  return start + (r - start + BORDER - 1) / BORDER * BORDER;
}
template <typename F>
__device__ __forceinline__ void split_pieces(const Params& p, int range, int which, F f) {
  const int64_t r0 = range * p.run, r1 = min(r0 + p.run, p.T);
  for (int s = first_sequence(p.cu, p.NS, which == GOES_ON ? r1 - 1 : r0); s < p.NS; ++s) {
    const int64_t start = bound(p.cu, s, p.T), end = bound(p.cu, s + 1, p.T);
    if (start >= r1 || (which == CAME_IN && start >= r0)) break;
    const int64_t lo = start >= r0 ? start : border(r0, start), hi = r1 < p.T ? min(end, border(r1, start)) : end;
    if (hi > lo && (which != GOES_ON || end > hi)) f(s, start, end, lo, hi);
  }
}
template <typename F>
__device__ __forceinline__ void for_pieces(const Params& p, int range, int which, F f) {
  if (p.run) return split_pieces(p, range, which, f);
  const int64_t start = bound(p.cu, range, p.T), end = max(start, bound(p.cu, range + 1, p.T));
  f(range, start, end, start, end);
}

// K rows of V elements, the rows base + row(k) * st. `all`: one access each; else
// the `valid` first elements one by one, zeros for the others. One branch for
// all rows, so that their loads are in flight together.
template <typename T, int V, int K, typename R>
__device__ __forceinline__ void load_rows(Vec<T, V> (&x)[K], const T* base, int64_t st, int valid, bool all, R row) {
  if (all) {
#pragma unroll
    for (int k = 0; k < K; ++k) x[k].load(base + row(k) * st);
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) x[k].load_some(base + row(k) * st, valid);
  }
}

constexpr int ROLE = NTHREADS;              // threads that make tiles; as many finish outputs

// What a scan leaves: the outputs; the states (every KT tokens, or a time split's
// carries); or the states' gradients before a time split's pieces, backwards.
enum { OUTPUTS, STATES, BACK };

// Two shapes of the forward scan. DEEP: one block per SM, longer tiles and more
// straight-line code, for grids that give an SM no second block; else two
// blocks per SM share it.
template <typename T, int L, int S, int CH, int MODE, bool DEEP>
struct FwdShared {
  static constexpr bool OUT = MODE == OUTPUTS;
  static constexpr int TT = DEEP ? 64 : 32;  // tokens per tile
  static constexpr int GT = DEEP ? 16 : 8;   // tokens of straight-line code in the states' loop
  static constexpr int STATE_THREADS = CH * L, THREADS = STATE_THREADS + (OUT ? 2 : 1) * ROLE;
  // The parts of the outputs: 16 bytes (four tokens) per thread and four
  // tokens, even channels before odd ones. The strides put the eight threads
  // of a store and of a load into different banks.
  static constexpr int ODD = CH / 2 * 16 + 64, QS = 2 * ODD + 16;
  float2 d[STAGES][TT][CH];        // d, d u
  alignas(16) float b[STAGES][TT][L * S], c[OUT ? STAGES : 1][OUT ? TT : 1][L * S];
  alignas(16) unsigned char y[YSLOTS][OUT ? TT / 4 : 1][L][QS];
  unsigned long long full[STAGES], empty[STAGES], y_full[YSLOTS], y_empty[YSLOTS];
};

// A ring of `n` slots: the slot in use and the parity of its current round.
template <int n>
struct Ring {
  int slot = 0;
  uint32_t phase;
  __device__ explicit Ring(uint32_t first) : phase(first) {}
  __device__ __forceinline__ void next() {
    if (++slot == n) {
      slot = 0;
      phase ^= 1;
    }
  }
};

// 128 / L channels of one range of tokens per block, in three roles of four
// warps: the states (L threads of S states per channel, one token after
// another), the tiles (TT tokens of d, d u, B and C into shared memory, a ring
// of STAGES) and the outputs (D u, the gate).
// Backwards (BACK) a tile holds the tokens from the last one on, C for B and the
// outputs' gradient for d u: g <- a (g + dy C).
//
// Why roles: with the same warps for everything the special-function unit waits
// for loads, softplus and stores (3.70 ms against 0.29 ms for 8192 x 4096 x 16).
// Why shared memory between them: B and C are one copy for all channels, and a
// shuffle costs a clock of the same pipe as a load. Counters at 4096 tokens, one
// sequence: exponentials 57 %, shared-memory wavefronts 54 %, issue 47 %.
template <typename T, int L, int S, int CH, int MODE, bool DEEP>
__global__ void __launch_bounds__(FwdShared<T, L, S, CH, MODE, DEEP>::THREADS,
                                  DEEP || L >= 16 ? 1 : MODE == OUTPUTS ? 2 : 3) ssm_fwd_kernel(Params p) {
  using Sh = FwdShared<T, L, S, CH, MODE, DEEP>;
  constexpr bool OUT = MODE == OUTPUTS;
  constexpr int SN = Sh::STATE_THREADS, TT = Sh::TT, GT = OUT ? Sh::GT : KT;
  extern __shared__ __align__(16) unsigned char smem[];
  Sh& sm = *reinterpret_cast<Sh*>(smem);
  const int role = threadIdx.x < SN ? 0 : 1 + (threadIdx.x - SN) / ROLE;
  const int tid = role == 0 ? threadIdx.x : (threadIdx.x - SN) % ROLE;
  const int range = blockIdx.y + (MODE == BACK ? 1 : 0);
  const int group = blockIdx.x / p.blocks_per_group, cg = p.C / p.G;
  const int c0 = group * cg + (blockIdx.x % p.blocks_per_group) * CH, c_end = min(c0 + CH, (group + 1) * cg);
  const bool split_pass = MODE == STATES && !p.ck;  // the time split's first pass
  const int which = MODE == BACK ? CAME_IN : split_pass ? GOES_ON : ALL_PIECES;
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&sm.full[i], ROLE / 32);
      mbar_init(&sm.empty[i], SN / 32);
    }
    for (int i = 0; i < YSLOTS; ++i) {
      mbar_init(&sm.y_full[i], SN / 32);
      mbar_init(&sm.y_empty[i], ROLE / 32);
    }
  }
  if (MODE != BACK && !split_pass && blockIdx.x == 0 && range == 0)
    for (int s = threadIdx.x; s < p.NS; s += Sh::THREADS) check_packing(p.cu, s, p.T);
  __syncthreads();
  if (role == 0) {  // -------------------------------------------- the states
    // Lanes: bit 1 (and the highest bits) the channel, the others the channel's
    // thread q. Wide loads from shared memory take half the time where lanes
    // that differ in bit 0 alone, or in bit 1 alone, read the same address: of
    // B and C the latter, of d the former (measured: 2 and 1 clocks, not 4 and 2).
    const int lane = tid % 32, rest = (lane & 1) | (lane >> 2 << 1);
    const int q = L == 32 ? lane : rest % L;
    const int ch = tid / 32 * (32 / L) + (L == 32 ? 0 : (lane >> 1 & 1) | rest / L << 1);
    const bool live = c0 + ch < c_end;
    constexpr int H = (S + 1) / 2;  // pairs
    float2 a[H], h[H];
    float av[2 * H], hv[2 * H];
    const int64_t row = static_cast<int64_t>(c0 + ch) * p.N + q * S, cn = static_cast<int64_t>(p.C) * p.N;
#pragma unroll
    for (int i = 0; i < 2 * H; ++i) av[i] = i < S && live && q * S + i < p.N ? p.A[row + i] * kLog2e : 0.f;
#pragma unroll
    for (int i = 0; i < H; ++i) a[i] = make_float2(av[2 * i], av[2 * i + 1]);
    Ring<STAGES> in(0);
    Ring<YSLOTS> yr(1);
    for_pieces(p, range, which, [&](int seq, int64_t start, int64_t end, int64_t lo, int64_t hi) {
      const int64_t at = seq * cn + row;
#pragma unroll
      for (int i = 0; i < 2 * H; ++i) {
        const bool on = i < S && live && q * S + i < p.N;
        if (MODE == BACK)
          hv[i] = on && p.dfin && hi == end ? p.dfin[at + i] : 0.f;
        else
          hv[i] = on && p.init && lo == start ? p.init[at + i] : 0.f;
        if (MODE != BACK && on && p.run && !split_pass && lo > start) {
          // the state before this range: those of the ranges since the sequence's start, decayed
          for (int64_t r = start / p.run; r < range; ++r)
            hv[i] = (r * p.run <= start ? 0.f : decayed(hv[i], av[i] * p.sum_d[r * p.C + c0 + ch])) +
                    p.carry[r * cn + row + i];
        }
      }
#pragma unroll
      for (int i = 0; i < H; ++i) h[i] = make_float2(hv[2 * i], hv[2 * i + 1]);
      float sum = 0.f;
      for (int64_t t0 = lo; t0 < hi; t0 += TT) {
        const int nt = static_cast<int>(min(static_cast<int64_t>(TT), hi - t0));
        mbar_wait(&sm.full[in.slot], in.phase);
        if (OUT) mbar_wait(&sm.y_empty[yr.slot], yr.phase);
        const float2* dp = &sm.d[in.slot][0][ch];
        const float* bp = &sm.b[in.slot][0][q * S];
        const float* cp = &sm.c[OUT ? in.slot : 0][0][q * S];
        unsigned char* yp = &sm.y[yr.slot][0][q][ch % 2 * Sh::ODD + ch / 2 * 16];
        for (int t = 0; t < nt; t += GT, dp += GT * CH, bp += GT * L * S, cp += GT * L * S, yp += GT / 4 * L * Sh::QS) {
          if (MODE == STATES && p.ck && live) {  // the state before token t, for the gradients
            const int64_t k = (first_kept(start, seq) + (t0 - start + t) / KT) * cn + row;
#pragma unroll
            for (int i = 0; i < H; ++i) hv[2 * i] = h[i].x, hv[2 * i + 1] = h[i].y;
            if (S == 4 && p.N % 4 == 0) {
              if (q * S < p.N) *reinterpret_cast<float4*>(p.ck + k) = make_float4(hv[0], hv[1], hv[2 % (2 * H)], hv[3 % (2 * H)]);
            } else {
#pragma unroll
              for (int i = 0; i < S; ++i)
                if (q * S + i < p.N) p.ck[k + i] = hv[i];
            }
          }
          float y[GT];
#pragma unroll
          for (int j = 0; j < GT; ++j) {  // past the piece's end d = 0: the state stays
            const float2 d = dp[j * CH];
            float2 b[H], c[H], acc;
            load_pairs<S>(b, bp + j * L * S);
            if (OUT) load_pairs<S>(c, cp + j * L * S);
            const float2 dd = make_float2(d.x, d.x), du = make_float2(d.y, d.y);
#pragma unroll
            for (int i = 0; i < H; ++i) {
              const float2 e = pdecay<sizeof(T) == 4>(dd, a[i]);
              h[i] = MODE == BACK ? __fmul2_rn(e, __ffma2_rn(du, b[i], h[i])) : __ffma2_rn(e, h[i], __fmul2_rn(du, b[i]));
              if (OUT) acc = i ? __ffma2_rn(c[i], h[i], acc) : __fmul2_rn(c[i], h[i]);
            }
            if (OUT) y[j] = S > 1 ? acc.x + acc.y : acc.x;
            if (split_pass) sum += d.x;
          }
          if (OUT) {
#pragma unroll
            for (int j = 0; j < GT; j += 4)
              *reinterpret_cast<float4*>(yp + j / 4 * L * Sh::QS) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
          }
        }
        mbar_arrive_warp(&sm.empty[in.slot]);
        if (OUT) mbar_arrive_warp(&sm.y_full[yr.slot]);
        in.next();
        yr.next();
      }
#pragma unroll
      for (int i = 0; i < H; ++i) hv[2 * i] = h[i].x, hv[2 * i + 1] = h[i].y;
      float* to = MODE == BACK ? p.back + range * cn + row
                  : split_pass ? p.carry + range * cn + row
                  : hi == end && p.fin ? p.fin + at : nullptr;
      if (live && to) {
#pragma unroll
        for (int i = 0; i < S; ++i)
          if (q * S + i < p.N) to[i] = hv[i];
      }
      if (split_pass && live && q == 0) p.sum_d[static_cast<int64_t>(range) * p.C + c0 + ch] = sum;
    });
    if (MODE != BACK && p.run && !split_pass && range == 0 && p.fin && live) {  // sequences without tokens
      for (int s = 0; s < p.NS; ++s) {
        if (bound(p.cu, s + 1, p.T) > bound(p.cu, s, p.T)) continue;
#pragma unroll
        for (int i = 0; i < S; ++i)
          if (q * S + i < p.N) p.fin[s * cn + row + i] = p.init ? p.init[s * cn + row + i] : 0.f;
      }
    }
    return;
  }
  // a thread's part of a tile: two channels of every TK-th token
  constexpr int ROWT = CH / 2, TK = ROLE / ROWT, NU = (TT + TK - 1) / TK;
  const int k0 = tid % ROWT * 2, tk = tid / ROWT, valid = max(0, min(2, c_end - c0 - k0));
  if (role == 1) {  // --------------------------------------------- the tiles
    constexpr bool BACKWARDS = MODE == BACK;
    const T* u = static_cast<const T*>(BACKWARDS ? p.dout : p.u) + c0 + k0;
    const T* dt = static_cast<const T*>(p.dt) + c0 + k0;
    const T* z = static_cast<const T*>(p.z) + c0 + k0;
    const T* bb = BACKWARDS ? static_cast<const T*>(p.c) + group * p.c_sg : static_cast<const T*>(p.b) + group * p.b_sg;
    const T* cc = static_cast<const T*>(p.c) + group * p.c_sg;
    const int64_t u_st = BACKWARDS ? p.dout_st : p.u_st, b_st = BACKWARDS ? p.c_st : p.b_st;
    float bias[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) bias[i] = p.dt_bias && i < valid ? p.dt_bias[c0 + k0 + i] : 0.f;
    constexpr int NB = (TT * L + ROLE - 1) / ROLE;
    Vec<T, 2> ru[NU], rd[NU], rz[BACKWARDS ? NU : 1];
    Vec<T, S> rb[NB], rc[NB];
    // rows past the piece's end: its last one again, set to 0 below
    const int n0 = tid % L * S, nv = max(0, min(S, p.N - n0));
    const bool all = !BACKWARDS && (p.wide & 1) && (p.wide & 2) && (p.wide & 8) && (p.wide & 16) && valid == 2 && nv == S &&
                     TT % TK == 0 && TT * L % ROLE == 0;
    auto load = [&](int64_t t0, int nt) {
      if (all && nt == TT) {  // nothing to check
        const T* pu = u + (t0 + tk) * p.u_st;
        const T* pd = dt + (t0 + tk) * p.dt_st;
        const T* pb = bb + n0 + (t0 + tid / L) * p.b_st;
        const T* pc = cc + n0 + (t0 + tid / L) * p.c_st;
#pragma unroll
        for (int k = 0; k < NU; ++k, pu += TK * p.u_st, pd += TK * p.dt_st) {
          ru[k].load(pu);
          rd[k].load(pd);
        }
#pragma unroll
        for (int k = 0; k < NB; ++k, pb += ROLE / L * p.b_st, pc += ROLE / L * p.c_st) {
          rb[k].load(pb);
          if (OUT) rc[k].load(pc);
        }
        return;
      }
      // backwards t0 is the tile's last token and the rows go down from it
      auto tok = [&](int k) { return t0 + (BACKWARDS ? -1 : 1) * min(tk + k * TK, nt - 1); };
      auto bct = [&](int k) { return t0 + (BACKWARDS ? -1 : 1) * min((tid + k * ROLE) / L, nt - 1); };
      load_rows(ru, u, u_st, valid, (p.wide & (BACKWARDS ? 32 : 1)) && valid == 2, tok);
      load_rows(rd, dt, p.dt_st, valid, (p.wide & 2) && valid == 2, tok);
      if constexpr (BACKWARDS) {
        if (p.z) load_rows(rz, z, p.z_st, valid, (p.wide & 4) && valid == 2, tok);
      }
      load_rows(rb, bb + n0, b_st, nv, (p.wide & (BACKWARDS ? 16 : 8)) && nv == S, bct);
      if (OUT) load_rows(rc, cc + n0, p.c_st, nv, (p.wide & 16) && nv == S, bct);
    };
    Ring<STAGES> to(1);
    for_pieces(p, range, which, [&](int, int64_t, int64_t, int64_t lo, int64_t hi) {
      auto first = [&](int64_t t0) { return BACKWARDS ? hi - 1 - (t0 - lo) : t0; };  // a tile's first row
      if (lo < hi) load(first(lo), static_cast<int>(min(static_cast<int64_t>(TT), hi - lo)));
      for (int64_t t0 = lo; t0 < hi; t0 += TT) {
        const int nt = static_cast<int>(min(static_cast<int64_t>(TT), hi - t0));
        // this tile's; the next one's loads go out before its arithmetic
        Vec<T, 2> tu[NU], td[NU], tz[BACKWARDS ? NU : 1];
        float wb[NB][S], wc[NB][S];
#pragma unroll
        for (int k = 0; k < NU; ++k) {
          tu[k] = ru[k];
          td[k] = rd[k];
          if constexpr (BACKWARDS) tz[k] = rz[k];
        }
#pragma unroll
        for (int k = 0; k < NB; ++k) {
#pragma unroll
          for (int i = 0; i < S; ++i) {
            wb[k][i] = rb[k].get(i);
            if (OUT) wc[k][i] = rc[k].get(i);
          }
          if (nt < TT && (tid + k * ROLE) / L >= nt) {
#pragma unroll
            for (int i = 0; i < S; ++i) wb[k][i] = wc[k][i] = 0.f;
          }
        }
        if (t0 + TT < hi) load(first(t0 + TT), static_cast<int>(min(static_cast<int64_t>(TT), hi - t0 - TT)));
        float4 v[NU];
        const bool short_tile = nt < TT || valid < 2;
#pragma unroll
        for (int k = 0; k < NU; ++k) {
          const float2 r = __fadd2_rn(make_float2(td[k].get(0), td[k].get(1)), make_float2(bias[0], bias[1]));
          const float2 d = pstep<sizeof(T) == 4>(r, p.softplus);
          float2 du = make_float2(tu[k].get(0), tu[k].get(1));
          if constexpr (BACKWARDS) {
            const float2 zz = make_float2(tz[k].get(0), tz[k].get(1));
            if (p.z) du = __fmul2_rn(du, psilu(zz));
          } else {
            du = __fmul2_rn(d, du);
          }
          v[k] = make_float4(d.x, du.x, d.y, du.y);
          if (short_tile) {
            const bool on = tk + k * TK < nt;
            v[k] = make_float4(on && valid > 0 ? v[k].x : 0.f, on && valid > 0 ? v[k].y : 0.f,
                               on && valid > 1 ? v[k].z : 0.f, on && valid > 1 ? v[k].w : 0.f);
          }
        }
        mbar_wait(&sm.empty[to.slot], to.phase);
#pragma unroll
        for (int k = 0; k < NU; ++k)
          if (TT % TK == 0 || tk + k * TK < TT)
            *reinterpret_cast<float4*>(&sm.d[to.slot][tk + k * TK][k0]) = v[k];
#pragma unroll
        for (int k = 0; k < NB; ++k)
          if (TT * L % ROLE == 0 || tid + k * ROLE < TT * L) {
            const int i = tid + k * ROLE;
            store_f32<float, S>(&sm.b[to.slot][i / L][i % L * S], wb[k]);
            if (OUT) store_f32<float, S>(&sm.c[to.slot][i / L][i % L * S], wc[k]);
          }
        mbar_arrive_warp(&sm.full[to.slot]);
        to.next();
      }
    });
    return;
  }
  if (OUT) {  // -------------------------------------------------- the outputs
    // a thread's part of a tile: two channels of four tokens, of every GK-th four
    constexpr int GK = ROLE / ROWT, NG = (TT / 4 + GK - 1) / GK;
    const T* u = static_cast<const T*>(p.u) + c0 + k0;
    const T* z = static_cast<const T*>(p.z) + c0 + k0;
    T* out = static_cast<T*>(p.out) + c0 + k0;
    float skip[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) skip[i] = p.D && i < valid ? p.D[c0 + k0 + i] : 0.f;
    Vec<T, 2> ru[4 * NG], rz[4 * NG];
    auto load = [&](int64_t t0, int nt) {
      if ((p.wide & 1) && (p.wide & 4) && valid == 2 && nt == TT && p.D && p.z && TT / 4 % GK == 0) {  // nothing to check
        const T* pu = u + (t0 + tk * 4) * p.u_st;
        const T* pz = z + (t0 + tk * 4) * p.z_st;
#pragma unroll
        for (int g = 0; g < NG; ++g, pu += 4 * GK * p.u_st, pz += 4 * GK * p.z_st)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            ru[g * 4 + j].load(pu + j * p.u_st);
            rz[g * 4 + j].load(pz + j * p.z_st);
          }
        return;
      }
      auto tok = [&](int k) { return t0 + min((tk + k / 4 * GK) * 4 + k % 4, nt - 1); };
      if (p.D) load_rows(ru, u, p.u_st, valid, (p.wide & 1) && valid == 2, tok);
      if (p.z) load_rows(rz, z, p.z_st, valid, (p.wide & 4) && valid == 2, tok);
    };
    Ring<YSLOTS> yr(0);
    for_pieces(p, range, which, [&](int, int64_t, int64_t, int64_t lo, int64_t hi) {
      if (lo < hi) load(lo, static_cast<int>(min(static_cast<int64_t>(TT), hi - lo)));
      for (int64_t t0 = lo; t0 < hi; t0 += TT) {
        const int nt = static_cast<int>(min(static_cast<int64_t>(TT), hi - t0));
        float2 du[4 * NG], gate[4 * NG];
#pragma unroll
        for (int k = 0; k < 4 * NG; ++k) {
          const float2 zz = make_float2(rz[k].get(0), rz[k].get(1));
          du[k] = p.D ? __fmul2_rn(make_float2(skip[0], skip[1]), make_float2(ru[k].get(0), ru[k].get(1))) : pair_of(0.f);
          gate[k] = p.z ? __fmul2_rn(zz, psigmoid(zz)) : pair_of(1.f);
        }
        if (t0 + TT < hi) load(t0 + TT, static_cast<int>(min(static_cast<int64_t>(TT), hi - t0 - TT)));
        mbar_wait(&sm.y_full[yr.slot], yr.phase);
        // whole: a full tile of full pairs, nothing to check
        auto write = [&](auto whole) {
          T* row = out + (t0 + tk * 4) * p.o_st;
#pragma unroll
          for (int g = 0; g < NG; ++g, row += 4 * GK * p.o_st) {
            const int tg = tk + g * GK;
            if (!(whole.value && TT / 4 % GK == 0) && tg * 4 >= nt) break;
            float4 even = make_float4(0.f, 0.f, 0.f, 0.f), odd = even;
            const unsigned char* yp = &sm.y[yr.slot][tg][0][k0 / 2 * 16];
#pragma unroll
            for (int l = 0; l < L; ++l) {
              const float4 a = *reinterpret_cast<const float4*>(yp + l * Sh::QS);
              const float4 b = *reinterpret_cast<const float4*>(yp + l * Sh::QS + Sh::ODD);
              even.x += a.x;
              even.y += a.y;
              even.z += a.z;
              even.w += a.w;
              odd.x += b.x;
              odd.y += b.y;
              odd.z += b.z;
              odd.w += b.w;
            }
            const float ev[4] = {even.x, even.y, even.z, even.w}, od[4] = {odd.x, odd.y, odd.z, odd.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int k = g * 4 + j;
              const float2 v = __fmul2_rn(__fadd2_rn(make_float2(ev[j], od[j]), du[k]), gate[k]);
              const float y[2] = {v.x, v.y};
              T* to = row + j * p.o_st;
              if (whole.value) {
                store_f32<T, 2>(to, y);
              } else if (tg * 4 + j < nt) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  if (i < valid) to[i] = from_f32<T>(y[i]);
              }
            }
          }
        };
        if (nt == TT && (p.wide & 32) && valid == 2) write(std::true_type());
        else write(std::false_type());
        mbar_arrive_warp(&sm.y_empty[yr.slot]);
        yr.next();
      }
    });
  }
}

// ------------------------------------------------------------ single tokens
constexpr int S = 4;  // states per thread of the kernels below

struct DecodeParams {
  const void* u;
  const void* dt;
  const void* z;
  const void* b;
  const void* c;
  const float* A;
  const float* D;
  const float* dt_bias;
  float* state;             // [P, C, N], read and written in place
  const int32_t* idx;       // [B] or null: slot b
  void* out;
  int64_t pool;
  int64_t u_st, dt_st, z_st, o_st, b_st, b_sg, c_st, c_sg;
  int C, N, G;
  int softplus;
  int wide;                 // bits 0, 1, 2: rows of B, C, state and A can be moved four states at a time; 3: four channels, several groups
};

// One block: 512 / L channels of one request, four channels per group of L
// threads; a thread holds four states of each, all loaded before any
// arithmetic. The state is read and written once (8 bytes a state against about
// 8 bytes of tokens a channel), so HBM bounds it. Thread j < 4 of a group
// computes the step of the group's channel j for the others, and its output.
template <typename T, int L>
__global__ void __launch_bounds__(NTHREADS) ssm_decode_kernel(DecodeParams p) {
  constexpr unsigned ALL = 0xffffffffu;
  const int64_t r = blockIdx.x;
  const int q = threadIdx.x % L, c0 = blockIdx.y * (NTHREADS / L * 4) + threadIdx.x / L * 4;
  int64_t slot = r;
  if (p.idx) {
    slot = p.idx[r];
    if (slot < 0 || slot >= p.pool) {  // uniform over the block
      if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(&g_device_flags, KDA_DEVICE_BAD_STATE_INDEX);
      return;
    }
  }
  const int mine = c0 + (q & 3);
  const bool owner = q < 4 && mine < p.C;
  const bool wide = p.wide & 4;
  const int n0 = q * S, nv = max(0, min(S, p.N - n0));
  float h[4][S], a[4][S];
  float* st = p.state + (slot * p.C + c0) * p.N + n0;
  const float* A = p.A + static_cast<int64_t>(c0) * p.N + n0;
  if (wide && nv == S && c0 + 4 <= p.C) {
#pragma unroll
    for (int j = 0; j < 4; ++j) load_f32<float, S>(h[j], st + j * p.N);
#pragma unroll
    for (int j = 0; j < 4; ++j) load_f32<float, S>(a[j], A + j * p.N);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const bool on = c0 + j < p.C && i < nv;
        h[j][i] = on ? st[j * p.N + i] : 0.f;
        a[j][i] = on ? A[j * p.N + i] : 0.f;
      }
  }
  float uu = 0.f, raw = 0.f, gate = 1.f, skip = 0.f;
  if (owner) {
    uu = to_f32(static_cast<const T*>(p.u)[r * p.u_st + mine]);
    raw = to_f32(static_cast<const T*>(p.dt)[r * p.dt_st + mine]) + (p.dt_bias ? p.dt_bias[mine] : 0.f);
    if (p.z) gate = to_f32(static_cast<const T*>(p.z)[r * p.z_st + mine]);
    if (p.D) skip = p.D[mine];
  }
  // the four channels may belong to different groups of B and C
  const bool several = p.wide & 8;
  const int cg = p.G > 1 ? p.C / p.G : p.C;
  float b[S], c[S];
  int group = -1;
  auto load_bc = [&](int g) {
    Vec<T, S> vb[1], vc[1];
    const bool all = nv == S;
    load_rows(vb, static_cast<const T*>(p.b) + r * p.b_st + g * p.b_sg + n0, 0, nv, all && (p.wide & 1), [](int) { return 0; });
    load_rows(vc, static_cast<const T*>(p.c) + r * p.c_st + g * p.c_sg + n0, 0, nv, all && (p.wide & 2), [](int) { return 0; });
    vb[0].get(b);
    vc[0].get(c);
    group = g;
  };
  load_bc(p.G > 1 ? min(c0, p.C - 1) / cg : 0);
  const float d = step_of<sizeof(T) == 4>(raw, p.softplus), du = d * uu;
  float y[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float dj = __shfl_sync(ALL, d, j, L), uj = __shfl_sync(ALL, du, j, L);
    if (several && j && c0 + j < p.C && (c0 + j) / cg != group) load_bc((c0 + j) / cg);
    y[j] = 0.f;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      h[j][i] = fmaf(decay<sizeof(T) == 4>(dj, a[j][i] * kLog2e), h[j][i], uj * b[i]);
      y[j] = fmaf(c[i], h[j][i], y[j]);
    }
  }
  if (wide && nv == S && c0 + 4 <= p.C) {
#pragma unroll
    for (int j = 0; j < 4; ++j) store_f32<float, S>(st + j * p.N, h[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < S; ++i)
        if (c0 + j < p.C && i < nv) st[j * p.N + i] = h[j][i];
  }
  // over the group's threads: thread q ends with channel q % 4
  const bool up2 = q & 2, up1 = q & 1;
  const float y0 = (up2 ? y[2] : y[0]) + __shfl_xor_sync(ALL, up2 ? y[0] : y[2], 2);
  const float y1 = (up2 ? y[3] : y[1]) + __shfl_xor_sync(ALL, up2 ? y[1] : y[3], 2);
  float v = (up1 ? y1 : y0) + __shfl_xor_sync(ALL, up1 ? y0 : y1, 1);
#pragma unroll
  for (int o = 4; o < L; o <<= 1) v += __shfl_xor_sync(ALL, v, o);
  if (owner) {
    v = fmaf(skip, uu, v);
    if (p.z) v *= silu(gate);
    static_cast<T*>(p.out)[r * p.o_st + mine] = from_f32<T>(v);
  }
}

// ---------------------------------------------------------------- backward
struct BwdParams {
  Params f;                 // the forward's inputs, dout and dfin; ck filled by its states-only pass
  void* du;
  void* ddt;
  void* dz;                 // with z
  float* dinit;             // [NS, C, N] or null
  float* part_a;            // [ranges, C, N]
  float* part_d;            // [2, ranges, C]: dD, ddt_bias
  float* part_b;            // [channel blocks, T, N]
  float* part_c;
  int64_t du_st, ddt_st, dz_st;
};

constexpr int TB = 16;  // tokens per tile of the gradients, in two halves of KT

// The gradients' block: WARPS warps of 32 / L channels, L threads of four states
// per channel.
template <int L>
struct BwdShared {
  static constexpr int WARPS = L <= 8 ? 8 : 4, THREADS = 32 * WARPS;
  static constexpr int CH = WARPS * 32 / L;                  // channels
  static constexpr int FB = L <= 8 ? 4 : L == 16 ? 2 : 1;    // orders of B and C, see the kernel
  // parts of sums, 16 bytes (four tokens) per thread, even channels before odd
  // ones; the strides put the threads of a store and of a load into different banks
  static constexpr int ODD = CH / 2 * 16 + 64, QS = 2 * ODD + 16;
  float2 d[TB][CH];            // d, d u
  float dy[TB][CH];            // the output's gradient, through the gate
  float2 u[TB][CH / 2], sig[TB][CH / 2], zf[TB][CH / 2];  // u; softplus'; dout times the gate's slope
  alignas(16) float b[TB][FB][4 * L], c[TB][FB][4 * L];
  alignas(16) unsigned char sum[3][TB / 4][L][QS];  // sum_n g B, sum_n w A, sum_n C h by threads
  float db[WARPS][TB][4 * L], dc[WARPS][TB][4 * L];
  float4 da[THREADS];          // each thread's sum for dA over the tiles (its own; not in registers, for want of them)
};

// The sequence backwards, a tile at a time: from the kept states its states and
// decays again, KT tokens in registers, then the reverse recurrence
//   g_t = dy_t C_t + a_{t+1} g_{t+1},  w_t = a_t g_t h_{t-1}
//   dC += dy h,  dB += g d u,  dd = sum_n w A + u sum_n g B,  du = d sum_n g B + D dy,  dA += d w
//
// dB and dC are sums over channels, that is over lanes. A lane's register i holds
// state i ^ f of its four, f from two of the lane's channel bits: then the lanes
// of a pair that differ in a bit of f send registers of the same number and
// keep the others, two exchanges and one instead of four a step, without
// selecting by lane. B and C stand in shared memory in each order.
//
// KT = 8 tokens of decays and states are 64 registers a thread, which leaves 16
// warps an SM. Counters at 8 x 512 tokens x 4096 x 16: shared-memory wavefronts
// 66 %, issue 58 %, exponentials 22 %; 839 us at 8 x 1024.
//
// SPLIT: a range of the time split, its pieces one after another. The states'
// gradient behind a piece comes from the reverse scans (BACK) of the ranges up to
// its sequence's end. A form of its own: the unsplit one is short of registers
// (the same loop with g's start where the split needs it: 44 bytes more spilled,
// 5 % of the time).
template <typename T, int L, bool SPLIT>
__global__ void __launch_bounds__(BwdShared<L>::THREADS, L == 4 ? 2 : 1) ssm_bwd_kernel(BwdParams bp) {
  using Sh = BwdShared<L>;
  const Params& p = bp.f;
  constexpr int CH = Sh::CH, FB = Sh::FB, NT = Sh::THREADS, NP = 4 * L;
  constexpr unsigned ALL = 0xffffffffu;
  extern __shared__ __align__(16) unsigned char smem[];
  Sh& sm = *reinterpret_cast<Sh*>(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // lane bits of the thread's state group q, its channel and its order f
  const int b1 = lane >> 1 & 1, top = lane >> 3, rest = (lane & 1) | (lane >> 2 << 1);
  const int q = L == 32 ? lane : rest % L;
  const int chl = warp * (32 / L) + (L == 32 ? 0 : L == 4 ? b1 | top << 1 : b1 | rest / L << 1);
  const int f = L == 4 ? top : L == 8 ? b1 | (lane >> 4) << 1 : L == 16 ? b1 : 0;
  const int group = blockIdx.x / p.blocks_per_group, cg = p.C / p.G;
  const int c0 = group * cg + (blockIdx.x % p.blocks_per_group) * CH, c_end = min(c0 + CH, (group + 1) * cg);
  const int64_t cn = static_cast<int64_t>(p.C) * p.N;
  const int ch = c0 + chl;
  const bool live = ch < c_end;
  float2 a[2], g[2];
  {
    float av[4], gv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = q * 4 + (i ^ f);
      const bool on = live && n < p.N;
      const int64_t at = static_cast<int64_t>(ch) * p.N + n;
      av[i] = on ? p.A[at] * kLog2e : 0.f;
      gv[i] = !SPLIT && on && p.dfin ? p.dfin[blockIdx.y * cn + at] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a[i] = make_float2(av[2 * i], av[2 * i + 1]);
      g[i] = make_float2(gv[2 * i], gv[2 * i + 1]);
    }
  }
  sm.da[tid] = make_float4(0.f, 0.f, 0.f, 0.f);
  unsigned char* const sum_row = &sm.sum[0][0][q][chl % 2 * Sh::ODD + chl / 2 * 16];
  constexpr int SUM = TB / 4 * L * Sh::QS;  // bytes between the kinds of sums
  // this thread's part of a tile before and after the states: a channel pair's TG tokens
  constexpr int PAIRS = CH / 2, TG = TB * PAIRS / NT > 0 ? TB * PAIRS / NT : 1;
  const int mp = tid % PAIRS, m0 = tid / PAIRS * TG, mc = c0 + 2 * mp, valid = max(0, min(2, c_end - mc));
  float bias[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) bias[c] = p.dt_bias && c < valid ? p.dt_bias[mc + c] : 0.f;
  // and after them: a channel's four tokens from xt on
  const int xc = tid % CH, xt = tid / CH * 4;
  const float skip = p.D && c0 + xc < c_end ? p.D[c0 + xc] : 0.f;
  float sum_d = 0.f, sum_bias = 0.f;
  auto piece = [&](int seq, int64_t start, int64_t end, int64_t lo, int64_t hi) {
  if constexpr (SPLIT) {  // the states' gradient after the piece
    // pieces up to the sequence's end: theirs, decayed; the last one brings the final state's
    int64_t last = blockIdx.y;
    while (last + 1 < gridDim.y && border((last + 1) * p.run, start) < end) ++last;
    float gv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = q * 4 + (i ^ f);
      const bool on = live && n < p.N;
      const int64_t at = static_cast<int64_t>(ch) * p.N + n;
      gv[i] = on && p.dfin && hi == end ? p.dfin[seq * cn + at] : 0.f;
      for (int64_t r = hi < end && on ? last : 0; r > blockIdx.y; --r)
        gv[i] = (r == last ? 0.f : decayed(gv[i], p.A[at] * kLog2e * p.sum_d[r * p.C + ch])) + p.back[r * cn + at];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) g[i] = make_float2(gv[2 * i], gv[2 * i + 1]);
  }
  const int64_t tiles = (hi - start + TB - 1) / TB, tile0 = (lo - start) / TB;
  // A tile's rows as they came and the state kept before its last half: loaded
  // while the tile after it is finished.
  constexpr int NB = (TB * L + NT - 1) / NT;
  Vec<T, 2> vu[TG], vd[TG], vz[TG], vo[TG];
  Vec<T, 4> vb[NB], vc[NB];
  float kept[4] = {0.f, 0.f, 0.f, 0.f};
  const int64_t kept0 = (first_kept(start, seq) * p.C + ch) * p.N + q * 4;
  auto load_kept = [&](int64_t tile, int half) {
    const int64_t at = kept0 + (tile * (TB / KT) + half) * cn;
    if (p.N % 4 == 0) {
      if (live && q * 4 < p.N) load_f32<float, 4>(kept, p.ck + at);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (live && q * 4 + i < p.N) kept[i] = p.ck[at + i];
    }
  };
  const int n0 = tid % L * 4, nv = max(0, min(4, p.N - n0));
  auto load_tile = [&](int64_t tile) {
    const int64_t t0 = start + tile * TB;
    const int nt = static_cast<int>(min(static_cast<int64_t>(TB), hi - t0));
    if (m0 < TB) {
      auto tok = [&](int j) { return t0 + min(m0 + j, nt - 1); };
      load_rows(vd, static_cast<const T*>(p.dt) + mc, p.dt_st, valid, (p.wide & 2) && valid == 2, tok);
      load_rows(vu, static_cast<const T*>(p.u) + mc, p.u_st, valid, (p.wide & 1) && valid == 2, tok);
      load_rows(vo, static_cast<const T*>(p.dout) + mc, p.dout_st, valid, (p.wide & 32) && valid == 2, tok);
      if (p.z) load_rows(vz, static_cast<const T*>(p.z) + mc, p.z_st, valid, (p.wide & 4) && valid == 2, tok);
    }
    if (tid < TB * L) {
      auto tok = [&](int j) { return t0 + min((tid + j * NT) / L, nt - 1); };
      load_rows(vb, static_cast<const T*>(p.b) + group * p.b_sg + n0, p.b_st, nv, (p.wide & 8) && nv == 4, tok);
      load_rows(vc, static_cast<const T*>(p.c) + group * p.c_sg + n0, p.c_st, nv, (p.wide & 16) && nv == 4, tok);
    }
    load_kept(tile, nt > KT ? 1 : 0);
  };
  if (tiles > tile0) load_tile(tiles - 1);
  for (int64_t k = tiles - 1; k >= tile0; --k) {
    const int64_t t0 = start + k * TB;
    const int nt = static_cast<int>(min(static_cast<int64_t>(TB), hi - t0));
    // ------------------------------------------------ the tile's operands
    if (m0 < TB) {
#pragma unroll
      for (int j = 0; j < TG; ++j) {
        const int t = m0 + j;
        float d[2], du[2], dy[2], uu[2], sg[2], zf[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float r = vd[j].get(c) + bias[c];
          d[c] = step_of<sizeof(T) == 4>(r, p.softplus);
          sg[c] = p.softplus ? sigmoid(r) : 1.f;
          uu[c] = vu[j].get(c);
          dy[c] = vo[j].get(c);
          zf[c] = 0.f;
          if (p.z) {
            const float zz = vz[j].get(c), s = sigmoid(zz);
            zf[c] = dy[c] * s * fmaf(zz, 1.f - s, 1.f);
            dy[c] *= zz * s;
          }
          du[c] = d[c] * uu[c];
          if (t >= nt || c >= valid) d[c] = du[c] = dy[c] = uu[c] = 0.f;  // the state stays, nothing is added
        }
        *reinterpret_cast<float4*>(&sm.d[t][2 * mp]) = make_float4(d[0], du[0], d[1], du[1]);
        *reinterpret_cast<float2*>(&sm.dy[t][2 * mp]) = make_float2(dy[0], dy[1]);
        sm.u[t][mp] = make_float2(uu[0], uu[1]);
        sm.sig[t][mp] = make_float2(sg[0], sg[1]);
        if (p.z) sm.zf[t][mp] = make_float2(zf[0], zf[1]);
      }
    }
    if (tid < TB * L) {
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int t = (tid + j * NT) / L;
        float fb[4], fc[4];
        vb[j].get(fb);
        vc[j].get(fc);
        if (t >= nt) {
#pragma unroll
          for (int i = 0; i < 4; ++i) fb[i] = fc[i] = 0.f;
        }
#pragma unroll
        for (int o = 0; o < FB; ++o) {
          *reinterpret_cast<float4*>(&sm.b[t][o][n0]) = make_float4(fb[0 ^ o], fb[1 ^ o], fb[2 ^ o], fb[3 ^ o]);
          *reinterpret_cast<float4*>(&sm.c[t][o][n0]) = make_float4(fc[0 ^ o], fc[1 ^ o], fc[2 ^ o], fc[3 ^ o]);
        }
      }
    }
    __syncthreads();
    // -------------------------------------------------------- the states
    float2 da_tile[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};  // by tile: fewer roundings than one long sum
#pragma unroll 1
    for (int half = 1; half >= 0; --half) {
      if (half * KT >= nt) continue;
      float2 h0[2], e[KT][2], h[KT][2];
      {  // the kept state, into the lane's order
        const float* v = kept;
        const bool f0 = f & 1, f1 = f & 2;
        const float w0 = f0 ? v[1] : v[0], w1 = f0 ? v[0] : v[1], w2 = f0 ? v[3] : v[2], w3 = f0 ? v[2] : v[3];
        h0[0] = f1 ? make_float2(w2, w3) : make_float2(w0, w1);
        h0[1] = f1 ? make_float2(w0, w1) : make_float2(w2, w3);
      }
      if (half == 1) load_kept(k, 0);
      const float2* const dp = &sm.d[half * KT][chl];
      const float* const yp = &sm.dy[half * KT][chl];
      const float* const bq = &sm.b[half * KT][f][q * 4];
      const float* const cq = &sm.c[half * KT][f][q * 4];
      unsigned char* const sr = sum_row + half * (KT / 4) * (L * Sh::QS);
      float y[4];
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        const float2 d = dp[t * CH];
        const float4 b4 = *reinterpret_cast<const float4*>(bq + t * FB * NP);
        const float2 b[2] = {make_float2(b4.x, b4.y), make_float2(b4.z, b4.w)};
        const float2 dd = make_float2(d.x, d.x), du = make_float2(d.y, d.y);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          e[t][i] = pdecay<sizeof(T) == 4>(dd, a[i]);
          h[t][i] = __ffma2_rn(e[t][i], t ? h[t - 1][i] : h0[i], __fmul2_rn(du, b[i]));
        }
        if (p.z) {
          const float4 c4 = *reinterpret_cast<const float4*>(cq + t * FB * NP);
          const float2 s = __ffma2_rn(make_float2(c4.z, c4.w), h[t][1], __fmul2_rn(make_float2(c4.x, c4.y), h[t][0]));
          y[t % 4] = s.x + s.y;
          if (t % 4 == 3)
            *reinterpret_cast<float4*>(sr + 2 * SUM + t / 4 * (L * Sh::QS)) = make_float4(y[0], y[1], y[2], y[3]);
        }
      }
      float s1[4], s2[4];
      float hold_b = 0.f, hold_c = 0.f;
#pragma unroll
      for (int t = KT - 1; t >= 0; --t) {
        const int at = half * KT + t;
        const float2 d = dp[t * CH];
        const float yy = yp[t * CH];
        const float4 b4 = *reinterpret_cast<const float4*>(bq + t * FB * NP);
        const float4 c4 = *reinterpret_cast<const float4*>(cq + t * FB * NP);
        const float2 b[2] = {make_float2(b4.x, b4.y), make_float2(b4.z, b4.w)};
        const float2 cv[2] = {make_float2(c4.x, c4.y), make_float2(c4.z, c4.w)};
        const float2 dd = make_float2(d.x, d.x), du = make_float2(d.y, d.y), y2 = make_float2(yy, yy);
        float2 vb[2], vc[2], p1, p2;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 gg = __ffma2_rn(y2, cv[i], g[i]);
          vc[i] = __fmul2_rn(y2, h[t][i]);
          vb[i] = __fmul2_rn(du, gg);
          p1 = i ? __ffma2_rn(gg, b[i], p1) : __fmul2_rn(gg, b[i]);
          g[i] = __fmul2_rn(gg, e[t][i]);
          const float2 w = __fmul2_rn(g[i], t ? h[t - 1][i] : h0[i]);
          p2 = i ? __ffma2_rn(w, a[i], p2) : __fmul2_rn(w, a[i]);
          da_tile[i] = __ffma2_rn(w, dd, da_tile[i]);
        }
        s1[t % 4] = p1.x + p1.y;
        s2[t % 4] = p2.x + p2.y;
        if (t % 4 == 0) {
          *reinterpret_cast<float4*>(sr + t / 4 * (L * Sh::QS)) = make_float4(s1[0], s1[1], s1[2], s1[3]);
          *reinterpret_cast<float4*>(sr + SUM + t / 4 * (L * Sh::QS)) = make_float4(s2[0], s2[1], s2[2], s2[3]);
        }
        // dB and dC over the warp's channels
        if constexpr (L <= 8) {
          vb[0].x += __shfl_xor_sync(ALL, vb[1].x, 16);
          vb[0].y += __shfl_xor_sync(ALL, vb[1].y, 16);
          vc[0].x += __shfl_xor_sync(ALL, vc[1].x, 16);
          vc[0].y += __shfl_xor_sync(ALL, vc[1].y, 16);
          float rb = vb[0].x + __shfl_xor_sync(ALL, vb[0].y, L == 4 ? 8 : 2);
          float rc = vc[0].x + __shfl_xor_sync(ALL, vc[0].y, L == 4 ? 8 : 2);
          if constexpr (L == 4) {
            // two tokens: the lanes with bit 1 end with the earlier one
            if (t % 2 == 1) {
              hold_b = rb;
              hold_c = rc;
            } else {
              rb = (b1 ? rb : hold_b) + __shfl_xor_sync(ALL, b1 ? hold_b : rb, 2);
              rc = (b1 ? rc : hold_c) + __shfl_xor_sync(ALL, b1 ? hold_c : rc, 2);
              sm.db[warp][at + 1 - b1][q * 4 + f] = rb;
              sm.dc[warp][at + 1 - b1][q * 4 + f] = rc;
            }
          } else {
            sm.db[warp][at][q * 4 + f] = rb;
            sm.dc[warp][at][q * 4 + f] = rc;
          }
        } else if constexpr (L == 16) {
          sm.db[warp][at][q * 4 + f] = vb[0].x + __shfl_xor_sync(ALL, vb[0].y, 2);
          sm.db[warp][at][q * 4 + (2 ^ f)] = vb[1].x + __shfl_xor_sync(ALL, vb[1].y, 2);
          sm.dc[warp][at][q * 4 + f] = vc[0].x + __shfl_xor_sync(ALL, vc[0].y, 2);
          sm.dc[warp][at][q * 4 + (2 ^ f)] = vc[1].x + __shfl_xor_sync(ALL, vc[1].y, 2);
        } else {
          *reinterpret_cast<float4*>(&sm.db[warp][at][q * 4]) = make_float4(vb[0].x, vb[0].y, vb[1].x, vb[1].y);
          *reinterpret_cast<float4*>(&sm.dc[warp][at][q * 4]) = make_float4(vc[0].x, vc[0].y, vc[1].x, vc[1].y);
        }
      }
    }
    const float4 da = sm.da[tid];
    sm.da[tid] = make_float4(da.x + da_tile[0].x, da.y + da_tile[0].y, da.z + da_tile[1].x, da.w + da_tile[1].y);
    __syncthreads();
    // ------------------------------------------------------- the gradients
    if (k > tile0) load_tile(k - 1);
    for (int i = tid; i < nt * NP; i += NT) {
      const int t = i / NP, n = i % NP;
      if (n >= p.N) continue;
      float vb = 0.f, vc = 0.f;
#pragma unroll
      for (int w = 0; w < Sh::WARPS; ++w) {
        vb += sm.db[w][t][n];
        vc += sm.dc[w][t][n];
      }
      const int64_t at = (static_cast<int64_t>(blockIdx.x) * p.T + t0 + t) * p.N + n;
      bp.part_b[at] = vb;
      bp.part_c[at] = vc;
    }
    if (xt < nt) {
      float s[3][4] = {};
#pragma unroll
      for (int m = 0; m < 3; ++m) {
        if (m == 2 && !p.z) break;
#pragma unroll
        for (int l = 0; l < L; ++l) {
          const float4 v = *reinterpret_cast<const float4*>(&sm.sum[m][xt / 4][l][xc % 2 * Sh::ODD + xc / 2 * 16]);
          s[m][0] += v.x;
          s[m][1] += v.y;
          s[m][2] += v.z;
          s[m][3] += v.w;
        }
      }
      const int64_t row = t0 + xt;
      T* gd = static_cast<T*>(bp.ddt) + row * bp.ddt_st + c0 + xc;
      T* gu = static_cast<T*>(bp.du) + row * bp.du_st + c0 + xc;
      T* gz = static_cast<T*>(bp.dz) + row * bp.dz_st + c0 + xc;
#pragma unroll
      for (int j = 3; j >= 0; --j) {
        const int t = xt + j;
        if (t >= nt || c0 + xc >= c_end) continue;
        const float2 d = sm.d[t][xc];
        const float dy = sm.dy[t][xc], uu = (&sm.u[t][0].x)[xc];
        const float dd = (&sm.sig[t][0].x)[xc] * fmaf(uu, s[0][j], s[1][j] * kLn2);  // A came times log2(e)
        sum_bias += dd;
        sum_d = fmaf(dy, uu, sum_d);
        gd[j * bp.ddt_st] = from_f32<T>(dd);
        gu[j * bp.du_st] = from_f32<T>(fmaf(d.x, s[0][j], skip * dy));
        if (p.z) gz[j * bp.dz_st] = from_f32<T>((&sm.zf[t][0].x)[xc] * fmaf(skip, uu, s[2][j]));
      }
    }
    __syncthreads();
  }
  if (bp.dinit && lo == start) {
    const float gv[4] = {g[0].x, g[0].y, g[1].x, g[1].y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = q * 4 + (i ^ f);
      if (live && n < p.N) bp.dinit[seq * cn + static_cast<int64_t>(ch) * p.N + n] = gv[i];
    }
  }
  };
  if constexpr (SPLIT) {
    split_pieces(p, blockIdx.y, ALL_PIECES, piece);
    if (blockIdx.y == 0 && bp.dinit && live) {  // sequences without tokens
      for (int s = 0; s < p.NS; ++s) {
        if (bound(p.cu, s + 1, p.T) > bound(p.cu, s, p.T)) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = q * 4 + (i ^ f);
          const int64_t at = s * cn + static_cast<int64_t>(ch) * p.N + n;
          if (n < p.N) bp.dinit[at] = p.dfin ? p.dfin[at] : 0.f;
        }
      }
    }
  } else {
    const int64_t start = bound(p.cu, blockIdx.y, p.T), end = max(start, bound(p.cu, blockIdx.y + 1, p.T));
    piece(blockIdx.y, start, end, start, end);
  }
  const float4 da = sm.da[tid];
  const float dv[4] = {da.x, da.y, da.z, da.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = q * 4 + (i ^ f);
    if (live && n < p.N) bp.part_a[blockIdx.y * cn + static_cast<int64_t>(ch) * p.N + n] = dv[i];
  }
  // dD and ddt_bias: over the threads of a channel
  float2* sums = reinterpret_cast<float2*>(sm.sum);
  static_assert(sizeof(float2) * NT <= sizeof(sm.sum), "");
  sums[tid] = make_float2(sum_d, sum_bias);
  __syncthreads();
  if (tid < CH && c0 + tid < c_end) {
    float2 v = sums[tid];
    for (int i = tid + CH; i < NT; i += CH) {
      v.x += sums[i].x;
      v.y += sums[i].y;
    }
    bp.part_d[static_cast<int64_t>(blockIdx.y) * p.C + c0 + tid] = v.x;
    bp.part_d[(static_cast<int64_t>(gridDim.y) + blockIdx.y) * p.C + c0 + tid] = v.y;
  }
}

struct ReduceParams {
  const float* part_a;
  const float* part_d;
  const float* part_b;
  const float* part_c;
  const int32_t* cu;
  float* dA;
  float* dD;                // or null
  float* ddt_bias;          // or null
  void* dB;
  void* dC;
  void* du;
  void* ddt;
  void* dz;                 // or null
  int64_t T, dB_st, dB_sg, dC_st, dC_sg, du_st, ddt_st, dz_st;
  int NS, parts, C, N, G, blocks_per_group;  // parts: ranges with sums for dA, dD, ddt_bias
};

// Sums over the ranges (dA, dD, ddt_bias) and the channel blocks of a group
// (dB, dC), in order; zeros at tokens of no sequence.
template <typename T>
__global__ void __launch_bounds__(256) ssm_reduce_kernel(ReduceParams p) {
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, stride = static_cast<int64_t>(gridDim.x) * 256;
  const int64_t cn = static_cast<int64_t>(p.C) * p.N;
  for (int64_t i = i0; i < cn; i += stride) {
    float a = 0.f;
    for (int s = 0; s < p.parts; ++s) a += p.part_a[s * cn + i];
    p.dA[i] = a;
  }
  for (int64_t i = i0; i < 2 * static_cast<int64_t>(p.C); i += stride) {
    float* to = i < p.C ? p.dD : p.ddt_bias;
    if (!to) continue;
    const int64_t c = i < p.C ? i : i - p.C;
    float a = 0.f;
    for (int s = 0; s < p.parts; ++s) a += p.part_d[((i < p.C ? 0 : static_cast<int64_t>(p.parts)) + s) * p.C + c];
    to[c] = a;
  }
  const int64_t lo = bound(p.cu, 0, p.T), hi = bound(p.cu, p.cu ? p.NS : 1, p.T);
  const int64_t gn = static_cast<int64_t>(p.G) * p.N;
  for (int64_t i = i0; i < p.T * gn; i += stride) {
    const int64_t t = i / gn;
    const int g = static_cast<int>(i % gn / p.N), n = static_cast<int>(i % p.N);
    float vb = 0.f, vc = 0.f;
    if (t >= lo && t < hi) {
#pragma unroll 16
      for (int k = 0; k < p.blocks_per_group; ++k) {  // loads in flight
        const int64_t at = (static_cast<int64_t>(g * p.blocks_per_group + k) * p.T + t) * p.N + n;
        vb += p.part_b[at];
        vc += p.part_c[at];
      }
    }
    static_cast<T*>(p.dB)[t * p.dB_st + g * p.dB_sg + n] = from_f32<T>(vb);
    static_cast<T*>(p.dC)[t * p.dC_st + g * p.dC_sg + n] = from_f32<T>(vc);
  }
  const int64_t out = p.T - (hi > lo ? hi - lo : 0);
  for (int64_t i = i0; i < out * p.C; i += stride) {
    int64_t t = i / p.C;
    const int64_t c = i % p.C;
    if (hi > lo && t >= lo) t += hi - lo;
    static_cast<T*>(p.du)[t * p.du_st + c] = from_f32<T>(0.f);
    static_cast<T*>(p.ddt)[t * p.ddt_st + c] = from_f32<T>(0.f);
    if (p.dz) static_cast<T*>(p.dz)[t * p.dz_st + c] = from_f32<T>(0.f);
  }
}

}  // namespace ssm
}  // namespace kda
