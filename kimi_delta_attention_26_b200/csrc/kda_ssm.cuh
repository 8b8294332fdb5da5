// kda_ssm.cuh -- the selective state space scan: a recurrence with one
// diagonal state per channel, for packed sequences, for training and for
// single tokens.
//
// Per channel c with N states, group g = c / (C / G), and a step d_t > 0:
//   d_t = dt_t + dt_bias, or log(1 + exp(dt_t + dt_bias))
//   h_t[n] = exp(d_t A[n]) h_{t-1}[n] + d_t u_t B_t[g, n]
//   y_t = sum_n C_t[g, n] h_t[n] + D u_t,   out_t = y_t or y_t z_t sigmoid(z_t)
#pragma once

#include "kda_io.cuh"

namespace kda {
namespace ssm {

constexpr int NTHREADS = 128;
constexpr int S = 4;    // states per thread
constexpr int TT = 16;  // tokens per tile

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
  float* ck;                // states before each tile, or null
  int64_t T;
  int64_t u_st, dt_st, z_st, o_st, b_st, b_sg, c_st, c_sg;  // element strides over tokens and groups
  int NS, C, N, G;          // sequences, channels, states, groups
  int blocks_per_group;     // channel blocks of a group
  int softplus;
};

__device__ __forceinline__ float step_of(float r, int softplus) {
  return softplus ? (r > 20.f ? r : log1pf(expf(r))) : r;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// The tiles of all sequences are numbered from start / TT + seq on: distinct,
// and at most T / TT + NS of them.
__device__ __forceinline__ int64_t first_tile(int64_t start, int seq) { return start / TT + seq; }

// One sequence and 128 / L channels per block, L threads of S states per channel.
template <typename T, int L, bool OUT>
__global__ void __launch_bounds__(NTHREADS) ssm_fwd_kernel(Params p) {
  constexpr int CH = NTHREADS / L, NP = L * S;
  __shared__ float2 s_d[TT][CH];
  __shared__ __align__(16) float s_b[TT][NP], s_c[TT][NP];
  __shared__ float s_y[TT][CH];
  const int tid = threadIdx.x, q = tid % L, ch = tid / L;
  const int seq = blockIdx.y;
  const int group = blockIdx.x / p.blocks_per_group, cg = p.C / p.G;
  const int c0 = group * cg + (blockIdx.x % p.blocks_per_group) * CH, c_end = min(c0 + CH, (group + 1) * cg);
  if (blockIdx.x == 0 && tid == 0) check_packing(p.cu, seq, p.T);
  const int64_t start = bound(p.cu, seq, p.T), end = bound(p.cu, seq + 1, p.T);
  const T* u = static_cast<const T*>(p.u);
  const T* dt = static_cast<const T*>(p.dt);
  const T* z = static_cast<const T*>(p.z);
  const T* bb = static_cast<const T*>(p.b) + group * p.b_sg;
  const T* cc = static_cast<const T*>(p.c) + group * p.c_sg;
  const bool live = c0 + ch < c_end;
  float a[S], h[S];
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const int n = q * S + i;
    const int64_t at = static_cast<int64_t>(c0 + ch) * p.N + n;
    a[i] = live && n < p.N ? p.A[at] * kLog2e : 0.f;
    h[i] = live && n < p.N && p.init ? p.init[static_cast<int64_t>(seq) * p.C * p.N + at] : 0.f;
  }
  int64_t tile = first_tile(start, seq);
  for (int64_t t0 = start; t0 < end; t0 += TT, ++tile) {
    const int nt = static_cast<int>(min(static_cast<int64_t>(TT), end - t0));
    __syncthreads();
    for (int i = tid; i < TT * CH; i += NTHREADS) {
      const int t = i / CH, k = i % CH;
      float2 v = make_float2(0.f, 0.f);
      if (t < nt && c0 + k < c_end) {
        const float r = to_f32(dt[(t0 + t) * p.dt_st + c0 + k]) + (p.dt_bias ? p.dt_bias[c0 + k] : 0.f);
        v.x = step_of(r, p.softplus);
        v.y = v.x * to_f32(u[(t0 + t) * p.u_st + c0 + k]);
      }
      s_d[t][k] = v;
    }
    for (int i = tid; i < TT * NP; i += NTHREADS) {
      const int t = i / NP, n = i % NP;
      const bool in = t < nt && n < p.N;
      s_b[t][n] = in ? to_f32(bb[(t0 + t) * p.b_st + n]) : 0.f;
      if (OUT) s_c[t][n] = in ? to_f32(cc[(t0 + t) * p.c_st + n]) : 0.f;
    }
    __syncthreads();
    if (!OUT && live) {
#pragma unroll
      for (int i = 0; i < S; ++i)
        if (q * S + i < p.N) p.ck[(tile * p.C + c0 + ch) * p.N + q * S + i] = h[i];
    }
    for (int t = 0; t < nt; ++t) {
      const float2 d = s_d[t][ch];
      const float4 b4 = *reinterpret_cast<const float4*>(&s_b[t][q * S]);
      const float bv[S] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
      for (int i = 0; i < S; ++i) h[i] = fmaf(exp2_approx(d.x * a[i]), h[i], d.y * bv[i]);
      if (OUT) {
        const float4 c4 = *reinterpret_cast<const float4*>(&s_c[t][q * S]);
        float y = c4.x * h[0];
        y = fmaf(c4.y, h[1], y);
        y = fmaf(c4.z, h[2], y);
        y = fmaf(c4.w, h[3], y);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (q == 0) s_y[t][ch] = y;
      }
    }
    if (OUT) {
      __syncthreads();
      for (int i = tid; i < nt * CH; i += NTHREADS) {
        const int t = i / CH, k = i % CH;
        if (c0 + k >= c_end) continue;
        float y = s_y[t][k];
        if (p.D) y = fmaf(p.D[c0 + k], to_f32(u[(t0 + t) * p.u_st + c0 + k]), y);
        if (z) y *= silu(to_f32(z[(t0 + t) * p.z_st + c0 + k]));
        static_cast<T*>(p.out)[(t0 + t) * p.o_st + c0 + k] = from_f32<T>(y);
      }
    }
  }
  if (p.fin && live) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int n = q * S + i;
      if (n < p.N) p.fin[(static_cast<int64_t>(seq) * p.C + c0 + ch) * p.N + n] = h[i];
    }
  }
}

// ------------------------------------------------------------ single tokens
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
};

// One block: 128 / L channels of one request.
template <typename T, int L>
__global__ void __launch_bounds__(NTHREADS) ssm_decode_kernel(DecodeParams p) {
  constexpr int CH = NTHREADS / L;
  const int64_t r = blockIdx.x;
  const int q = threadIdx.x % L, ch = blockIdx.y * CH + threadIdx.x / L;
  int64_t slot = r;
  if (p.idx) {
    slot = p.idx[r];
    if (slot < 0 || slot >= p.pool) {
      if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(&g_device_flags, KDA_DEVICE_BAD_STATE_INDEX);
      return;
    }
  }
  const bool live = ch < p.C;
  float y = 0.f, uu = 0.f;
  if (live) {
    const int group = ch / (p.C / p.G);
    uu = to_f32(static_cast<const T*>(p.u)[r * p.u_st + ch]);
    const float d = step_of(to_f32(static_cast<const T*>(p.dt)[r * p.dt_st + ch]) + (p.dt_bias ? p.dt_bias[ch] : 0.f),
                            p.softplus);
    const T* bb = static_cast<const T*>(p.b) + r * p.b_st + group * p.b_sg;
    const T* cc = static_cast<const T*>(p.c) + r * p.c_st + group * p.c_sg;
    float* st = p.state + (slot * p.C + ch) * p.N;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int n = q * S + i;
      if (n >= p.N) continue;
      const float h = fmaf(exp2_approx(d * (p.A[static_cast<int64_t>(ch) * p.N + n] * kLog2e)), st[n],
                           d * uu * to_f32(bb[n]));
      st[n] = h;
      y = fmaf(to_f32(cc[n]), h, y);
    }
  }
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
  if (live && q == 0) {
    if (p.D) y = fmaf(p.D[ch], uu, y);
    if (p.z) y *= silu(to_f32(static_cast<const T*>(p.z)[r * p.z_st + ch]));
    static_cast<T*>(p.out)[r * p.o_st + ch] = from_f32<T>(y);
  }
}

// ---------------------------------------------------------------- backward
struct BwdParams {
  Params f;                 // the forward's inputs; ck filled by its states-only pass
  const void* dout;
  const float* dfin;        // [NS, C, N] or null: zeros
  void* du;
  void* ddt;
  void* dz;                 // with z
  float* dinit;             // [NS, C, N] or null
  float* part_a;            // [NS, C, N]
  float* part_d;            // [2, NS, C]: dD, ddt_bias
  float* part_b;            // [channel blocks, T, N]
  float* part_c;
  int64_t dout_st, du_st, ddt_st, dz_st;
};

template <int L>
struct BwdShared {
  float4 d[TT][NTHREADS / L];  // d, d u, dy (through the gate), u
  float b[TT][L * S], c[TT][L * S];
  float y[TT][NTHREADS / L], sum1[TT][NTHREADS / L], sum2[TT][NTHREADS / L];
  float db[NTHREADS / 32][TT][L * S], dc[NTHREADS / 32][TT][L * S];  // each warp's
};

// The sequence backwards, a tile at a time: from the state kept before the
// tile its states and decays again (in registers), then the reverse recurrence
//   g_t = dy_t C_t + a_{t+1} g_{t+1},  q_t = a_t g_t h_{t-1}
//   dC += dy h,  dB += g d u,  ds = sum_n q A + u sum_n g B,  du = d sum_n g B + D dy,  dA += d q
template <typename T, int L>
__global__ void __launch_bounds__(NTHREADS) ssm_bwd_kernel(BwdParams bp) {
  const Params& p = bp.f;
  constexpr int CH = NTHREADS / L;
  extern __shared__ __align__(16) unsigned char smem[];
  BwdShared<L>& sm = *reinterpret_cast<BwdShared<L>*>(smem);
  auto& s_d = sm.d;
  auto& s_b = sm.b;
  auto& s_c = sm.c;
  auto& s_y = sm.y;
  auto& s_1 = sm.sum1;
  auto& s_2 = sm.sum2;
  auto& s_db = sm.db;
  auto& s_dc = sm.dc;
  constexpr int NP = L * S;
  const int tid = threadIdx.x, q = tid % L, ch = tid / L, warp = tid / 32, lane = tid % 32;
  const int seq = blockIdx.y;
  const int group = blockIdx.x / p.blocks_per_group, cg = p.C / p.G;
  const int c0 = group * cg + (blockIdx.x % p.blocks_per_group) * CH, c_end = min(c0 + CH, (group + 1) * cg);
  const int64_t start = bound(p.cu, seq, p.T), end = max(start, bound(p.cu, seq + 1, p.T));
  const T* u = static_cast<const T*>(p.u);
  const T* dt = static_cast<const T*>(p.dt);
  const T* z = static_cast<const T*>(p.z);
  const T* bb = static_cast<const T*>(p.b) + group * p.b_sg;
  const T* cc = static_cast<const T*>(p.c) + group * p.c_sg;
  const T* dout = static_cast<const T*>(bp.dout);
  const bool live = c0 + ch < c_end;
  float a[S], g[S], da[S] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const int n = q * S + i;
    const int64_t at = static_cast<int64_t>(c0 + ch) * p.N + n;
    a[i] = live && n < p.N ? p.A[at] : 0.f;
    g[i] = live && n < p.N && bp.dfin ? bp.dfin[static_cast<int64_t>(seq) * p.C * p.N + at] : 0.f;
  }
  float sum_d = 0.f, sum_bias = 0.f;  // thread tid < CH: channel c0 + tid
  const int64_t tiles = (end - start + TT - 1) / TT;
  for (int64_t k = tiles - 1; k >= 0; --k) {
    const int64_t t0 = start + k * TT;
    const int nt = static_cast<int>(min(static_cast<int64_t>(TT), end - t0));
    __syncthreads();
    for (int i = tid; i < TT * CH; i += NTHREADS) {
      const int t = i / CH, m = i % CH;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (t < nt && c0 + m < c_end) {
        const float r = to_f32(dt[(t0 + t) * p.dt_st + c0 + m]) + (p.dt_bias ? p.dt_bias[c0 + m] : 0.f);
        v.x = step_of(r, p.softplus);
        v.w = to_f32(u[(t0 + t) * p.u_st + c0 + m]);
        v.y = v.x * v.w;
        v.z = to_f32(dout[(t0 + t) * bp.dout_st + c0 + m]);
        if (z) v.z *= silu(to_f32(z[(t0 + t) * p.z_st + c0 + m]));
      }
      s_d[t][m] = v;
    }
    for (int i = tid; i < TT * NP; i += NTHREADS) {
      const int t = i / NP, n = i % NP;
      const bool in = t < nt && n < p.N;
      s_b[t][n] = in ? to_f32(bb[(t0 + t) * p.b_st + n]) : 0.f;
      s_c[t][n] = in ? to_f32(cc[(t0 + t) * p.c_st + n]) : 0.f;
    }
    __syncthreads();
    float h0[S], e[TT][S], h[TT][S];
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int n = q * S + i;
      h0[i] = live && n < p.N ? p.ck[((first_tile(start, seq) + k) * p.C + c0 + ch) * p.N + n] : 0.f;
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {  // past the sequence's end d = 0: the state stays
      const float4 d = s_d[t][ch];
      float y = 0.f;
#pragma unroll
      for (int i = 0; i < S; ++i) {
        e[t][i] = exp2_approx(d.x * (a[i] * kLog2e));
        h[t][i] = fmaf(e[t][i], t ? h[t - 1][i] : h0[i], d.y * s_b[t][q * S + i]);
        y = fmaf(s_c[t][q * S + i], h[t][i], y);
      }
      if (z) {
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (q == 0) s_y[t][ch] = y;
      }
    }
#pragma unroll
    for (int t = TT - 1; t >= 0; --t) {
      const float4 d = s_d[t][ch];
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const int n = q * S + i;
        g[i] = fmaf(d.z, s_c[t][n], g[i]);
        float vc = d.z * h[t][i], vb = d.y * g[i];
        s1 = fmaf(g[i], s_b[t][n], s1);
        g[i] *= e[t][i];
        const float w = g[i] * (t ? h[t - 1][i] : h0[i]);
        s2 = fmaf(w, a[i], s2);
        da[i] = fmaf(w, d.x, da[i]);
        // over the warp's channels
#pragma unroll
        for (int o = L; o < 32; o <<= 1) {
          vc += __shfl_xor_sync(0xffffffffu, vc, o);
          vb += __shfl_xor_sync(0xffffffffu, vb, o);
        }
        if (lane < L) {
          s_db[warp][t][n] = vb;
          s_dc[warp][t][n] = vc;
        }
      }
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) {
        s1 += __shfl_xor_sync(0xffffffffu, s1, o);
        s2 += __shfl_xor_sync(0xffffffffu, s2, o);
      }
      if (q == 0) {
        s_1[t][ch] = s1;
        s_2[t][ch] = s2;
      }
    }
    __syncthreads();
    for (int i = tid; i < nt * p.N; i += NTHREADS) {
      const int t = i / p.N, n = i % p.N;
      float vb = 0.f, vc = 0.f;
#pragma unroll
      for (int w = 0; w < NTHREADS / 32; ++w) {
        vb += s_db[w][t][n];
        vc += s_dc[w][t][n];
      }
      const int64_t at = (static_cast<int64_t>(blockIdx.x) * p.T + t0 + t) * p.N + n;
      bp.part_b[at] = vb;
      bp.part_c[at] = vc;
    }
    if (tid < CH && c0 + tid < c_end) {
      const int c = c0 + tid;
      const float bias = p.dt_bias ? p.dt_bias[c] : 0.f, D = p.D ? p.D[c] : 0.f;
      for (int t = nt - 1; t >= 0; --t) {
        const float4 d = s_d[t][tid];
        float dd = fmaf(d.w, s_1[t][tid], s_2[t][tid]);
        if (p.softplus) dd *= sigmoid(to_f32(dt[(t0 + t) * p.dt_st + c]) + bias);
        sum_bias += dd;
        sum_d = fmaf(d.z, d.w, sum_d);
        static_cast<T*>(bp.ddt)[(t0 + t) * bp.ddt_st + c] = from_f32<T>(dd);
        static_cast<T*>(bp.du)[(t0 + t) * bp.du_st + c] = from_f32<T>(fmaf(d.x, s_1[t][tid], D * d.z));
        if (z)
          static_cast<T*>(bp.dz)[(t0 + t) * bp.dz_st + c] =
              from_f32<T>(to_f32(dout[(t0 + t) * bp.dout_st + c]) * fmaf(D, d.w, s_y[t][tid]) *
                          dsilu(to_f32(z[(t0 + t) * p.z_st + c])));
      }
    }
  }
  if (live) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int n = q * S + i;
      if (n >= p.N) continue;
      const int64_t at = (static_cast<int64_t>(seq) * p.C + c0 + ch) * p.N + n;
      bp.part_a[at] = da[i];
      if (bp.dinit) bp.dinit[at] = g[i];
    }
  }
  if (tid < CH && c0 + tid < c_end) {
    bp.part_d[static_cast<int64_t>(seq) * p.C + c0 + tid] = sum_d;
    bp.part_d[(static_cast<int64_t>(p.NS) + seq) * p.C + c0 + tid] = sum_bias;
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
  int NS, C, N, G, blocks_per_group;
};

// Sums over the sequences (dA, dD, ddt_bias) and the channel blocks of a group
// (dB, dC), in order; zeros at tokens of no sequence.
template <typename T>
__global__ void __launch_bounds__(256) ssm_reduce_kernel(ReduceParams p) {
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, stride = static_cast<int64_t>(gridDim.x) * 256;
  const int64_t cn = static_cast<int64_t>(p.C) * p.N;
  for (int64_t i = i0; i < cn; i += stride) {
    float a = 0.f;
    for (int s = 0; s < p.NS; ++s) a += p.part_a[s * cn + i];
    p.dA[i] = a;
  }
  for (int64_t i = i0; i < 2 * static_cast<int64_t>(p.C); i += stride) {
    float* to = i < p.C ? p.dD : p.ddt_bias;
    if (!to) continue;
    const int64_t c = i < p.C ? i : i - p.C;
    float a = 0.f;
    for (int s = 0; s < p.NS; ++s) a += p.part_d[((i < p.C ? 0 : static_cast<int64_t>(p.NS)) + s) * p.C + c];
    to[c] = a;
  }
  const int64_t lo = bound(p.cu, 0, p.T), hi = bound(p.cu, p.cu ? p.NS : 1, p.T);
  const int64_t gn = static_cast<int64_t>(p.G) * p.N;
  for (int64_t i = i0; i < p.T * gn; i += stride) {
    const int64_t t = i / gn;
    const int g = static_cast<int>(i % gn / p.N), n = static_cast<int>(i % p.N);
    float vb = 0.f, vc = 0.f;
    if (t >= lo && t < hi) {
      for (int k = 0; k < p.blocks_per_group; ++k) {
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
