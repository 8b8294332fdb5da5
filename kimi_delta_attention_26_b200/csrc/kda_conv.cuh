// kda_conv.cuh -- the short causal depthwise convolution in front of the
// recurrences, for packed sequences, for training and for single tokens.
//
// Per channel c, with W taps (2 to 4) and the sequence's inputs continued
// backwards by its state (the W - 1 inputs before its first token, oldest first):
//   p_t = bias + sum_j w_j x_{t-W+1+j},   y_t = p_t  or  p_t sigmoid(p_t)
// and for a gradient dy of y:
//   dp_t = dy_t act'(p_t),  dx_s = sum_j w_j dp_{s+W-1-j},
//   dw_j = sum_t dp_t x_{t-W+1+j},  dbias = sum_t dp_t
// (dp is 0 outside the sequence; the gradient of the state is dx at the
// positions before the first token).
//
// Each input is read once and each output written once: bound by HBM. A warp
// takes 32 x V channels (V = 16 bytes of them where strides and addresses
// allow, else 1) of a run of tokens and carries the last inputs in registers.
// All arithmetic is fp32; the outputs are rounded once.
#pragma once

#include "kda_io.cuh"

namespace kda {
namespace conv {

constexpr int NTHREADS = 128;
constexpr int NWARPS = NTHREADS / 32;

struct Params {
  const void* x;
  const float* weight;      // [C, W]
  const float* bias;        // [C] or null
  const int32_t* cu;        // [N + 1] or null: one sequence
  const void* init;         // [N, W - 1, C] or null: zeros
  void* out;
  void* fin;                // [N, W - 1, C] or null
  int64_t T, C, x_st, o_st;
  int64_t run;              // tokens per warp
  int64_t run_blocks;       // blocks that take runs; the blocks after them take the sequences' states
  int N;
  int silu;
};

template <int V, int W>
__device__ __forceinline__ void load_weights(float (&w)[W][V], float (&b)[V], const float* weight, const float* bias,
                                             int64_t c) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][i] = weight[(c + i) * W + j];
    b[i] = bias ? bias[c + i] : 0.f;
  }
}

// Position `pos` of sequence `seq` (first token `start`): a token, a row of
// the state before it, or 0.
template <typename T, int V, int W>
__device__ __forceinline__ void load_position(float (&x)[V], const T* x_base, int64_t x_st, const T* init, int64_t C,
                                              int64_t c, int seq, int64_t start, int64_t pos) {
  if (pos >= start) {
    load_f32<T, V>(x, x_base + pos * x_st + c);
  } else if (init) {
    load_f32<T, V>(x, init + (static_cast<int64_t>(seq) * (W - 1) + (pos - start + W - 1)) * C + c);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = 0.f;
  }
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(NTHREADS) conv_fwd_kernel(Params p) {
  constexpr int KT = 8;  // tokens loaded together
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * 32 + lane) * V;
  const T* x = static_cast<const T*>(p.x);
  const T* init = static_cast<const T*>(p.init);
  if (blockIdx.x >= p.run_blocks) {  // the sequences' states
    const int64_t s = (blockIdx.x - p.run_blocks) * NWARPS + warp;
    if (s >= p.N) return;
    if (blockIdx.y == 0 && lane == 0) check_packing(p.cu, static_cast<int>(s), p.T);
    if (!p.fin || c >= p.C) return;
    const int64_t start = bound(p.cu, static_cast<int>(s), p.T);
    const int64_t end = max(start, bound(p.cu, static_cast<int>(s) + 1, p.T));
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      float r[V];
      load_position<T, V, W>(r, x, p.x_st, init, p.C, c, static_cast<int>(s), start, end - (W - 1) + i);
      store_f32<T, V>(static_cast<T*>(p.fin) + (s * (W - 1) + i) * p.C + c, r);
    }
    return;
  }
  const int64_t r0 = (static_cast<int64_t>(blockIdx.x) * NWARPS + warp) * p.run;
  const int64_t r1 = min(r0 + p.run, p.T);
  if (r0 >= p.T) return;
  int s = first_sequence(p.cu, p.N, r0);
  if (c >= p.C) return;
  float w[W][V], b[V];
  load_weights<V, W>(w, b, p.weight, p.bias, c);
  T* out = static_cast<T*>(p.out);
  for (int64_t pos = r0; s < p.N && pos < r1; ++s) {
    const int64_t start = bound(p.cu, s, p.T), lo = max(start, pos), hi = min(bound(p.cu, s + 1, p.T), r1);
    if (hi <= lo) continue;
    pos = hi;
    float win[W + KT - 1][V];  // inputs t - W + 1 .. t + KT - 1
#pragma unroll
    for (int i = 0; i < W - 1; ++i)
      load_position<T, V, W>(win[i], x, p.x_st, init, p.C, c, s, start, lo - (W - 1) + i);
    for (int64_t t = lo; t < hi; t += KT) {
      Vec<T, V> raw[KT];
#pragma unroll
      for (int k = 0; k < KT; ++k)
        if (t + k < hi) raw[k].load(x + (t + k) * p.x_st + c);
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        if (t + k >= hi) break;
        float y[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          win[W - 1 + k][i] = raw[k].get(i);
          float a = b[i];
#pragma unroll
          for (int j = 0; j < W; ++j) a = fmaf(w[j][i], win[k + j][i], a);
          y[i] = p.silu ? silu(a) : a;
        }
        store_f32<T, V>(out + (t + k) * p.o_st + c, y);
      }
#pragma unroll
      for (int i = 0; i < W - 1; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) win[i][v] = win[KT + i][v];
    }
  }
}

// ------------------------------------------------------------ single tokens
struct DecodeParams {
  const void* x;
  const float* weight;
  const float* bias;
  void* state;              // [P, W - 1, C]
  const int32_t* idx;       // [B] or null: slot b
  void* out;
  int64_t B, C, x_st, o_st, pool;
  int silu;
};

// One thread: V channels of one request. It reads the W - 1 kept inputs and
// the token before it writes any of them back, so out may be x itself.
template <typename T, int V, int W>
__global__ void __launch_bounds__(NTHREADS) conv_decode_kernel(DecodeParams p) {
  const int64_t b = blockIdx.x;
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * NTHREADS + threadIdx.x) * V;
  int64_t slot = b;
  if (p.idx) {
    slot = p.idx[b];
    if (slot < 0 || slot >= p.pool) {
      if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(&g_device_flags, KDA_DEVICE_BAD_STATE_INDEX);
      return;
    }
  }
  if (c >= p.C) return;
  T* st = static_cast<T*>(p.state) + slot * (W - 1) * p.C + c;
  Vec<T, V> raw[W];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) raw[j].load(st + j * p.C);
  raw[W - 1].load(static_cast<const T*>(p.x) + b * p.x_st + c);
  float w[W][V], y[V];
  load_weights<V, W>(w, y, p.weight, p.bias, c);
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int j = 0; j < W; ++j) y[i] = fmaf(w[j][i], raw[j].get(i), y[i]);
    if (p.silu) y[i] = silu(y[i]);
  }
  store_f32<T, V>(static_cast<T*>(p.out) + b * p.o_st + c, y);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) raw[j + 1].store(st + j * p.C);
}

// ---------------------------------------------------------------- backward
struct BwdParams {
  const void* x;
  const void* dout;
  const float* weight;
  const float* bias;
  const int32_t* cu;
  const void* init;
  const void* dfin;         // [N, W - 1, C] or null: zeros
  void* dx;
  void* dinit;              // [N, W - 1, C] or null
  float* part;              // [run_blocks, W + 1, C]: each block's sums for dw and dbias
  int64_t T, C, x_st, d_st, g_st;  // strides of x, dout, dx
  int64_t run, run_blocks;
  int N;
  int silu;
};

// dp at a token whose W inputs are win[0 .. W - 1]
template <int V, int W>
__device__ __forceinline__ void pre_gradient(float (&dp)[V], const float (&dy)[V], const float (*win)[V],
                                             const float (&w)[W][V], const float (&b)[V], int act) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    dp[i] = dy[i];
    if (act) {
      float a = b[i];
#pragma unroll
      for (int j = 0; j < W; ++j) a = fmaf(w[j][i], win[j][i], a);
      dp[i] *= dsilu(a);
    }
  }
}

// A warp walks its run of tokens forwards: at token t it has the inputs
// t - W + 1 .. t and the last W - 1 values of dp, so dx_{t-W+1} is complete. It
// goes W - 1 tokens past its run (or past the sequence's end, with dp = 0) for
// the last dx; those tokens add nothing to its sums for dw and dbias.
template <typename T, int V, int W>
__global__ void __launch_bounds__(NTHREADS) conv_bwd_kernel(BwdParams p) {
  constexpr int KT = 4;
  __shared__ float s_part[NWARPS][W + 1][32 * V];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * 32 + lane) * V;
  const T* x = static_cast<const T*>(p.x);
  const T* dout = static_cast<const T*>(p.dout);
  const T* init = static_cast<const T*>(p.init);
  const T* dfin = static_cast<const T*>(p.dfin);
  float w[W][V], b[V];
  if (blockIdx.x >= p.run_blocks) {  // the gradients of the initial states
    const int64_t s = (blockIdx.x - p.run_blocks) * NWARPS + warp;
    if (s >= p.N) return;
    const int seq = static_cast<int>(s);
    if (blockIdx.y == 0 && lane == 0) check_packing(p.cu, seq, p.T);
    if (!p.dinit || c >= p.C) return;
    load_weights<V, W>(w, b, p.weight, p.bias, c);
    const int64_t start = bound(p.cu, seq, p.T), end = max(start, bound(p.cu, seq + 1, p.T));
    float win[2 * W - 2][V], acc[W - 1][V];
#pragma unroll
    for (int i = 0; i < 2 * W - 2; ++i) {
      const int64_t pos = start - (W - 1) + i;
#pragma unroll
      for (int v = 0; v < V; ++v) win[i][v] = 0.f;
      if (pos < end) load_position<T, V, W>(win[i], x, p.x_st, init, p.C, c, seq, start, pos);
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      const int64_t row = start + i - end;  // the position's row in the final state
#pragma unroll
      for (int v = 0; v < V; ++v) acc[i][v] = 0.f;
      if (dfin && row >= 0) load_f32<T, V>(acc[i], dfin + (s * (W - 1) + row) * p.C + c);
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      if (start + k >= end) break;
      float dy[V], dp[V];
      load_f32<T, V>(dy, dout + (start + k) * p.d_st + c);
      pre_gradient<V, W>(dp, dy, &win[k], w, b, p.silu);
      // token start + k sees position start - (W - 1) + i by tap j = i - k
#pragma unroll
      for (int i = k; i < W - 1; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) acc[i][v] = fmaf(w[i - k][v], dp[v], acc[i][v]);
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i)
      store_f32<T, V>(static_cast<T*>(p.dinit) + (s * (W - 1) + i) * p.C + c, acc[i]);
    return;
  }
  const int64_t r0 = min((static_cast<int64_t>(blockIdx.x) * NWARPS + warp) * p.run, p.T);
  const int64_t r1 = min(r0 + p.run, p.T);
  int s = first_sequence(p.cu, p.N, r0);
  float dw[W][V], db[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    db[v] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][v] = 0.f;
  }
  if (c < p.C && r0 < r1) {
    T* dx = static_cast<T*>(p.dx);
    load_weights<V, W>(w, b, p.weight, p.bias, c);
    const float zero[V] = {};
    int64_t pos = r0;
    for (; s < p.N && pos < r1; ++s) {
      const int64_t start = bound(p.cu, s, p.T), end = bound(p.cu, s + 1, p.T);
      const int64_t lo = max(start, pos), hi = min(end, r1);
      if (hi <= lo) continue;
      for (; pos < lo; ++pos) store_f32<T, V>(dx + pos * p.g_st + c, zero);  // tokens of no sequence
      pos = hi;
      float win[W + KT - 1][V], dp[W + KT - 1][V];  // inputs t - W + 1 ..; dp of the same tokens
#pragma unroll
      for (int i = 0; i < W - 1; ++i) {
        load_position<T, V, W>(win[i], x, p.x_st, init, p.C, c, s, start, lo - (W - 1) + i);
#pragma unroll
        for (int v = 0; v < V; ++v) dp[i][v] = 0.f;
      }
      const int64_t stop = hi + W - 1;
      for (int64_t t = lo; t < stop; t += KT) {
        Vec<T, V> rx[KT], rd[KT];
#pragma unroll
        for (int k = 0; k < KT; ++k)
          if (t + k < stop && t + k < end) {
            rx[k].load(x + (t + k) * p.x_st + c);
            rd[k].load(dout + (t + k) * p.d_st + c);
          }
#pragma unroll
        for (int k = 0; k < KT; ++k) {
          if (t + k >= stop) break;
          float (&now)[V] = dp[W - 1 + k];
          if (t + k < end) {
            float dy[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
              win[W - 1 + k][v] = rx[k].get(v);
              dy[v] = rd[k].get(v);
            }
            pre_gradient<V, W>(now, dy, &win[k], w, b, p.silu);
            if (t + k < hi) {
#pragma unroll
              for (int v = 0; v < V; ++v) {
                db[v] += now[v];
#pragma unroll
                for (int j = 0; j < W; ++j) dw[j][v] = fmaf(now[v], win[k + j][v], dw[j][v]);
              }
            }
          } else {
#pragma unroll
            for (int v = 0; v < V; ++v) now[v] = 0.f;
          }
          const int64_t at = t + k - (W - 1);
          if (at >= lo) {
            float g[V];
            const int64_t row = at - (end - (W - 1));
#pragma unroll
            for (int v = 0; v < V; ++v) g[v] = 0.f;
            if (dfin && row >= 0) load_f32<T, V>(g, dfin + (static_cast<int64_t>(s) * (W - 1) + row) * p.C + c);
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
              for (int j = 0; j < W; ++j) g[v] = fmaf(w[j][v], dp[W - 1 + k - j][v], g[v]);
            store_f32<T, V>(dx + at * p.g_st + c, g);
          }
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
#pragma unroll
          for (int v = 0; v < V; ++v) {
            win[i][v] = win[KT + i][v];
            dp[i][v] = dp[KT + i][v];
          }
      }
    }
    for (; pos < r1; ++pos) store_f32<T, V>(dx + pos * p.g_st + c, zero);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int j = 0; j < W; ++j) s_part[warp][j][lane * V + v] = dw[j][v];
    s_part[warp][W][lane * V + v] = db[v];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < (W + 1) * 32 * V; i += NTHREADS) {
    const int j = i / (32 * V), k = i % (32 * V);
    const int64_t ch = static_cast<int64_t>(blockIdx.y) * 32 * V + k;
    if (ch >= p.C) continue;
    float a = 0.f;
#pragma unroll
    for (int q = 0; q < NWARPS; ++q) a += s_part[q][j][k];
    p.part[(static_cast<int64_t>(blockIdx.x) * (W + 1) + j) * p.C + ch] = a;
  }
}

// The blocks' sums in order: dw[c][j] and dbias[c].
static __global__ void __launch_bounds__(NTHREADS) conv_reduce_kernel(const float* part, int64_t blocks, int W, int64_t C,
                                                              float* dw, float* db) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * NTHREADS + threadIdx.x;
  const int j = blockIdx.y;
  if (c >= C) return;
  float a = 0.f;
  for (int64_t i = 0; i < blocks; ++i) a += part[(i * (W + 1) + j) * C + c];
  if (j < W) dw[c * W + j] = a;
  else if (db) db[c] = a;
}

}  // namespace conv
}  // namespace kda
