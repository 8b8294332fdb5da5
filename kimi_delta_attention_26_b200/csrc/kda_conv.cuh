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
// takes 32 x V channels (V = 8 bytes of them where strides and addresses allow,
// else 1) of a run of tokens, carries the last inputs in registers and loads four
// tokens while it computes four.
// All arithmetic is fp32; the outputs are rounded once.
//
// Measured (bf16, 4 taps, SiLU): 18264 tokens x 12288 channels 175 us (5.1 TB/s,
// 78 % of the copy rate; 16-byte accesses, 183 to 231 registers: 284 us), the
// gradients of 8192 tokens 150 + 5 us (4.0 TB/s; two channels a thread: 190 us),
// one token of 256 requests 10 us (4.9 TB/s). fp32: 8192 tokens 143 us (5.6
// TB/s; bf16 88), their gradients 241, one token of 256 requests 14.2 us (7.1 TB/s,
// part of it from L2).
#pragma once

#include <type_traits>

#include "kda_io.cuh"

namespace kda {
namespace conv {

constexpr int NTHREADS = 128;
constexpr int NWARPS = NTHREADS / 32;
constexpr int RUN_BYTES = 8;  // of a row per access, prompts and gradients

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

// The weights of V channels, by tap. W = 4 comes as 16 bytes a channel where
// the address allows.
template <int V, int W>
__device__ __forceinline__ void load_weights(float (&w)[W][V], float (&b)[V], const float* weight, const float* bias,
                                             int64_t c) {
  const bool wide = W == 4 && reinterpret_cast<uintptr_t>(weight) % 16 == 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (wide) {
      const float4 v = *reinterpret_cast<const float4*>(weight + (c + i) * W);
      const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][i] = x[j];
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][i] = weight[(c + i) * W + j];
    }
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

// acc += x * y, in pairs where there are any
template <int V>
__device__ __forceinline__ void fma_to(float (&acc)[V], const float (&x)[V], const float (&y)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 r = __ffma2_rn(make_float2(x[i], x[i + 1]), make_float2(y[i], y[i + 1]), make_float2(acc[i], acc[i + 1]));
      acc[i] = r.x;
      acc[i + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = fmaf(x[i], y[i], acc[i]);
  }
}

// the activation of a row, and dp = dy act'(a)
template <int V>
__device__ __forceinline__ void activate(float (&a)[V], int act) {
  if (!act) return;
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 y = psilu(make_float2(a[i], a[i + 1]));
      a[i] = y.x;
      a[i + 1] = y.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = silu(a[i]);
  }
}

template <int V>
__device__ __forceinline__ void pre_gradient(float (&dp)[V], const float (&dy)[V], const float (&a)[V], int act) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      float2 g = make_float2(dy[i], dy[i + 1]);
      if (act) g = __fmul2_rn(g, pdsilu(make_float2(a[i], a[i + 1])));
      dp[i] = g.x;
      dp[i + 1] = g.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) dp[i] = act ? dy[i] * dsilu(a[i]) : dy[i];
  }
}

constexpr int KT = 4;  // tokens loaded together; the last inputs are a ring of KT rows, row t % KT

template <typename T, int V, int W>
__global__ void __launch_bounds__(NTHREADS) conv_fwd_kernel(Params p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * 32 + lane) * V;
  const T* init = static_cast<const T*>(p.init);
  if (blockIdx.x >= p.run_blocks) {  // the sequences' states
    const T* x = static_cast<const T*>(p.x);
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
  for (int64_t pos = r0; s < p.N && pos < r1; ++s) {
    const int64_t start = bound(p.cu, s, p.T), lo = max(start, pos), hi = min(bound(p.cu, s + 1, p.T), r1);
    if (hi <= lo) continue;
    pos = hi;
    const T* x = static_cast<const T*>(p.x) + c + lo * p.x_st;  // the next token to load
    T* out = static_cast<T*>(p.out) + c + lo * p.o_st;
    float ring[KT][V];
#pragma unroll
    for (int i = 1; i < W; ++i)
      load_position<T, V, W>(ring[KT - i], static_cast<const T*>(p.x), p.x_st, init, p.C, c, s, start, lo - i);
    Vec<T, V> next[KT];
    int left = static_cast<int>(hi - lo);  // tokens not yet loaded
    auto fetch = [&] {
      if (left >= KT) {
#pragma unroll
        for (int k = 0; k < KT; ++k) next[k].load(x + k * p.x_st);
      } else {
#pragma unroll
        for (int k = 0; k < KT; ++k)
          if (k < left) next[k].load(x + k * p.x_st);
      }
      x += KT * p.x_st;
      left -= KT;
    };
    auto token = [&](int k) {
      float a[V];
#pragma unroll
      for (int i = 0; i < V; ++i) a[i] = b[i];
#pragma unroll
      for (int j = 0; j < W; ++j) fma_to<V>(a, w[j], ring[(k + KT - (W - 1) + j) % KT]);
      activate<V>(a, p.silu);
      store_f32<T, V>(out + k * p.o_st, a);
    };
    fetch();
    for (int todo = static_cast<int>(hi - lo); todo > 0; todo -= KT) {
      Vec<T, V> now[KT];
#pragma unroll
      for (int k = 0; k < KT; ++k) now[k] = next[k];
      if (left > 0) fetch();
      if (todo >= KT) {
#pragma unroll
        for (int k = 0; k < KT; ++k) {
          now[k].get(ring[k]);
          token(k);
        }
      } else {
#pragma unroll
        for (int k = 0; k < KT; ++k)
          if (k < todo) {
            now[k].get(ring[k]);
            token(k);
          }
      }
      out += KT * p.o_st;
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

// One thread: V channels of every gridDim.y-th request, so that several requests
// share one load of the weights. It reads the W - 1 kept inputs and the token
// before it writes any of them back, so out may be x itself.
template <typename T, int V, int W>
__global__ void __launch_bounds__(NTHREADS) conv_decode_kernel(DecodeParams p) {
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * NTHREADS + threadIdx.x) * V;
  if (c >= p.C) return;
  float w[W][V], bias[V];
  load_weights<V, W>(w, bias, p.weight, p.bias, c);
  // the next request's rows are loaded before this one's arithmetic
  Vec<T, V> next[W];
  int64_t next_slot = -1;
  auto fetch = [&](int64_t b) {
    next_slot = p.idx ? p.idx[b] : b;
    if (next_slot < 0 || next_slot >= p.pool) {  // uniform over the block
      if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(&g_device_flags, KDA_DEVICE_BAD_STATE_INDEX);
      next_slot = -1;
      return;
    }
    const T* st = static_cast<const T*>(p.state) + next_slot * (W - 1) * p.C + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) next[j].load(st + j * p.C);
    next[W - 1].load(static_cast<const T*>(p.x) + b * p.x_st + c);
  };
  fetch(blockIdx.y);
  for (int64_t b = blockIdx.y; b < p.B; b += gridDim.y) {
    const int64_t slot = next_slot;
    Vec<T, V> raw[W];
#pragma unroll
    for (int j = 0; j < W; ++j) raw[j] = next[j];
    if (b + gridDim.y < p.B) fetch(b + gridDim.y);
    if (slot < 0) continue;
    T* st = static_cast<T*>(p.state) + slot * (W - 1) * p.C + c;
    float y[V];
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = bias[i];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      float x[V];
      raw[j].get(x);
      fma_to<V>(y, w[j], x);
    }
    activate<V>(y, p.silu);
    store_f32<T, V>(static_cast<T*>(p.out) + b * p.o_st + c, y);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) raw[j + 1].store(st + j * p.C);
  }
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

// A warp walks its run of tokens forwards: at token t it has the inputs
// t - W + 1 .. t and the last W - 1 values of dp, so dx_{t-W+1} is complete. It
// goes W - 1 tokens past its run (or past the sequence's end, with dp = 0) for
// the last dx; those tokens add nothing to its sums for dw and dbias.
template <typename T, int V, int W>
__global__ void __launch_bounds__(NTHREADS) conv_bwd_kernel(BwdParams p) {
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
      float dy[V], dp[V], a[V];
      load_f32<T, V>(dy, dout + (start + k) * p.d_st + c);
#pragma unroll
      for (int v = 0; v < V; ++v) a[v] = b[v];
#pragma unroll
      for (int j = 0; j < W; ++j) fma_to<V>(a, w[j], win[k + j]);
      pre_gradient<V>(dp, dy, a, p.silu);
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
    load_weights<V, W>(w, b, p.weight, p.bias, c);
    const float zero[V] = {};
    int64_t pos = r0;
    auto clear = [&](int64_t to) {  // tokens of no sequence
      for (; pos < to; ++pos) store_f32<T, V>(static_cast<T*>(p.dx) + pos * p.g_st + c, zero);
    };
    for (; s < p.N && pos < r1; ++s) {
      const int64_t start = bound(p.cu, s, p.T), end = bound(p.cu, s + 1, p.T);
      const int64_t lo = max(start, pos), hi = min(end, r1);
      if (hi <= lo) continue;
      clear(lo);
      pos = hi;
      // rings of the last inputs and of their dp; 0 before lo: no dx there is this warp's
      float ring[KT][V], dp[KT][V];
#pragma unroll
      for (int i = 1; i < W; ++i)
        load_position<T, V, W>(ring[KT - i], x, p.x_st, init, p.C, c, s, start, lo - i);
#pragma unroll
      for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) dp[k][v] = 0.f;
      const int own = static_cast<int>(hi - lo);                              // tokens of the run
      const int real = own + static_cast<int>(min(end - hi, static_cast<int64_t>(W - 1)));  // and those seen past it
      const T* xp = x + c + lo * p.x_st;
      const T* yp = dout + c + lo * p.d_st;
      T* dx = static_cast<T*>(p.dx) + c + (lo - (W - 1)) * p.g_st;  // dx of the first token's oldest input
      const int to_final = static_cast<int>(min(end - lo, static_cast<int64_t>(INT32_MAX)));  // token lo + to_final is the end
      Vec<T, V> nx[KT], ny[KT];
      int left = real;
      auto fetch = [&] {
        if (left >= KT) {
#pragma unroll
          for (int k = 0; k < KT; ++k) {
            nx[k].load(xp + k * p.x_st);
            ny[k].load(yp + k * p.d_st);
          }
        } else {
#pragma unroll
          for (int k = 0; k < KT; ++k)
            if (k < left) {
              nx[k].load(xp + k * p.x_st);
              ny[k].load(yp + k * p.d_st);
            }
        }
        xp += KT * p.x_st;
        yp += KT * p.d_st;
        left -= KT;
      };
      fetch();
      for (int t = 0; t < own + W - 1; t += KT) {
        Vec<T, V> cx[KT], cy[KT];
#pragma unroll
        for (int k = 0; k < KT; ++k) {
          cx[k] = nx[k];
          cy[k] = ny[k];
        }
        if (left > 0) fetch();
        // FULL: four tokens of the run whose dx are tokens of the run too, none of them in the final state
        auto step = [&](int k, auto full) {
          if (full.value || t + k < real) {
            float dy[V], a[V];
            cx[k].get(ring[k]);
            cy[k].get(dy);
#pragma unroll
            for (int v = 0; v < V; ++v) a[v] = b[v];
#pragma unroll
            for (int j = 0; j < W; ++j) fma_to<V>(a, w[j], ring[(k + KT - (W - 1) + j) % KT]);
            pre_gradient<V>(dp[k], dy, a, p.silu);
            if (full.value || t + k < own) {
#pragma unroll
              for (int v = 0; v < V; ++v) db[v] += dp[k][v];
#pragma unroll
              for (int j = 0; j < W; ++j) fma_to<V>(dw[j], dp[k], ring[(k + KT - (W - 1) + j) % KT]);
            }
          } else {
#pragma unroll
            for (int v = 0; v < V; ++v) dp[k][v] = 0.f;
          }
          const int at = t + k - (W - 1);  // the token whose dx is complete, from lo
          if (full.value || (at >= 0 && at < own)) {
            float g[V];
#pragma unroll
            for (int v = 0; v < V; ++v) g[v] = 0.f;
            const int row = at - (to_final - (W - 1));
            if (!full.value && dfin && row >= 0)
              load_f32<T, V>(g, dfin + (static_cast<int64_t>(s) * (W - 1) + row) * p.C + c);
#pragma unroll
            for (int j = 0; j < W; ++j) fma_to<V>(g, w[j], dp[(k + KT - j) % KT]);
            store_f32<T, V>(dx + k * p.g_st, g);
          }
        };
        if (t >= W - 1 && t + KT <= own && t + KT <= to_final - (W - 1)) {
#pragma unroll
          for (int k = 0; k < KT; ++k) step(k, std::true_type());
        } else {
#pragma unroll
          for (int k = 0; k < KT; ++k) step(k, std::false_type());
        }
        dx += KT * p.g_st;
      }
    }
    clear(r1);
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
