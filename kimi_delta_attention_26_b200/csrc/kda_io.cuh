// kda_io.cuh -- what the convolution and the scan share: loads and stores of
// bf16, fp16 and fp32 rows, the activations, and finding a token's sequence.
#pragma once

#include <cuda_fp16.h>

#include "kda_prims.cuh"

namespace kda {

// V consecutive elements of a row, moved as one access of 2, 4, 8 or 16 bytes.
// Held as 32-bit words: as 16-bit members the compiler moves them one by one.
template <int BYTES>
struct Words;
template <>
struct Words<2> { using type = uint16_t; };
template <>
struct Words<4> { using type = uint32_t; };
template <>
struct Words<8> { using type = uint2; };
template <>
struct Words<16> { using type = uint4; };

template <typename T>
__device__ __forceinline__ float lo_f32(uint32_t w);
template <typename T>
__device__ __forceinline__ float hi_f32(uint32_t w);
template <>
__device__ __forceinline__ float lo_f32<__nv_bfloat16>(uint32_t w) { return __uint_as_float(w << 16); }
template <>
__device__ __forceinline__ float hi_f32<__nv_bfloat16>(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
template <>
__device__ __forceinline__ float lo_f32<__half>(uint32_t w) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(w)));
}
template <>
__device__ __forceinline__ float hi_f32<__half>(uint32_t w) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(w >> 16)));
}
template <>
__device__ __forceinline__ float lo_f32<float>(uint32_t w) { return __uint_as_float(w); }

template <typename T>
__device__ __forceinline__ uint32_t pair_bits(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pair_bits<__nv_bfloat16>(float lo, float hi) { return pack_bf16(lo, hi); }
template <>
__device__ __forceinline__ uint32_t pair_bits<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}

template <typename T, int V>
struct Vec {
  static constexpr int BYTES = V * sizeof(T);
  using Raw = typename Words<BYTES>::type;
  Raw raw;

  __device__ __forceinline__ void load(const void* p) { raw = *static_cast<const Raw*>(p); }
  __device__ __forceinline__ void store(void* p) const { *static_cast<Raw*>(p) = raw; }
  __device__ __forceinline__ uint32_t word(int i) const {
    if constexpr (BYTES <= 4) return raw;
    else if constexpr (BYTES == 8) return i == 0 ? raw.x : raw.y;
    else return i == 0 ? raw.x : i == 1 ? raw.y : i == 2 ? raw.z : raw.w;
  }
  __device__ __forceinline__ void set_word(int i, uint32_t w) {
    if constexpr (BYTES <= 4) raw = static_cast<Raw>(w);
    else if constexpr (BYTES == 8) (i == 0 ? raw.x : raw.y) = w;
    else (i == 0 ? raw.x : i == 1 ? raw.y : i == 2 ? raw.z : raw.w) = w;
  }
  __device__ __forceinline__ float get(int i) const {  // i known at compile time
    if constexpr (sizeof(T) == 4) return __uint_as_float(word(i));
    else return i % 2 ? hi_f32<T>(word(i / 2)) : lo_f32<T>(word(i / 2));
  }
  __device__ __forceinline__ void get(float (&x)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = get(i);
  }
  __device__ __forceinline__ void set(const float (&x)[V]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) set_word(i, __float_as_uint(x[i]));
    } else if constexpr (V == 1) {
      set_word(0, pair_bits<T>(x[0], 0.f));
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 2) set_word(i / 2, pair_bits<T>(x[i], x[i + 1]));
    }
  }
  // the first `valid` elements one by one, zeros for the others
  __device__ __forceinline__ void load_some(const T* p, int valid) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) set_word(i, i < valid ? reinterpret_cast<const uint32_t*>(p)[i] : 0u);
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const uint32_t lo = i < valid ? h[i] : 0u, hi = i + 1 < valid && i + 1 < V ? h[i + 1] : 0u;
        set_word(i / 2, lo | hi << 16);
      }
    }
  }
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

template <typename T, int V>
__device__ __forceinline__ void load_f32(float (&x)[V], const T* p) {
  Vec<T, V> a;
  a.load(p);
  a.get(x);
}

template <typename T, int V>
__device__ __forceinline__ void store_f32(T* p, const float (&x)[V]) {
  Vec<T, V> a;
  a.set(x);
  a.store(p);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// Pairs are multiplied and added as one instruction: half the instructions, the
// same time on the multiply-add pipe.
__device__ __forceinline__ float2 pair_of(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 pexp2(float2 x) { return make_float2(exp2_approx(x.x), exp2_approx(x.y)); }
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 prcp(float2 x) { return make_float2(rcp_approx(x.x), rcp_approx(x.y)); }

// sigmoid of a pair; exp(-x) overflows to infinity for x below -88, whose
// reciprocal is the right 0
__device__ __forceinline__ float2 psigmoid(float2 x) {
  return prcp(__fadd2_rn(pair_of(1.f), pexp2(__fmul2_rn(x, pair_of(-kLog2e)))));
}

// x sigmoid(x)
__device__ __forceinline__ float2 psilu(float2 x) { return __fmul2_rn(x, psigmoid(x)); }
// and its derivative s (1 + x (1 - s)) with s = sigmoid(x)
__device__ __forceinline__ float2 pdsilu(float2 x) {
  const float2 s = psigmoid(x);
  return __ffma2_rn(__fmul2_rn(x, s), make_float2(1.f - s.x, 1.f - s.y), s);
}
__device__ __forceinline__ float sigmoid(float x) { return rcp_approx(1.f + exp2_approx(x * -kLog2e)); }
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }
__device__ __forceinline__ float dsilu(float x) {
  const float s = sigmoid(x);
  return fmaf(x * s, 1.f - s, s);
}

// Boundary i of a packed batch, clamped into [0, T]; without cu_seqlens the
// batch is one sequence.
__device__ __forceinline__ int64_t bound(const int32_t* cu, int i, int64_t T) {
  if (!cu) return i == 0 ? 0 : T;
  const int64_t x = cu[i];
  return x < 0 ? 0 : (x > T ? T : x);
}

// Records boundaries that are no packing: cu[0] = 0, non-decreasing, cu[N] <= T.
__device__ __forceinline__ void check_packing(const int32_t* cu, int seq, int64_t T) {
  if (!cu) return;
  const int64_t a = cu[seq], b = cu[seq + 1];
  if (a < 0 || b < a || b > T || (seq == 0 && a != 0)) atomicOr(&g_device_flags, kFlagBadCuSeqlens);
}

// The first sequence that ends after token t (nseq if none): a search in 32
// parts by one warp, one round of loads up to 32 sequences. In bounds whatever
// cu holds.
__device__ __forceinline__ int first_sequence(const int32_t* cu, int nseq, int64_t t) {
  if (!cu) return 0;
  const int lane = threadIdx.x & 31;
  int lo = 0, n = nseq;
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int64_t i = lo + static_cast<int64_t>(lane + 1) * step - 1;  // last sequence of this lane's part
    const bool before = i < lo + n && cu[i + 1] <= t;
    const int k = __popc(__ballot_sync(0xffffffffu, before));
    const int skip = k * step;
    lo += skip;
    n = min(step - 1, n - skip);  // the part's last sequence is known to end after t
    if (step == 1) break;
  }
  return lo;
}

}  // namespace kda
