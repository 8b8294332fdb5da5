// kda_io.cuh -- what the convolution and the scan share: loads and stores of
// bf16, fp16 and fp32 rows, the activations, and finding a token's sequence.
#pragma once

#include <cuda_fp16.h>

#include "kda_prims.cuh"

namespace kda {

// V consecutive elements of a row, moved as one access.
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T v[V];
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
  const Pack<T, V> a = *reinterpret_cast<const Pack<T, V>*>(p);
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = to_f32(a.v[i]);
}

template <typename T, int V>
__device__ __forceinline__ void store_f32(T* p, const float (&x)[V]) {
  Pack<T, V> a;
#pragma unroll
  for (int i = 0; i < V; ++i) a.v[i] = from_f32<T>(x[i]);
  *reinterpret_cast<Pack<T, V>*>(p) = a;
}

// sigmoid, x sigmoid(x) and its derivative. exp(-x) overflows to infinity for
// x below -88, where the quotient is the right 0.
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }
__device__ __forceinline__ float dsilu(float x) {
  const float g = sigmoid(x);
  return g * fmaf(x, 1.f - g, 1.f);
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
