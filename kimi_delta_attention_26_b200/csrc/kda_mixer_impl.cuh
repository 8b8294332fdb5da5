// kda_mixer_impl.cuh -- Mixer<T> (kda_mixer.cuh), for its three translation units.
#pragma once

#include <type_traits>

#include "kda_mixer.cuh"

namespace kda {
namespace {

template <int N>
using Int = std::integral_constant<int, N>;

// f(vector width of BYTES or one element, taps)
template <typename T, int BYTES, typename F>
void by_conv(int W, bool vec, F f) {
  auto width = [&](auto v) {
    if (W == 2) f(v, Int<2>());
    else if (W == 3) f(v, Int<3>());
    else f(v, Int<4>());
  };
  if (vec) width(Int<BYTES / sizeof(T)>());
  else width(Int<1>());
}

// f(threads per channel, states per thread) for N states
template <typename F>
void by_states(int N, F f) {
  if (N <= 4) f(Int<4>(), Int<1>());
  else if (N <= 8) f(Int<4>(), Int<2>());
  else if (N <= 16) f(Int<4>(), Int<4>());
  else if (N <= 32) f(Int<8>(), Int<4>());
  else if (N <= 64) f(Int<16>(), Int<4>());
  else f(Int<32>(), Int<4>());
}

template <typename K>
cudaError_t allow_shared(K* kernel, size_t bytes) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}

}  // namespace

template <typename T>
cudaError_t Mixer<T>::conv_fwd(const conv::Params& p, int W, bool vec, dim3 grid, cudaStream_t stream) {
  by_conv<T, conv::RUN_BYTES>(W, vec, [&](auto v, auto w) {
    conv::conv_fwd_kernel<T, v.value, w.value><<<grid, conv::NTHREADS, 0, stream>>>(p);
  });
  return cudaGetLastError();
}

template <typename T>
cudaError_t Mixer<T>::conv_decode(const conv::DecodeParams& p, int W, bool vec, dim3 grid, cudaStream_t stream) {
  by_conv<T, conv::RUN_BYTES>(W, vec, [&](auto v, auto w) {
    conv::conv_decode_kernel<T, v.value, w.value><<<grid, conv::NTHREADS, 0, stream>>>(p);
  });
  return cudaGetLastError();
}

template <typename T>
cudaError_t Mixer<T>::conv_bwd(const conv::BwdParams& p, int W, bool vec, dim3 grid, cudaStream_t stream) {
  by_conv<T, conv::RUN_BYTES>(W, vec, [&](auto v, auto w) {
    conv::conv_bwd_kernel<T, v.value, w.value><<<grid, conv::NTHREADS, 0, stream>>>(p);
  });
  return cudaGetLastError();
}

// With no more blocks than SMs the deeper shape (where its shared memory fits
// and states come in fours), else two blocks per SM. Measured (8192 tokens x 4096
// channels x 16 states, bf16): one sequence, 128 blocks, 286 us deep and 331 us
// not; 8 sequences, 1024 blocks, 264 us and 236 us.
template <typename T>
cudaError_t Mixer<T>::scan(ssm::Params p, int mode, int ranges, int sms, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  by_states(p.N, [&](auto l, auto s) {
    constexpr int CH = 128 / l.value;
    p.blocks_per_group = (p.C / p.G + CH - 1) / CH;
    const int64_t blocks = static_cast<int64_t>(p.G) * p.blocks_per_group;
    auto go = [&](auto o, auto deep) {
      using Sh = ssm::FwdShared<T, l.value, s.value, CH, o.value, deep.value>;
      auto* kernel = ssm::ssm_fwd_kernel<T, l.value, s.value, CH, o.value, deep.value>;
      if ((e = allow_shared(kernel, sizeof(Sh))) == cudaSuccess)
        kernel<<<dim3(static_cast<unsigned>(blocks), ranges), Sh::THREADS, sizeof(Sh), stream>>>(p);
    };
    auto shape = [&](auto o) {
      if constexpr (s.value == 4 && l.value <= 8 && o.value != ssm::BACK) {
        if (blocks * ranges <= sms) return go(o, std::true_type());
      }
      go(o, std::false_type());
    };
    if (mode == ssm::OUTPUTS) shape(Int<ssm::OUTPUTS>());
    else if (mode == ssm::STATES) shape(Int<ssm::STATES>());
    else shape(Int<ssm::BACK>());
  });
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t Mixer<T>::scan_decode(const ssm::DecodeParams& p, int64_t requests, cudaStream_t stream) {
  by_states(p.N, [&](auto l, auto) {
    constexpr int CH = ssm::NTHREADS / l.value * 4;
    ssm::ssm_decode_kernel<T, l.value>
        <<<dim3(static_cast<unsigned>(requests), (p.C + CH - 1) / CH), ssm::NTHREADS, 0, stream>>>(p);
  });
  return cudaGetLastError();
}

template <typename T>
cudaError_t Mixer<T>::scan_bwd(ssm::BwdParams p, int ranges, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  by_states(p.f.N, [&](auto l, auto) {
    constexpr size_t bytes = sizeof(ssm::BwdShared<l.value>);
    auto go = [&](auto split) {
      auto* kernel = ssm::ssm_bwd_kernel<T, l.value, split.value>;
      if ((e = allow_shared(kernel, bytes)) == cudaSuccess)
        kernel<<<dim3(p.f.G * p.f.blocks_per_group, ranges), ssm::BwdShared<l.value>::THREADS, bytes, stream>>>(p);
    };
    if (p.f.run) go(std::true_type());
    else go(std::false_type());
  });
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t Mixer<T>::scan_reduce(const ssm::ReduceParams& p, unsigned blocks, cudaStream_t stream) {
  ssm::ssm_reduce_kernel<T><<<blocks, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t Mixer<T>::status(uint32_t* flags, uint32_t* waits, bool reset_flags, bool reset_waits) {
  const uint32_t zero = 0;
  uint32_t f = 0, w = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&f, g_device_flags, sizeof(f));
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&w, g_wait_timeouts, sizeof(w));
  if (e == cudaSuccess && reset_flags && f) e = cudaMemcpyToSymbol(g_device_flags, &zero, sizeof(zero));
  if (e == cudaSuccess && reset_waits && w) e = cudaMemcpyToSymbol(g_wait_timeouts, &zero, sizeof(zero));
  *flags |= f;
  *waits += w;
  return e;
}

}  // namespace kda
