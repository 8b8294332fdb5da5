// kda_mixer.cuh -- the launches of the convolution and the scan for one element
// type. Each type is a translation unit of its own (kda_mixer_bf16.cu,
// kda_mixer_f16.cu, kda_mixer_f32.cu), which compile side by side.
#pragma once

#include "kda_conv.cuh"
#include "kda_ssm.cuh"

namespace kda {

template <typename T>
struct Mixer {
  // `vec`: accesses of conv::RUN_BYTES are possible
  static cudaError_t conv_fwd(const conv::Params& p, int W, bool vec, dim3 grid, cudaStream_t stream);
  static cudaError_t conv_decode(const conv::DecodeParams& p, int W, bool vec, dim3 grid, cudaStream_t stream);
  static cudaError_t conv_bwd(const conv::BwdParams& p, int W, bool vec, dim3 grid, cudaStream_t stream);
  // a scan over `ranges` ranges (mode: ssm::OUTPUTS, STATES or BACK) on a device of `sms` SMs
  static cudaError_t scan(ssm::Params p, int mode, int ranges, int sms, cudaStream_t stream);
  static cudaError_t scan_decode(const ssm::DecodeParams& p, int64_t requests, cudaStream_t stream);
  static cudaError_t scan_bwd(ssm::BwdParams p, int ranges, cudaStream_t stream);
  static cudaError_t scan_reduce(const ssm::ReduceParams& p, unsigned blocks, cudaStream_t stream);
  // this translation unit's status words: OR-ed and added to the two words, then cleared where asked
  static cudaError_t status(uint32_t* flags, uint32_t* waits, bool reset_flags, bool reset_waits);
};

extern template struct Mixer<__nv_bfloat16>;
extern template struct Mixer<__half>;
extern template struct Mixer<float>;

}  // namespace kda
