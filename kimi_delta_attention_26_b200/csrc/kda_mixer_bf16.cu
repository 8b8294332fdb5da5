// kda_mixer_bf16.cu -- the convolution's and the scan's kernels for bf16 tensors.
#include "kda_mixer_impl.cuh"

template struct kda::Mixer<__nv_bfloat16>;
