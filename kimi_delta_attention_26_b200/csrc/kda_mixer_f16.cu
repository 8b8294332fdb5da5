// kda_mixer_f16.cu -- the convolution's and the scan's kernels for fp16 tensors.
#include "kda_mixer_impl.cuh"

template struct kda::Mixer<__half>;
