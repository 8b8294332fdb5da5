// kda_mixer_f32.cu -- the convolution's and the scan's kernels for fp32 tensors.
#include "kda_mixer_impl.cuh"

template struct kda::Mixer<float>;
