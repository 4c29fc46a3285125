// vn_sample_f32.cu -- drawing an index from fp32 logits.
#include "vn_sample.cuh"

namespace vn {

cudaError_t launch_sample_f32(const SampleArgs& a, cudaStream_t stream) { return sample_rows<float>(a, stream); }

}  // namespace vn
