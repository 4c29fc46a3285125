// vn_sample_bf16.cu -- drawing an index from bf16 logits.
#include "vn_sample.cuh"

namespace vn {

cudaError_t launch_sample_bf16(const SampleArgs& a, cudaStream_t stream) { return sample_rows<__nv_bfloat16>(a, stream); }

}  // namespace vn
