// Single-token attention over a paged cache of 8-bit codes: e4m3 (the kernel: attention_decode8.cuh).
#include "attention_decode8.cuh"

namespace rpp {

cudaError_t launch_attention_decode8_e4m3(const void* params, cudaStream_t stream) {
  return launch_codes<false>(*static_cast<const Decode8Params*>(params), stream);
}

}  // namespace rpp
