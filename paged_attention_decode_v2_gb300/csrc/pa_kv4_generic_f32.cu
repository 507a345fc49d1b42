// CUDA-core decode over the 4-bit cache, f32.
#include "pa_kv4_generic.cuh"

namespace pa {

cudaError_t launch_kv4_generic_f32(const Kv4Args& a, cudaStream_t s) {
  return launch_kv4_generic<float>(a, s);
}

}  // namespace pa
