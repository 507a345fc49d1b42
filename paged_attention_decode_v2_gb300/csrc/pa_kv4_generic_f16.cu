// CUDA-core decode over the 4-bit cache, f16.
#include "pa_kv4_generic.cuh"

namespace pa {

cudaError_t launch_kv4_generic_f16(const Kv4Args& a, cudaStream_t s) {
  return launch_kv4_generic<__half>(a, s);
}

}  // namespace pa
