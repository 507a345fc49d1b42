// CUDA-core decode over the 4-bit cache, bf16.
#include "pa_kv4_generic.cuh"

namespace pa {

cudaError_t launch_kv4_generic_bf16(const Kv4Args& a, cudaStream_t s) {
  return launch_kv4_generic<__nv_bfloat16>(a, s);
}

}  // namespace pa
