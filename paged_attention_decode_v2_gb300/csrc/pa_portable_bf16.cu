// pa_portable_bf16.cu -- bf16 instantiations of the CUDA-core list attention.
#include "pa_portable.cuh"

namespace pa {

cudaError_t launch_portable_bf16(const ListArgs& a, cudaStream_t s) {
  return launch_portable_t<__nv_bfloat16>(a, s);
}

}  // namespace pa
