// pa_portable_f32.cu -- f32 instantiations of the CUDA-core list attention.
#include "pa_portable.cuh"

namespace pa {

cudaError_t launch_portable_f32(const ListArgs& a, cudaStream_t s) {
  return launch_portable_t<float>(a, s);
}

}  // namespace pa
