// pa_portable_f16.cu -- f16 instantiations of the CUDA-core list attention.
#include "pa_portable.cuh"

namespace pa {

cudaError_t launch_portable_f16(const ListArgs& a, cudaStream_t s) {
  return launch_portable_t<__half>(a, s);
}

}  // namespace pa
