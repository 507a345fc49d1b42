// Tensor-core decode over the 4-bit cache, f16.
#include "pa_kv4_tc.cuh"

namespace pa {

cudaError_t launch_kv4_tc_f16(const Kv4Args& a, int64_t items, cudaStream_t s) {
  return kv4::launch<__half>(a, items, s);
}

}  // namespace pa
