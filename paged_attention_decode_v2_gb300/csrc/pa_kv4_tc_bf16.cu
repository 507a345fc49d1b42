// Tensor-core decode over the 4-bit cache, bf16.
#include "pa_kv4_tc.cuh"

namespace pa {

cudaError_t launch_kv4_tc_bf16(const Kv4Args& a, int64_t items, cudaStream_t s) {
  return kv4::launch<__nv_bfloat16>(a, items, s);
}

}  // namespace pa
