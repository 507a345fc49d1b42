// pa_rows_window_bf16.cu -- bf16 instantiations of the row attention kernel (window).
#include "pa_rows.cuh"

namespace pa {

cudaError_t launch_rows_window_bf16(const RowsArgs& a, const CUtensorMap (&m)[5], int grid, bool pdl,
                                cudaStream_t s) {
  return launch_rows_t<__nv_bfloat16, false>(a, m, grid, pdl, s);
}

}  // namespace pa
