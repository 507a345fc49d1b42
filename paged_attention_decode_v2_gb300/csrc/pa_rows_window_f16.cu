// pa_rows_window_f16.cu -- f16 instantiations of the row attention kernel (window).
#include "pa_rows.cuh"

namespace pa {

cudaError_t launch_rows_window_f16(const RowsArgs& a, const CUtensorMap (&m)[5], int grid, bool pdl,
                                cudaStream_t s) {
  return launch_rows_t<__half, false>(a, m, grid, pdl, s);
}

}  // namespace pa
