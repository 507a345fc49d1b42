// pa_rows_host.cu -- host side of the row attention kernel (pa_rows.cuh): when
// it applies, its TMA tensor maps and its grid.
#include <algorithm>
#include <cstdint>

#include "pa_internal.h"

namespace pa {

cudaError_t launch_rows_prefix_bf16(const RowsArgs& a, const CUtensorMap (&m)[5], int grid,
                                    bool pdl, cudaStream_t s);
cudaError_t launch_rows_prefix_f16(const RowsArgs& a, const CUtensorMap (&m)[5], int grid,
                                   bool pdl, cudaStream_t s);
cudaError_t launch_rows_window_bf16(const RowsArgs& a, const CUtensorMap (&m)[5], int grid,
                                    bool pdl, cudaStream_t s);
cudaError_t launch_rows_window_f16(const RowsArgs& a, const CUtensorMap (&m)[5], int grid,
                                   bool pdl, cudaStream_t s);

int rows_applicable(pa_dtype_t t, int num_heads, int num_kv_heads, int head_dim, int block_size,
                    int64_t num_blocks, int64_t num_tokens, float scale) {
  if (t != PA_BF16 && t != PA_F16) return 0;
  if (num_heads / num_kv_heads > 64) return 0;
  const bool shape = (head_dim == 256 && (block_size == 16 || block_size == 32)) ||
                     (head_dim == 128 && (block_size == 16 || block_size == 32 || block_size == 64));
  if (!shape) return 0;
  if (!(scale > 0.f) || scale > 3.0e38f) return 0;  // the masked logits are -inf * scale
  // TMA coordinates are int32
  if (num_blocks * num_kv_heads * block_size + block_size >= (int64_t(1) << 31)) return 0;
  if (num_tokens + 512 >= (int64_t(1) << 31)) return 0;
  return sm100_num_sms();
}

cudaError_t launch_rows(RowsArgs a, pa_dtype_t t, const RowsTensors& x, int sms, bool pdl,
                        cudaStream_t s) {
  const uint64_t D = static_cast<uint64_t>(a.head_dim), BS = static_cast<uint64_t>(a.block_size);
  const uint64_t Hq = static_cast<uint64_t>(a.num_heads), Hkv = static_cast<uint64_t>(a.num_kv_heads);
  const uint64_t rows = static_cast<uint64_t>(a.num_blocks) * Hkv * BS;
  const uint64_t T = static_cast<uint64_t>(a.num_tokens);
  CUtensorMap m[5];
  {
    const uint64_t dims[4] = {64, Hq, T, D / 64};
    const uint64_t strides[3] = {D * 2, Hq * D * 2, 128};
    const uint32_t box[4] = {64, static_cast<uint32_t>(a.group),
                             static_cast<uint32_t>(a.row_tokens), 1};
    if (cudaError_t e = encode_tiled(&m[0], t, 4, x.q, dims, strides, box)) return e;
  }
  if (x.k) {
    const uint64_t dims[4] = {64, Hkv, T, D / 64};
    const uint64_t strides[3] = {D * 2, Hkv * D * 2, 128};
    const uint32_t box_k[4] = {64, 1, 128, 1};
    const uint32_t box_v[4] = {64, 1, static_cast<uint32_t>(BS), static_cast<uint32_t>(D / 64)};
    if (cudaError_t e = encode_tiled(&m[1], t, 4, x.k, dims, strides, box_k)) return e;
    if (cudaError_t e = encode_tiled(&m[2], t, 4, x.v, dims, strides, box_v)) return e;
  } else {
    m[1] = m[2] = m[0];  // never read
  }
  {
    const uint64_t dims[2] = {D, rows};
    const uint64_t strides[1] = {D * 2};
    const uint32_t box[2] = {64, static_cast<uint32_t>(BS)};
    if (cudaError_t e = encode_tiled(&m[3], t, 2, x.k_cache, dims, strides, box)) return e;
  }
  {
    const uint64_t dims[3] = {64, rows, D / 64};
    const uint64_t strides[2] = {D * 2, 128};
    const uint32_t box[3] = {64, static_cast<uint32_t>(BS), static_cast<uint32_t>(D / 64)};
    if (cudaError_t e = encode_tiled(&m[4], t, 3, x.v_cache, dims, strides, box)) return e;
  }
  const bool prefix = !x.k;
  const int64_t units = prefix ? static_cast<int64_t>(a.key_blocks) * a.row_groups
                               : static_cast<int64_t>(a.row_groups) * a.num_seqs * a.num_kv_heads;
  if (units == 0) return cudaSuccess;
  const int grid = static_cast<int>(std::min<int64_t>(units, sms));
  if (prefix)
    return t == PA_BF16 ? launch_rows_prefix_bf16(a, m, grid, pdl, s)
                        : launch_rows_prefix_f16(a, m, grid, pdl, s);
  return t == PA_BF16 ? launch_rows_window_bf16(a, m, grid, pdl, s)
                      : launch_rows_window_f16(a, m, grid, pdl, s);
}

}  // namespace pa
