// pa_kv4.cu -- pa_decode_kv4: argument checks, workspace, split and launch of
// decode over the 4-bit cache.
#include <algorithm>
#include <cstdint>

#include "pa.h"
#include "pa_internal.h"

namespace pa {

pa_status_t check_kv4(pa_dtype_t dtype, int head_dim, int group_size) {
  if (dtype != PA_F32 && dtype != PA_BF16 && dtype != PA_F16) return PA_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (group_size != 32 && group_size != 64 && group_size != 128) return PA_ERR_INVALID_ARG;
  return head_dim % group_size ? PA_ERR_INVALID_ARG : PA_OK;
}

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int64_t head_groups(const pa_params_t* p) {
  return (p->num_heads / p->num_kv_heads + kKv4Heads - 1) / kKv4Heads;
}

pa_status_t check(const pa_params_t* p, const pa_kv4_t* kv4) {
  if (pa_status_t st = check_params(p, false)) return st;
  if (!kv4 || p->partition_size < 1) return PA_ERR_INVALID_ARG;
  if (pa_status_t st = check_kv4(p->kv_dtype, p->head_dim, kv4->group_size)) return st;
  if (p->flags & ~PA_FLAG_PORTABLE) return PA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(p->num_seqs) * p->num_heads >= (int64_t(1) << 31))
    return PA_ERR_UNSUPPORTED;  // a CTA of the join per row
  if (static_cast<int64_t>(p->num_kv_heads) * head_groups(p) > 65535) return PA_ERR_UNSUPPORTED;
  // token positions up to some tiles past the longest sequence are int32
  if (static_cast<int64_t>(p->max_seq_len) + 4096 >= (int64_t(1) << 31) ||
      static_cast<int64_t>(p->partition_size) + 4096 >= (int64_t(1) << 31))
    return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

// Slots of a row for partials.  The tensor-core kernel chooses the parts from the
// lengths, which may all be the longest or one long among short ones: by partition_size, at
// most kKv4Longest, where there are many sequences, else up to kSplit items for each CTA that
// may be resident (four on each of this GPU's 152 SMs; on others the slots are more or fewer
// than they need be, and the results the same).  Up to single() tokens a row has one part, and
// the call one launch: a join costs about the time that a CTA needs for them.  Where the pairs
// leave most SMs idle, parts pay from half as many on.  Measured, us, undivided and in parts,
// 32 / 8 heads of 128: two sequences of 300 tokens 7.8 and 8.1, 600 9.4 and 8.2, 1000 11.2 and
// 8.6; eight of 600 9.6 and 9.9, 1000 11.3 and 11.7, thirty of 1000 16.3 and 18.9.  Where they
// give every CTA several items whatever happens, rows are undivided up to twice as many: 500 of
// 1200 158 and 163, of 50 to 2000 104 and 108; 256 of 2000 125 and 128, of 50 to 2000 64 and 63;
// but 160 of 50 to 2000 53 and 47 (of 1200 59 and 61).
constexpr int64_t kSplit = 8, kRoom = 608;
int64_t pairs_of(const pa_params_t* p, int64_t seqs) {
  return seqs * p->num_kv_heads * head_groups(p);
}
int64_t single(const pa_params_t* p, int64_t seqs) {
  const int64_t pairs = pairs_of(p, seqs);
  return (pairs <= kRoom / 32 ? 65536 : pairs <= 3 * kRoom ? 131072 : 262144) / p->head_dim;
}
int64_t cover(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t by_size(const pa_params_t* p) {
  return cover(p->max_seq_len, std::min(p->partition_size, kKv4Longest));
}

int64_t most_parts(const pa_params_t* p) {
  const int64_t len = p->max_seq_len;
  if (len <= single(p, p->num_seqs)) return 1;
  const int64_t by_room = cover(kSplit * kRoom, pairs_of(p, p->num_seqs));
  return std::max<int64_t>(1, std::min(cover(len, 64), std::max(by_size(p), by_room)));
}

// The bytes of a workspace: room for the slots of this many sequences and of fewer, which
// may have more parts in all (B * cover(n, B * h) <= n / h + B); never falls as sequences
// or lengths are added.
size_t workspace_bytes_of(const pa_params_t* p) {
  const int64_t B = p->num_seqs, len = p->max_seq_len;
  int64_t slots = B;
  if (len > single(p, 1))
    slots = std::min(B * cover(len, 64), std::max(B * by_size(p),
                                                  kSplit * kRoom / pairs_of(p, 1) + B));
  return workspace_layout(1, p->num_heads, p->head_dim, slots).total;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

size_t pa_kv4_workspace_size(const pa_params_t* p, const pa_kv4_t* kv4) {
  if (check(p, kv4) != PA_OK) return 0;
  return workspace_bytes_of(p);
}

pa_status_t pa_decode_kv4(const pa_params_t* p, const pa_kv4_t* kv4, const void* q,
                          const void* k_codes, const void* v_codes, const void* k_scales,
                          const void* v_scales, const int32_t* block_tables,
                          const int32_t* seq_lens, void* workspace, size_t workspace_bytes,
                          void* out, cudaStream_t stream) {
  if (pa_status_t st = check(p, kv4)) return st;
  if (p->num_seqs == 0) return PA_OK;
  if (pa_status_t st = check_tensors(q, k_codes, v_codes, block_tables, seq_lens, out)) return st;
  if (!k_scales || !v_scales || !workspace) return PA_ERR_INVALID_ARG;
  if (!aligned(k_scales, 16) || !aligned(v_scales, 16) || !aligned(workspace, 256))
    return PA_ERR_MISALIGNED;
  if (workspace_bytes < workspace_bytes_of(p)) return PA_ERR_WORKSPACE_TOO_SMALL;
  const int64_t parts = most_parts(p);
  const WorkspaceLayout lay = workspace_layout(p->num_seqs, p->num_heads, p->head_dim, parts);
  char* base = static_cast<char*>(workspace);

  Kv4Args a{};
  a.q = q;
  a.k_codes = static_cast<const uint8_t*>(k_codes);
  a.v_codes = static_cast<const uint8_t*>(v_codes);
  a.k_pairs = k_scales;
  a.v_pairs = v_scales;
  a.block_tables = block_tables;
  a.lens = seq_lens;
  a.out = out;
  a.status = reinterpret_cast<int32_t*>(base);
  a.part_max = reinterpret_cast<float*>(base + lay.max_logits_off);
  a.part_sum = reinterpret_cast<float*>(base + lay.exp_sums_off);
  a.part_out = reinterpret_cast<float*>(base + lay.tmp_out_off);
  a.num_seqs = p->num_seqs;
  a.num_heads = p->num_heads;
  a.num_kv_heads = p->num_kv_heads;
  a.head_dim = p->head_dim;
  a.block_size = p->block_size;
  a.num_blocks = p->num_blocks;
  a.max_blocks_per_seq = p->max_blocks_per_seq;
  a.max_len = p->max_seq_len;
  a.group = p->num_heads / p->num_kv_heads;
  a.head_groups = static_cast<int32_t>(head_groups(p));
  a.group_size = kv4->group_size;
  a.block_shift = (p->block_size & (p->block_size - 1)) ? -1 : __builtin_ctz(p->block_size);
  // offsets within a page are 32 bits
  a.paged16 = p->block_size % 16 == 0 &&
              static_cast<double>(p->num_kv_heads) * p->block_size * p->head_dim < 2147483648.0;
  a.out_dtype = p->out_dtype;
  a.scale_log2 = p->scale * 1.442695040888963407360f;
  // whole tiles; slots as the parts of that size need them
  a.part_floor = static_cast<int32_t>(
      std::max<int64_t>(64, cover(cover(p->max_seq_len, parts), 64) * 64));
  a.part_at = reinterpret_cast<int32_t*>(base + kPartOffset);
  a.num_parts = static_cast<int32_t>(
      std::max<int64_t>(1, cover(p->max_seq_len, a.part_floor)));
  // work items, counted in 31 bits by the tensor-core kernel
  const double items = static_cast<double>(a.num_seqs) * a.num_parts * a.num_kv_heads *
                       a.head_groups;
  const bool tc = p->kv_dtype != PA_F32 && !(p->flags & PA_FLAG_PORTABLE) && items < 2e9 &&
                  sm100_num_sms() > 0;
  cudaError_t e;
  if (tc) {
    e = (p->kv_dtype == PA_BF16 ? launch_kv4_tc_bf16 : launch_kv4_tc_f16)(
        a, static_cast<int64_t>(items), stream);
  } else {
    a.part_size = std::max(a.part_floor, 512);
    a.num_parts = static_cast<int32_t>(
        std::max<int64_t>(1, cover(p->max_seq_len, a.part_size)));
    e = (p->kv_dtype == PA_F32    ? launch_kv4_generic_f32
         : p->kv_dtype == PA_BF16 ? launch_kv4_generic_bf16
                                  : launch_kv4_generic_f16)(a, stream);
  }
  if (e != cudaSuccess) return PA_ERR_CUDA;
  if (a.num_parts == 1) return PA_OK;
  if (!tc) a.part_at = nullptr;
  return launch_kv4_join(a, stream) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"
