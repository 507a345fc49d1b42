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
  // token positions up to two parts past the longest sequence are int32
  if (static_cast<int64_t>(p->max_seq_len) + 2LL * p->partition_size + 256 >= (int64_t(1) << 31))
    return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

int64_t parts_of(int64_t len, int64_t size) { return std::max<int64_t>(1, (len + size - 1) / size); }

// Parts of the longest of `seqs` sequences.  There is room for some work items --
// (part, KV head, eight query heads) -- at a time, a CTA each on 152 SMs.
//   * Many sequences, two rounds of items undivided: partition_size.
//   * Fewer: the split that takes the least time, as for the windowed decode: a
//     round costs as much as its part is long plus a start, a partial the join.
int64_t room_for(const pa_params_t* p) { return 152 * kv4_tc_ctas(p->head_dim); }
constexpr int64_t kMostParts = 640;

int64_t parts_for(const pa_params_t* p, int64_t seqs) {
  constexpr int64_t kStart = 128, kJoin = 2, kLeast = 64;
  const int64_t len = p->max_seq_len, room = room_for(p);
  const int64_t pairs = seqs * p->num_kv_heads * head_groups(p);
  if (pairs >= 2 * room) return parts_of(len, p->partition_size);
  // the cost of n parts is a line in len: n never falls as len grows
  int64_t parts = 1;
  double best = -1;
  for (int64_t n = 1; n <= kMostParts && (n == 1 || n * kLeast <= len); ++n) {
    const double rounds = static_cast<double>((pairs * n + room - 1) / room);
    const double cost = rounds / n * len + rounds * kStart + (n > 1 ? n * kJoin : 0);
    if (best < 0 || cost < best) {
      best = cost;
      parts = n;
    }
  }
  return parts;
}

WorkspaceLayout layout_of(const pa_params_t* p, int64_t seqs) {
  return workspace_layout(seqs, p->num_heads, p->head_dim, parts_for(p, seqs));
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

size_t pa_kv4_workspace_size(const pa_params_t* p, const pa_kv4_t* kv4) {
  if (check(p, kv4) != PA_OK) return 0;
  size_t most = layout_of(p, p->num_seqs).total;
  // fewer sequences may have more parts in all
  for (int64_t s = 1; s < p->num_seqs && s * p->num_kv_heads < 2 * room_for(p); ++s)
    most = std::max(most, layout_of(p, s).total);
  return most;
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
  const WorkspaceLayout lay = layout_of(p, p->num_seqs);
  if (workspace_bytes < lay.total) return PA_ERR_WORKSPACE_TOO_SMALL;
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
  a.paged16 = p->block_size % 16 == 0;
  a.out_dtype = p->out_dtype;
  a.scale_log2 = p->scale * 1.442695040888963407360f;
  // parts of whole tiles; evened out over the longest sequence
  const int64_t parts = parts_for(p, p->num_seqs);
  a.part_size = static_cast<int32_t>(
      std::max<int64_t>(64, ((p->max_seq_len + parts - 1) / parts + 63) / 64 * 64));
  a.num_parts = static_cast<int32_t>(parts_of(p->max_seq_len, a.part_size));
  // work items, counted in 31 bits by the tensor-core kernel
  const double items = static_cast<double>(a.num_seqs) * a.num_parts * a.num_kv_heads *
                       a.head_groups;
  const bool tc = p->kv_dtype != PA_F32 && !(p->flags & PA_FLAG_PORTABLE) && items < 2e9 &&
                  sm100_num_sms() > 0;
  cudaError_t e;
  if (tc)
    e = (p->kv_dtype == PA_BF16 ? launch_kv4_tc_bf16 : launch_kv4_tc_f16)(
        a, static_cast<int64_t>(items), stream);
  else
    e = (p->kv_dtype == PA_F32    ? launch_kv4_generic_f32
         : p->kv_dtype == PA_BF16 ? launch_kv4_generic_bf16
                                  : launch_kv4_generic_f16)(a, stream);
  if (e != cudaSuccess) return PA_ERR_CUDA;
  if (a.num_parts == 1) return PA_OK;
  JoinArgs j{};
  JoinList& l = j.list[0];
  l.m = a.part_max;
  l.s = a.part_sum;
  l.o = a.part_out;
  l.lens = seq_lens;
  l.max_len = p->max_seq_len;
  l.stride = a.num_parts;
  l.part_size = a.part_size;
  l.block_size = p->block_size;
  j.out = out;
  j.num_rows = static_cast<int64_t>(p->num_seqs) * p->num_heads;
  j.num_heads = p->num_heads;
  j.head_dim = p->head_dim;
  j.group = a.group;
  j.out_dtype = p->out_dtype;
  return launch_join(j, stream, true) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"
