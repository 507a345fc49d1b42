// pa_window.cu -- pa_decode_window and pa_prefill_window: argument checks,
// workspace and the choice of kernels for attention with a sliding window
// and sinks (the token lists are in pa_span.cuh).
#include <algorithm>
#include <cstdint>

#include "pa.h"
#include "pa_internal.h"
#include "pa_span.cuh"

namespace pa {
namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

pa_status_t check_window(const pa_window_t* w) {
  return w && w->window >= 1 && w->num_sinks >= 0 ? PA_OK : PA_ERR_INVALID_ARG;
}

// The window with both counts cut to what a sequence of max_len tokens can
// show, so that sums of them stay in range.
pa_window_t clamped(const pa_window_t* w, int32_t max_len) {
  const int32_t most = std::max(max_len, 1);
  return pa_window_t{std::min(w->window, most), std::min(w->num_sinks, most)};
}

int64_t parts_of(int64_t len, int64_t size) { return std::max<int64_t>(1, (len + size - 1) / size); }

pa_status_t check_decode(const pa_params_t* p, const pa_window_t* w) {
  if (pa_status_t st = check_params(p, true)) return st;
  if (pa_status_t st = check_window(w)) return st;
  if (static_cast<int64_t>(p->num_seqs) * p->num_heads >= (int64_t(1) << 31))
    return PA_ERR_UNSUPPORTED;  // a CTA of the join per row
  // list positions up to a partition past the longest list are int32
  if (static_cast<int64_t>(p->max_seq_len) + p->partition_size + 2LL * p->block_size >=
      (int64_t(1) << 31))
    return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

// Parts of a list on the tensor-core kernel, whose persistent grid has room for
// kRoom items (two CTAs on each of 152 SMs) at a time.
//   * Many (sequence, KV head) pairs -- two rounds of them: partition_size,
//     evened out over the list, so that short lists do not wait for long ones.
//   * Fewer: the split that takes the least time, a round costing as much as
//     its part is long plus about 100 tokens (start and hand-over), a partial
//     about 2 (the join).  One part needs no join at all.
// Measured (window, heads 24 / 4 x 256, bf16; us with this split against parts of
// 512): 1 sequence, 4096: 19.8 / 23.2; 4, 4096: 25 / 27; 16, 2048: 36 / 44; 64,
// 1024: 52 / 55; 256 sequences, 8 KV heads of 128, 1024: 132, and 137 undivided.
constexpr int64_t kRoom = 304;

int64_t tc_parts(const pa_params_t* p, int64_t seqs, int64_t len) {
  constexpr int64_t kStart = 100, kJoin = 2, kLeast = 128;
  const int64_t pairs = seqs * p->num_kv_heads;
  int64_t parts = parts_of(len, p->partition_size);
  if (pairs < 2 * kRoom) {
    // The cost of n parts is a line in len; the least of some lines falls to
    // flatter ones, of more parts, as len grows: n never falls.
    double best = -1;
    for (int64_t n = 1; n <= 64 && (n == 1 || n * kLeast <= len); ++n) {
      const double rounds = static_cast<double>((pairs * n + kRoom - 1) / kRoom);
      const double cost = rounds / n * len + rounds * kStart + (n > 1 ? n * kJoin : 0);
      if (best < 0 || cost < best) {
        best = cost;
        parts = n;
      }
    }
  }
  return parts;
}

// Tokens of a part: whole blocks, of any size the kernel takes.
int32_t tc_part(const pa_params_t* p, int64_t len) {
  const int64_t parts = tc_parts(p, p->num_seqs, len);
  return static_cast<int32_t>(((len + parts - 1) / parts + 63) / 64 * 64);
}

int64_t list_len(const pa_params_t* p, const pa_window_t& w) {
  return window_max_len(p->max_seq_len, w.window, w.num_sinks, p->block_size);
}

// Room for the partials of either kernel, whatever the device, of `seqs`
// sequences.
WorkspaceLayout layout_of(const pa_params_t* p, const pa_window_t& w, int64_t seqs) {
  const int64_t len = list_len(p, w);
  return workspace_layout(static_cast<int32_t>(seqs), p->num_heads, p->head_dim,
                          std::max(parts_of(len, p->partition_size), tc_parts(p, seqs, len)));
}

cudaError_t launch_list(const ListArgs& a, pa_dtype_t t, cudaStream_t s) {
  switch (t) {
    case PA_F32: return launch_portable_f32(a, s);
    case PA_BF16: return launch_portable_bf16(a, s);
    default: return launch_portable_f16(a, s);
  }
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

size_t pa_window_workspace_size(const pa_params_t* p, const pa_window_t* window) {
  if (check_decode(p, window) != PA_OK) return 0;
  const pa_window_t w = clamped(window, p->max_seq_len);
  size_t most = layout_of(p, w, p->num_seqs).total;
  // fewer sequences may have more parts in all
  for (int64_t s = 1; s < p->num_seqs && s * p->num_kv_heads < 2 * kRoom; ++s)
    most = std::max(most, layout_of(p, w, s).total);
  return most;
}

pa_status_t pa_decode_window(const pa_params_t* p, const pa_window_t* window, const void* q,
                             const void* k_cache, const void* v_cache,
                             const int32_t* block_tables, const int32_t* seq_lens,
                             void* workspace, size_t workspace_bytes, void* out,
                             cudaStream_t stream) {
  if (pa_status_t st = check_decode(p, window)) return st;
  if (p->num_seqs == 0) return PA_OK;
  if (pa_status_t st = check_tensors(q, k_cache, v_cache, block_tables, seq_lens, out)) return st;
  if (!workspace) return PA_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return PA_ERR_MISALIGNED;
  const pa_window_t w = clamped(window, p->max_seq_len);
  const WorkspaceLayout lay = layout_of(p, w, p->num_seqs);
  if (workspace_bytes < lay.total) return PA_ERR_WORKSPACE_TOO_SMALL;
  char* base = static_cast<char*>(workspace);
  float* part_max = reinterpret_cast<float*>(base + lay.max_logits_off);
  float* part_sum = reinterpret_cast<float*>(base + lay.exp_sums_off);
  float* part_out = reinterpret_cast<float*>(base + lay.tmp_out_off);

  JoinArgs j{};
  JoinList& l = j.list[0];
  l.m = part_max;
  l.s = part_sum;
  l.o = part_out;
  l.lens = seq_lens;
  l.max_len = p->max_seq_len;
  l.part_size = p->partition_size;
  l.window = w.window;
  l.num_sinks = w.num_sinks;
  l.block_size = p->block_size;
  j.out = out;
  j.num_rows = static_cast<int64_t>(p->num_seqs) * p->num_heads;
  j.num_heads = p->num_heads;
  j.head_dim = p->head_dim;
  j.group = p->num_heads / p->num_kv_heads;
  j.out_dtype = p->out_dtype;

  if (tc_applicable(p)) {
    KernelArgs a = make_args(p, q, k_cache, v_cache, block_tables, seq_lens, out);
    a.status = reinterpret_cast<int32_t*>(base);
    a.max_logits = part_max;
    a.exp_sums = part_sum;
    a.tmp_out = part_out;
    a.window = w.window;
    a.num_sinks = w.num_sinks;
    a.max_list = static_cast<int32_t>(list_len(p, w));
    a.partition_size = a.max_list > 0 ? tc_part(p, a.max_list) : p->partition_size;
    const int64_t parts = parts_of(a.max_list, a.partition_size);
    a.num_partitions = static_cast<int32_t>(parts);
    const bool v2 = parts > 1;
    if (launch_tc(a, p->kv_dtype, v2, stream) != cudaSuccess) return PA_ERR_CUDA;
    if (!v2) return PA_OK;
    l.stride = a.num_partitions;
    l.part_size = a.partition_size;
    l.block_list = 1;
    return launch_join(j, stream, true) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
  }

  ListArgs a{};
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_tables = block_tables;
  a.lens = seq_lens;
  a.out = out;
  a.part_max = part_max;
  a.part_sum = part_sum;
  a.part_out = part_out;
  a.status = reinterpret_cast<int32_t*>(base);
  a.rows = p->num_seqs;
  a.mode = kDecodeWindow;
  a.num_seqs = p->num_seqs;
  a.num_heads = p->num_heads;
  a.num_kv_heads = p->num_kv_heads;
  a.head_dim = p->head_dim;
  a.block_size = p->block_size;
  a.num_blocks = p->num_blocks;
  a.max_blocks_per_seq = p->max_blocks_per_seq;
  a.max_len = p->max_seq_len;
  a.window = w.window;
  a.num_sinks = w.num_sinks;
  a.part_size = p->partition_size;
  const int64_t parts = parts_of(
      std::min<int64_t>(p->max_seq_len, static_cast<int64_t>(w.window) + w.num_sinks),
      p->partition_size);
  if (parts > 65535) return PA_ERR_UNSUPPORTED;
  a.num_parts = static_cast<int32_t>(parts);
  a.group = p->num_heads / p->num_kv_heads;
  a.out_dtype = p->out_dtype;
  a.split_x = (p->flags & PA_FLAG_SPLIT_X) ? 1 : 0;
  a.scale_log2 = p->scale * 1.442695040888963407360f;
  if (launch_list(a, p->kv_dtype, stream) != cudaSuccess) return PA_ERR_CUDA;
  if (parts == 1) return PA_OK;
  l.stride = a.num_parts;
  return launch_join(j, stream, true) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status_t pa_prefill_window(const pa_prefill_params_t* p, const pa_window_t* window,
                              const void* q, const void* k, const void* v, const void* k_cache,
                              const void* v_cache, const int32_t* block_tables,
                              const int32_t* query_start, const int32_t* ctx_lens, void* out,
                              cudaStream_t stream) {
  if (!p) return PA_ERR_INVALID_ARG;
  if (p->num_seqs < 0 || p->num_heads < 1 || p->num_kv_heads < 1) return PA_ERR_INVALID_ARG;
  if (p->num_heads % p->num_kv_heads) return PA_ERR_INVALID_ARG;
  if (p->total_tokens < 0 || p->max_query_len < 0 || p->max_ctx_len < 0) return PA_ERR_INVALID_ARG;
  if (p->block_size < 1 || p->num_blocks < 1 || p->max_blocks_per_seq < 1) return PA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(p->max_ctx_len) >
      static_cast<int64_t>(p->max_blocks_per_seq) * p->block_size)
    return PA_ERR_INVALID_ARG;
  if (!(p->scale > 0.f) || p->scale > 3.0e38f) return PA_ERR_INVALID_ARG;
  if (p->flags & ~(PA_FLAG_PORTABLE | PA_FLAG_SELFTEST_STALL | PA_FLAG_SPLIT_X))
    return PA_ERR_INVALID_ARG;
  if (pa_status_t st = check_window(window)) return st;
  if (p->kv_dtype != PA_F32 && p->kv_dtype != PA_BF16 && p->kv_dtype != PA_F16)
    return PA_ERR_UNSUPPORTED;
  if (p->out_dtype != PA_F32 && p->out_dtype != p->kv_dtype) return PA_ERR_UNSUPPORTED;
  if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (p->num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
  // positions are int32
  if (static_cast<int64_t>(p->max_ctx_len) + p->max_query_len + 256 >= (int64_t(1) << 31) ||
      static_cast<int64_t>(p->total_tokens) + 256 >= (int64_t(1) << 31))
    return PA_ERR_UNSUPPORTED;
  if (p->num_seqs == 0 || p->total_tokens == 0 || p->max_query_len == 0) return PA_OK;
  for (const void* ptr : {q, k, v, k_cache, v_cache, static_cast<const void*>(out)})
    if (!ptr) return PA_ERR_INVALID_ARG;
  if (!block_tables || !query_start || !ctx_lens) return PA_ERR_INVALID_ARG;
  for (const void* ptr : {q, k, v, k_cache, v_cache, static_cast<const void*>(out)})
    if (!aligned(ptr, 16)) return PA_ERR_MISALIGNED;
  if (!aligned(block_tables, 4) || !aligned(query_start, 4) || !aligned(ctx_lens, 4))
    return PA_ERR_MISALIGNED;
  const pa_window_t w = clamped(window, p->max_ctx_len + p->max_query_len);
  // row tiles of the tensor-core kernel: 128 rows are 128 / G tokens, one or
  // two tiles to a unit; it counts its units in 31 bits
  const int G = p->num_heads / p->num_kv_heads;
  const int dual = p->head_dim == 128, row_tokens = std::max(128 / G, 1);
  const int group_tokens = row_tokens * (dual ? 2 : 1);
  const int64_t row_groups = (static_cast<int64_t>(p->max_query_len) + group_tokens - 1) /
                             group_tokens;
  const bool counts = static_cast<int64_t>(p->num_seqs) * p->num_kv_heads <
                      (int64_t(1) << 30) / row_groups;
  const int sms = (p->flags & (PA_FLAG_PORTABLE | PA_FLAG_SPLIT_X)) || !counts
                      ? 0
                      : rows_applicable(p->kv_dtype, p->num_heads, p->num_kv_heads, p->head_dim,
                                        p->block_size, p->num_blocks, p->total_tokens, p->scale);
  if (sms > 0) {
    RowsArgs a{};
    a.block_tables = block_tables;
    a.query_start = query_start;
    a.lens = ctx_lens;
    a.out = out;
    a.num_seqs = p->num_seqs;
    a.num_heads = p->num_heads;
    a.num_kv_heads = p->num_kv_heads;
    a.head_dim = p->head_dim;
    a.block_size = p->block_size;
    a.num_blocks = p->num_blocks;
    a.max_blocks_per_seq = p->max_blocks_per_seq;
    a.num_tokens = p->total_tokens;
    a.max_query_len = p->max_query_len;
    a.max_ctx_len = p->max_ctx_len;
    a.window = w.window;
    a.num_sinks = w.num_sinks;
    a.group = G;
    a.row_tokens = row_tokens;
    a.dual = dual;
    a.group_tokens = group_tokens;
    a.row_groups = static_cast<int32_t>(row_groups);
    a.out_dtype = p->out_dtype;
    a.selftest_stall = (p->flags & PA_FLAG_SELFTEST_STALL) ? 1 : 0;
    a.scale_log2 = p->scale * 1.442695040888963407360f;
    const RowsTensors x{q, k, v, k_cache, v_cache};
    return launch_rows(a, p->kv_dtype, x, sms, false, stream) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
  }

  ListArgs a{};
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_new = k;
  a.v_new = v;
  a.block_tables = block_tables;
  a.lens = ctx_lens;
  a.query_start = query_start;
  a.out = out;
  a.rows = p->total_tokens;
  a.mode = kPrefillWindow;
  a.num_seqs = p->num_seqs;
  a.num_heads = p->num_heads;
  a.num_kv_heads = p->num_kv_heads;
  a.head_dim = p->head_dim;
  a.block_size = p->block_size;
  a.num_blocks = p->num_blocks;
  a.max_blocks_per_seq = p->max_blocks_per_seq;
  a.max_len = p->max_ctx_len;
  a.total_tokens = p->total_tokens;
  a.max_query_len = p->max_query_len;
  a.window = w.window;
  a.num_sinks = w.num_sinks;
  a.num_parts = 1;
  a.group = p->num_heads / p->num_kv_heads;
  a.out_dtype = p->out_dtype;
  a.split_x = (p->flags & PA_FLAG_SPLIT_X) ? 1 : 0;
  a.scale_log2 = p->scale * 1.442695040888963407360f;
  return launch_list(a, p->kv_dtype, stream) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"
