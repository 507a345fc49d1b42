// pa_prefix.cu -- pa_decode_prefix: a batch that shares a prefix.
//
// The prefix is one product over all rows of a KV head, split over keys
// (pa_rows.cuh; on the CUDA cores pa_portable.cuh).  Short own lists of many
// sequences are then taken by one kernel that joins them with the prefix's
// partials (pa_own.cu): two launches.  Others go through pass 1 of V2 over
// their block tables, as in pa_decode_v2_partitions, first, and a third kernel
// joins both lists of partials (pa_join.cu).
#include <algorithm>
#include <cstdint>

#include "pa.h"
#include "pa_internal.h"
#include "pa_span.cuh"

namespace pa {
namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kPortablePart = 1024;  // prefix tokens of a partial on the CUDA cores

size_t up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

pa_status_t check_prefix(const pa_params_t* p, const pa_prefix_t* x) {
  if (pa_status_t st = check_params(p, true)) return st;
  if (!x || x->max_prefix_len < 0 || x->max_prefix_blocks < 0) return PA_ERR_INVALID_ARG;
  if (x->max_prefix_len > static_cast<int64_t>(x->max_prefix_blocks) * p->block_size)
    return PA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(p->num_seqs) * p->num_heads >= (int64_t(1) << 31))
    return PA_ERR_UNSUPPORTED;  // a CTA of the join per row
  if (static_cast<int64_t>(p->max_seq_len) + p->partition_size + 256 >= (int64_t(1) << 31) ||
      static_cast<int64_t>(x->max_prefix_len) + 2048 >= (int64_t(1) << 31))
    return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

// The tensor-core prefix pass's plan for these shapes, whatever the device:
// rows of a row tile and of a unit, and the number of key blocks.  Row groups x
// key blocks are the units; with k rounds of S CTAs there is room for
// floor(S k / groups) key blocks, and a round costs as much as its key block is
// long, so k minimises k / key blocks (and a little per round).
struct RowsPlan {
  bool shape;  // served by the tensor-core kernel as far as shapes go
  int row_tokens, group_tokens, row_groups, dual, lanes, key_blocks;
  int64_t np;  // partials of a row
};

constexpr int kSms = 152;

int key_blocks(int row_groups, int room) {
  const int k0 = static_cast<int>(ceil_div(row_groups, room));
  double best = 0;
  int got = 1;
  for (int k = k0; k < k0 + 4; ++k) {
    const int blocks = k * room / row_groups;
    const double cost = static_cast<double>(k) / blocks * (1.0 + 0.02 * k);
    if (k == k0 || cost < best) {
      best = cost;
      got = blocks;
    }
  }
  return got;
}

// For `seqs` sequences; on all SMs, or with room for the own lists.
RowsPlan rows_plan(const pa_params_t* p, const pa_prefix_t* x, int seqs, bool all) {
  // The own lists' pass 1 runs beside this one.  16 to 76 work items of it (half
  // the SMs) get SMs of their own; fewer delay a few of this pass's CTAs less
  // than the SMs are worth, more would leave it too few.  Measured, all SMs
  // against this: 8 sequences, 4 KV heads of 256, prefix 8192 21.4 and 18.4 us,
  // 32000 41.3 and 34.8 us; with 1 sequence (4 items) 16.9 and 17.9 us.
  const int64_t own = static_cast<int64_t>(seqs) * p->num_kv_heads *
                      ceil_div(p->max_seq_len, p->partition_size);
  const int room = !all && own >= 16 && own <= kSms / 2 ? kSms - static_cast<int>(own) : kSms;
  RowsPlan r{};
  const int G = p->num_heads / p->num_kv_heads;
  r.shape = G <= 64 && (p->head_dim == 128 || p->head_dim == 256) && seqs > 0 &&
            !(p->flags & (PA_FLAG_PORTABLE | PA_FLAG_SPLIT_X)) && x->max_prefix_len > 0 &&
            (ceil_div(x->max_prefix_len, 128) + 152) * p->num_kv_heads < (int64_t(1) << 30);
  if (!r.shape) return r;
  r.row_tokens = 128 / G;
  r.dual = p->head_dim == 128 && seqs > r.row_tokens;
  r.lanes = p->head_dim == 128 && !r.dual ? 2 : 1;
  r.group_tokens = r.row_tokens * (r.dual ? 2 : 1);
  r.row_groups = static_cast<int>(ceil_div(seqs, r.group_tokens));
  // never more than all SMs would get, which is what the workspace has room for
  r.key_blocks = std::min(key_blocks(r.row_groups, room), key_blocks(r.row_groups, kSms));
  const int64_t tiles = ceil_div(x->max_prefix_len, 128);
  r.np = r.lanes * std::min<int64_t>(tiles, r.key_blocks / p->num_kv_heads + 2);
  return r;
}

// Control block | prefix partials (max, sum, output) | own partials.
struct PrefixLayout {
  int64_t np_prefix, np_own;  // slots of a row in each list
  size_t m[2], s[2], o[2], total;
};

PrefixLayout layout_of(const pa_params_t* p, const pa_prefix_t* x, int seqs) {
  PrefixLayout w;
  w.np_prefix = std::max<int64_t>(std::max<int64_t>(1, ceil_div(x->max_prefix_len, kPortablePart)),
                                  rows_plan(p, x, seqs, true).np);
  w.np_own = std::max<int64_t>(1, ceil_div(p->max_seq_len, p->partition_size));
  const size_t rows = static_cast<size_t>(seqs) * p->num_heads;
  size_t at = kCtrlBytes;
  const int64_t np[2] = {w.np_prefix, w.np_own};
  for (int i = 0; i < 2; ++i) {
    w.m[i] = at;
    at += up(rows * np[i] * 4);
    w.s[i] = at;
    at += up(rows * np[i] * 4);
    w.o[i] = at;
    at += up(rows * np[i] * p->head_dim * 4);
  }
  w.total = at;
  return w;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

size_t pa_prefix_workspace_size(const pa_params_t* p, const pa_prefix_t* prefix) {
  if (check_prefix(p, prefix) != PA_OK) return 0;
  size_t most = layout_of(p, prefix, p->num_seqs).total;
  // Fewer sequences may have more partials in all.  Between them only the number
  // of row tiles counts: so whole ones, of 128 / G sequences.
  const int step = std::max(128 / (p->num_heads / p->num_kv_heads), 1);
  if (rows_plan(p, prefix, p->num_seqs, true).shape)
    for (int64_t s = step; s < p->num_seqs; s += step)
      most = std::max(most, layout_of(p, prefix, static_cast<int>(s)).total);
  return most;
}

pa_status_t pa_decode_prefix(const pa_params_t* p, const pa_prefix_t* prefix, const void* q,
                             const void* k_cache, const void* v_cache,
                             const int32_t* prefix_blocks, const int32_t* prefix_len,
                             const int32_t* block_tables, const int32_t* seq_lens,
                             void* workspace, size_t workspace_bytes, void* out,
                             cudaStream_t stream) {
  if (pa_status_t st = check_prefix(p, prefix)) return st;
  if (p->num_seqs == 0) return PA_OK;
  if (pa_status_t st = check_tensors(q, k_cache, v_cache, block_tables, seq_lens, out)) return st;
  if (!prefix_len || (prefix->max_prefix_len && !prefix_blocks)) return PA_ERR_INVALID_ARG;
  if (!aligned(prefix_len, 4) || !aligned(prefix_blocks, 4)) return PA_ERR_MISALIGNED;
  if (!workspace) return PA_ERR_INVALID_ARG;
  if (!aligned(workspace, kAlign)) return PA_ERR_MISALIGNED;
  const PrefixLayout w = layout_of(p, prefix, p->num_seqs);
  if (workspace_bytes < w.total) return PA_ERR_WORKSPACE_TOO_SMALL;
  char* base = static_cast<char*>(workspace);
  int32_t* status = reinterpret_cast<int32_t*>(base);
  const auto at = [&](size_t off) { return reinterpret_cast<float*>(base + off); };
  JoinArgs j{};
  const RowsPlan r = rows_plan(p, prefix, p->num_seqs, false);
  const int sms = r.shape ? rows_applicable(p->kv_dtype, p->num_heads, p->num_kv_heads,
                                            p->head_dim, p->block_size, p->num_blocks, p->num_seqs,
                                            p->scale)
                          : 0;
  // short own lists: one kernel for them and the join, after the prefix
  const bool fused = own_applicable(p) && (sms > 0 || prefix->max_prefix_len == 0);

  // the sequences' own tokens
  if (!fused && p->max_seq_len > 0) {
    KernelArgs a = make_args(p, q, k_cache, v_cache, block_tables, seq_lens, out);
    a.status = status;
    a.max_logits = at(w.m[1]);
    a.exp_sums = at(w.s[1]);
    a.tmp_out = at(w.o[1]);
    a.num_partitions = static_cast<int32_t>(w.np_own);
    if (launch_pass(p, a, true, stream) != cudaSuccess) return PA_ERR_CUDA;
    JoinList& l = j.list[1];
    l.m = a.max_logits;
    l.s = a.exp_sums;
    l.o = a.tmp_out;
    l.part_size = p->partition_size;
  }
  j.list[1].lens = seq_lens;
  j.list[1].max_len = p->max_seq_len;
  j.list[1].stride = static_cast<int32_t>(w.np_own);

  // the shared prefix
  if (prefix->max_prefix_len > 0) {
    JoinList& l = j.list[0];
    l.m = at(w.m[0]);
    l.s = at(w.s[0]);
    l.o = at(w.o[0]);
    if (sms > 0) {
      RowsArgs a{};
      a.block_tables = prefix_blocks;
      a.lens = prefix_len;
      a.part_max = at(w.m[0]);
      a.part_sum = at(w.s[0]);
      a.part_out = at(w.o[0]);
      a.status = status;
      a.num_seqs = p->num_seqs;
      a.num_heads = p->num_heads;
      a.num_kv_heads = p->num_kv_heads;
      a.head_dim = p->head_dim;
      a.block_size = p->block_size;
      a.num_blocks = p->num_blocks;
      a.num_tokens = p->num_seqs;
      a.max_ctx_len = prefix->max_prefix_len;
      a.group = p->num_heads / p->num_kv_heads;
      a.row_tokens = r.row_tokens;
      a.group_tokens = r.group_tokens;
      a.row_groups = r.row_groups;
      a.dual = r.dual;
      a.key_blocks = r.key_blocks;
      a.num_parts = static_cast<int32_t>(r.np);
      a.selftest_stall = (p->flags & PA_FLAG_SELFTEST_STALL) ? 1 : 0;
      a.scale_log2 = p->scale * 1.442695040888963407360f;
      const RowsTensors t{q, nullptr, nullptr, k_cache, v_cache};
      // may start while the pass above still runs; it ends after it
      if (launch_rows(a, p->kv_dtype, t, sms, !fused && p->max_seq_len > 0, stream) != cudaSuccess)
        return PA_ERR_CUDA;
      l.stride = a.num_parts;
      l.key_blocks = r.key_blocks;
      l.lanes = r.lanes;
    } else {
      const int64_t parts = std::max<int64_t>(1, ceil_div(prefix->max_prefix_len, kPortablePart));
      if (parts > 65535) return PA_ERR_UNSUPPORTED;
      ListArgs a{};
      a.q = q;
      a.k_cache = k_cache;
      a.v_cache = v_cache;
      a.block_tables = prefix_blocks;
      a.lens = prefix_len;
      a.part_max = at(w.m[0]);
      a.part_sum = at(w.s[0]);
      a.part_out = at(w.o[0]);
      a.status = status;
      a.rows = p->num_seqs;
      a.mode = kPrefix;
      a.num_seqs = p->num_seqs;
      a.num_heads = p->num_heads;
      a.num_kv_heads = p->num_kv_heads;
      a.head_dim = p->head_dim;
      a.block_size = p->block_size;
      a.num_blocks = p->num_blocks;
      a.max_len = prefix->max_prefix_len;
      a.part_size = static_cast<int32_t>(kPortablePart);
      a.num_parts = static_cast<int32_t>(parts);
      a.always_partial = 1;
      a.group = p->num_heads / p->num_kv_heads;
      a.split_x = (p->flags & PA_FLAG_SPLIT_X) ? 1 : 0;
      a.scale_log2 = p->scale * 1.442695040888963407360f;
      cudaError_t e;
      switch (p->kv_dtype) {
        case PA_F32: e = launch_portable_f32(a, stream); break;
        case PA_BF16: e = launch_portable_bf16(a, stream); break;
        default: e = launch_portable_f16(a, stream); break;
      }
      if (e != cudaSuccess) return PA_ERR_CUDA;
      l.stride = a.num_parts;
      l.part_size = a.part_size;
    }
  }
  j.list[0].lens = prefix_len;
  j.list[0].shared = 1;
  j.list[0].max_len = prefix->max_prefix_len;
  if (fused) {
    KernelArgs a = make_args(p, q, k_cache, v_cache, block_tables, seq_lens, out);
    a.status = status;
    return launch_own(a, j.list[0], p->kv_dtype, prefix->max_prefix_len > 0, stream) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
  }
  j.out = out;
  j.status = status;
  j.num_rows = static_cast<int64_t>(p->num_seqs) * p->num_heads;
  j.num_heads = p->num_heads;
  j.head_dim = p->head_dim;
  j.group = p->num_heads / p->num_kv_heads;
  j.out_dtype = p->out_dtype;
  // a dependent of the kernels above, which read the same lengths; where none ran
  // the kernel before may be the caller's, which still writes them
  const bool dependent = j.list[0].m || j.list[1].m;
  return launch_join(j, stream, dependent) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"
