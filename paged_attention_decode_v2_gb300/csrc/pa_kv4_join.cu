// pa_kv4_join.cu -- joins the parts of a row of pa_decode_kv4: the second launch of calls
// whose rows may have several.
//
// A part has its maximum m_p (base 2), the sum s_p of 2^(l - m_p) and its normalised output
// o_p, and with M = max m_p, w_p = 2^(m_p - M) s_p the row is sum w_p o_p / sum w_p.  A NaN
// maximum (a bad page) or sum (a NaN logit) makes it NaN; a row without a token is zeros.
// Rows of one part were written by the kernel before and are left alone.
//
// `warps` warps a row (every warps-th part is a warp's, four of its loads in flight), eight
// in a CTA.  The sums run in a fixed order.  Bound by latency: this kernel begins when the
// other has ended, and then waits for the parts' length and for the parts.  Where there are
// few rows, the first parts are loaded beside the length, before it is known how many there
// are (0.2 us).  Measured as what calls take beyond the first kernel: one sequence of 4000,
// 24 / 4 heads of 256, 2.8 us, 100K 3.5; 256 up to 16000, 32 / 8 of 128, 4.3; 500 of 1200, whose
// 16000 rows have one part each, 3.8 (a CTA a row 8.5; CTAs that take several rows in turn
// 6); eight warps a row where there are 8192 rows cost 13 us more than one.
#include <algorithm>

#include "pa_kv4.cuh"

namespace pa {

namespace {

constexpr int kWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kWarps) pa_kv4_join_kernel(const Kv4Args a, const int warps,
                                                                  const bool ahead) {
  constexpr int E = D / 32, kBatch = 4;
  __shared__ float acc_s[kWarps][D];
  __shared__ float m_s[kWarps], w_s[kWarps];
  const int lane = threadIdx.x & 31, all = threadIdx.x >> 5;
  const int warp = all & (warps - 1), first = all - warp;  // of the row's; the row's first
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * kWarps + all) / warps;
  if (row >= static_cast<int64_t>(a.num_seqs) * a.num_heads) return;
  // lengths are inputs of the call: read before the parts are waited for
  const int32_t L = __ldg(a.lens + row / a.num_heads);
  const bool ok = kv4_len_ok(a, L);
  cudaGridDependencySynchronize();

  // Parts base, base + warps, ...: element e of a lane is column (e / 4) * 128 + lane * 4 + e % 4
  // (2 * lane + e for D = 64).  Coherent loads: they were written while this kernel waited.
  float mp[kBatch], sp[kBatch], o[kBatch][E];
  const auto load = [&](int base, int end) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int p = base + i * warps;
      mp[i] = -INFINITY;
      sp[i] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[i][e] = 0.f;
      if (p >= end) continue;
      const int64_t at = row * a.num_parts + p;
      mp[i] = __ldcg(a.part_max + at);
      sp[i] = __ldcg(a.part_sum + at);
      if constexpr (E == 2) {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(a.part_out + at * D) + lane);
        o[i][0] = v.x;
        o[i][1] = v.y;
      } else {
#pragma unroll
        for (int g = 0; g < E / 4; ++g) {
          const float4 v =
              __ldcg(reinterpret_cast<const float4*>(a.part_out + at * D) + g * 32 + lane);
          o[i][4 * g] = v.x;
          o[i][4 * g + 1] = v.y;
          o[i][4 * g + 2] = v.z;
          o[i][4 * g + 3] = v.w;
        }
      }
    }
  };
  if (ahead) load(warp, a.num_parts);  // slots of the row, whether they are used or not
  const int32_t size = a.part_at ? __ldcg(a.part_at) : a.part_size;
  if (a.part_at && ok && L > 0 && L <= size) return;
  const int n = ok ? static_cast<int>((static_cast<uint32_t>(L) + size - 1) / size) : 0;
  if (!ahead) load(warp, n);

  float m = -INFINITY, w = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  bool nan_seen = !ok;
  for (int base = warp; base < n;) {
    float mb = m;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (base + i * warps >= n) mp[i] = -INFINITY, sp[i] = 0.f;  // loaded ahead
      nan_seen |= isnan(mp[i]) || isnan(sp[i]);
      mb = fmaxf(mb, mp[i]);
    }
    if (mb > m) {
      const float f = exp2f(m - mb);  // 0 when m is -inf
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= f;
      w *= f;
      m = mb;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (mp[i] == -INFINITY) continue;
      const float c = sp[i] * exp2f(mp[i] - m);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(c, o[i][e], acc[e]);
      w += c;
    }
    base += warps * kBatch;
    if (base < n) load(base, n);
  }
  if (nan_seen) m = qnan();
  if (warps > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) acc_s[all][e * 32 + lane] = acc[e];
    if (lane == 0) {
      m_s[all] = m;
      w_s[all] = w;
    }
    __syncthreads();  // of the threads that are still here
    if (warp) return;
    m = -INFINITY;
    bool nan_any = false;
    for (int q = first; q < first + warps; ++q) {
      nan_any |= isnan(m_s[q]);
      m = fmaxf(m, m_s[q]);
    }
    w = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int q = first; q < first + warps; ++q) {
      const float f = m_s[q] == -INFINITY ? 0.f : exp2f(m_s[q] - m);
      w = fmaf(w_s[q], f, w);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(acc_s[q][e * 32 + lane], f, acc[e]);
    }
    if (nan_any) m = qnan();
  }
  const float inv = isnan(m) ? qnan() : w > 0.f ? 1.f / w : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] *= inv;
  if constexpr (E == 2) {
    store_out(a.out, row * D + 2 * lane, a.out_dtype, acc[0]);
    store_out(a.out, row * D + 2 * lane + 1, a.out_dtype, acc[1]);
  } else {
#pragma unroll
    for (int g = 0; g < E / 4; ++g)
      store_out4(a.out, row * D + g * 128 + 4 * lane, a.out_dtype,
                 make_float4(acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]));
  }
}

}  // namespace

cudaError_t launch_kv4_join(const Kv4Args& a, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.num_seqs) * a.num_heads;
  // a warp for every four parts that a row can have, up to eight, while the SMs hold them all
  // at once
  const int64_t room = 64LL * std::max(sm100_num_sms(), 1);
  int warps = 1;
  while (warps < kWarps && warps * 4 < a.num_parts && 2 * warps * rows <= room) warps *= 2;
  const bool ahead = rows * kWarps <= room;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((rows * warps + kWarps - 1) / kWarps), 1, 1);
  cfg.blockDim = dim3(32 * kWarps, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto kern = a.head_dim == 64    ? pa_kv4_join_kernel<64>
                    : a.head_dim == 128 ? pa_kv4_join_kernel<128>
                                        : pa_kv4_join_kernel<256>;
  return cudaLaunchKernelEx(&cfg, kern, a, warps, ahead);
}

}  // namespace pa
