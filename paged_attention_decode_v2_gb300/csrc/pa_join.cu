// pa_join.cu -- joins the partial results of a query row: the last kernel of
// the windowed and shared-prefix decode calls.
//
// A row (sequence, query head) has up to two lists of partials (max m_p in
// natural-log units, sum s_p of exp(l - m_p), normalised output o_p), and
//   M = max m_p,  w_p = exp(m_p - M) s_p,  out = sum w_p o_p / sum w_p
// over both: the log-sum-exp identity of the V2 reduce.  An empty partial has
// m_p = -inf and s_p = 0 and weighs nothing; a NaN max (a bad block) or a NaN
// sum (a NaN logit, beside a max of -inf where all are) makes the row NaN; a row
// without a token is zeros.
//
// One CTA of `warps` warps per row; a warp folds every warps-th partial, four
// loads in flight, D / 32 output elements a lane, and the warps are joined in
// shared memory.  The sums run in a fixed order.  Bound by the partials' bytes
// (they are in L2, written just before) or, for few rows, by latency.  Measured
// alone with cold caches (in the calls they are warm and the launch overlaps):
// 8192 rows of 128 with 28 MB of partials 18.9 us, 24 rows of 256 6.6 us.  Two,
// four or eight rows in a CTA changed whole calls by less than 1.5 %.
#include "pa_device.cuh"
#include "pa_span.cuh"

namespace pa {

namespace {

constexpr int kMaxWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kMaxWarps) pa_join_kernel(const JoinArgs a) {
  constexpr int E = D / 32;
  __shared__ float acc_s[kMaxWarps][D];
  __shared__ float m_s[kMaxWarps], w_s[kMaxWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t row = blockIdx.x;
  const int b = static_cast<int>(row / a.num_heads);

  // partials of the row in each list, from the lengths (inputs, so they are
  // read before the passes' results are waited for)
  int n[2] = {0, 0};
  bool ok = true;
  for (int l = 0; l < 2; ++l) {
    const JoinList& x = a.list[l];
    if (!x.lens) continue;
    int32_t L = __ldg(x.lens + (x.shared ? 0 : b));
    const bool in = L >= 0 && L <= x.max_len;
    // a list with partials had its length checked by the kernel that made them
    if (!in && !x.m && threadIdx.x == 0) set_status(a.status, PA_ERR_BAD_SEQ_LEN);
    ok = ok && in;
    if (!ok || !x.m) continue;
    if (x.window > 0) {
      if (x.block_list) {
        L = window_span(L, x.window, x.num_sinks, x.block_size).len;
      } else {
        const int32_t lo = L > x.window ? L - x.window : 0;
        L = L - lo + min(x.num_sinks, lo);
      }
    }
    if (x.key_blocks > 0) {
      const int kvh = static_cast<int>(row % a.num_heads) / a.group;
      n[l] = prefix_split(L, a.num_heads / a.group, x.key_blocks).segments(kvh) * x.lanes;
    } else {
      n[l] = (L + x.part_size - 1) / x.part_size;
    }
  }
  // The partials were written while this kernel ran: coherent loads, no __ldg.
  cudaGridDependencySynchronize();

  float m = -INFINITY, w = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  bool nan_seen = !ok;
  for (int l = 0; l < 2 && ok; ++l) {
    const JoinList& x = a.list[l];
    const int64_t r = row * x.stride;
    constexpr int kBatch = 4;
    for (int base = warp; base < n[l]; base += warps * kBatch) {
      float mp[kBatch], sp[kBatch], o[kBatch][E];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int p = base + i * warps;
        mp[i] = -INFINITY;
        sp[i] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[i][e] = 0.f;
        if (p < n[l]) {
          const int64_t at = r + p;
          mp[i] = __ldcg(x.m + at);
          sp[i] = __ldcg(x.s + at);
          if constexpr (E == 2) {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(x.o + at * D) + lane);
            o[i][0] = v.x;
            o[i][1] = v.y;
          } else {
#pragma unroll
            for (int g = 0; g < E / 4; ++g) {
              const float4 v =
                  __ldcg(reinterpret_cast<const float4*>(x.o + at * D) + g * 32 + lane);
              o[i][4 * g] = v.x;
              o[i][4 * g + 1] = v.y;
              o[i][4 * g + 2] = v.z;
              o[i][4 * g + 3] = v.w;
            }
          }
        }
      }
      float mb = m;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        nan_seen |= isnan(mp[i]) || isnan(sp[i]);
        mb = fmaxf(mb, mp[i]);
      }
      if (mb > m) {
        const float f = expf(m - mb);  // 0 when m is -inf
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= f;
        w *= f;
        m = mb;
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (mp[i] == -INFINITY) continue;
        const float c = sp[i] * expf(mp[i] - m);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(c, o[i][e], acc[e]);
        w += c;
      }
    }
  }
  if (nan_seen) m = qnan();
  if (warps > 1) {
    // element e of lane: column (e / 4) * 128 + lane * 4 + e % 4 (2 * lane + e for D = 64)
#pragma unroll
    for (int e = 0; e < E; ++e) acc_s[warp][e * 32 + lane] = acc[e];
    if (lane == 0) {
      m_s[warp] = m;
      w_s[warp] = w;
    }
    __syncthreads();
    if (warp) return;
    m = -INFINITY;
    bool nan_any = false;
    for (int q = 0; q < warps; ++q) {
      nan_any |= isnan(m_s[q]);
      m = fmaxf(m, m_s[q]);
    }
    w = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int q = 0; q < warps; ++q) {
      const float f = m_s[q] == -INFINITY ? 0.f : expf(m_s[q] - m);
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

template <int D>
cudaError_t launch_join_d(const JoinArgs& a, cudaStream_t s, bool pdl) {
  // a warp for every four partials that a row can have, up to eight
  int most = 0;
  for (const JoinList& x : a.list) most += x.m ? x.stride : 0;
  int warps = 1;
  while (warps < kMaxWarps && warps * 4 < most) warps *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.num_rows), 1, 1);
  cfg.blockDim = dim3(32 * warps, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, pa_join_kernel<D>, a);
}

}  // namespace

cudaError_t launch_join(const JoinArgs& a, cudaStream_t s, bool pdl) {
  if (a.num_rows == 0) return cudaSuccess;
  switch (a.head_dim) {
    case 64: return launch_join_d<64>(a, s, pdl);
    case 128: return launch_join_d<128>(a, s, pdl);
    case 256: return launch_join_d<256>(a, s, pdl);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pa
