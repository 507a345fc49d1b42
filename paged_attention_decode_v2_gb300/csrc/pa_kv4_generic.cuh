// pa_kv4_generic.cuh -- CUDA-core decode over the 4-bit cache: every element type,
// head_dim, group size, block size and head layout of pa_decode_kv4.
//
// A CTA takes one (part of a sequence, KV head, up to eight of its query heads);
// its eight warps take tokens in turn.  A lane holds D / 32 elements of a token's
// key and value, widened once for all heads; a logit is a butterfly over the
// lanes, and every warp keeps its own running maxima, sums and weighted values,
// all float32, joined in shared memory at the end.  A part that is the whole
// sequence writes its output, others a partial for pa_kv4_join.cu.
// Bound by instructions: 4 D operations a token and head, and a butterfly.  Measured, bf16:
// one sequence of 100K, 24 / 4 heads of 256, 562 us (tensor cores 32); 256 sequences up to
// 100K, 32 / 8 of 128, 12.1 ms (627 us).
#pragma once

#include "pa_kv4.cuh"

namespace pa {

template <typename T, int D>
__global__ void __launch_bounds__(256) pa_kv4_generic_kernel(const Kv4Args a) {
  constexpr int E = D / 32, HP = kKv4Heads, kWarps = 8;
  constexpr unsigned kAll = 0xffffffffu;
  __shared__ float acc_s[kWarps][D];
  __shared__ float m_s[kWarps][HP], s_s[kWarps][HP];
  __shared__ int bad_s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = blockIdx.x, b = blockIdx.z;
  const int kvh = blockIdx.y / a.head_groups, hg = blockIdx.y % a.head_groups;
  const int nh = min(HP, a.group - hg * HP);           // query heads of this CTA
  const int h0 = kvh * a.group + hg * HP;
  const int32_t L = __ldg(a.lens + b);
  const bool ok = kv4_len_ok(a, L);
  if (!ok && threadIdx.x == 0 && part == 0) set_status(a.status, PA_ERR_BAD_SEQ_LEN);
  const int32_t t0 = part * a.part_size;
  // not past 31 bits in the last part of the longest rows
  const int32_t t1 = !ok ? 0 : L - t0 > a.part_size ? t0 + a.part_size : L;
  const bool direct = a.num_parts == 1;
  if (t0 >= t1 && !direct) return;                     // the join knows these rows' lengths
  if (threadIdx.x == 0) bad_s = !ok;
  __syncthreads();

  float q[HP][E];
#pragma unroll
  for (int h = 0; h < HP; ++h)
#pragma unroll
    for (int e = 0; e < E; ++e)
      q[h][e] = h < nh ? to_float(static_cast<const T*>(
                             a.q)[(static_cast<int64_t>(b) * a.num_heads + h0 + h) * D +
                                  lane * E + e]) * a.scale_log2
                       : 0.f;
  float m[HP], s[HP], acc[HP][E];
#pragma unroll
  for (int h = 0; h < HP; ++h) {
    m[h] = -INFINITY;
    s[h] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[h][e] = 0.f;
  }
  const int32_t* table = a.block_tables + static_cast<int64_t>(b) * a.max_blocks_per_seq;
  const int per = D / a.group_size, own = lane * E / a.group_size;
  // the lane's elements of a row of a pool, widened
  const auto widen = [&](const uint8_t* codes, const void* pairs, int64_t row, float (&x)[E]) {
    const uint8_t* c = codes + row * (D / 2) + lane * E / 2;
    uint32_t w;
    if constexpr (E == 2) w = __ldg(c);
    else if constexpr (E == 4) w = __ldg(reinterpret_cast<const uint16_t*>(c));
    else w = __ldg(reinterpret_cast<const uint32_t*>(c));
    const float2 p = load_pair<T>(pairs, row * per + own);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = fmaf(static_cast<float>(w >> (4 * e) & 15), p.x, p.y);
  };
  for (int32_t t = t0 + warp; t < t1; t += kWarps) {
    const int32_t block = __ldg(table + t / a.block_size);
    if (block < 0 || block >= a.num_blocks) {
      if (lane == 0) bad_s = 2;
      continue;
    }
    const int64_t row =
        (static_cast<int64_t>(block) * a.num_kv_heads + kvh) * a.block_size + t % a.block_size;
    float k[E], v[E];
    widen(a.k_codes, a.k_pairs, row, k);
    widen(a.v_codes, a.v_pairs, row, v);
#pragma unroll
    for (int h = 0; h < HP; ++h) {
      if (h >= nh) break;
      float l = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) l = fmaf(q[h][e], k[e], l);
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(kAll, l, o);
      if (l > m[h]) {  // the same in all lanes
        const float f = exp2f(m[h] - l);
        m[h] = l;
        s[h] *= f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[h][e] *= f;
      }
      // a NaN logit makes p NaN; where none has been larger than -inf the
      // difference is NaN too, which only logits that are not finite can cause
      const float p = exp2f(l - m[h]);
      s[h] += p;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[h][e] = fmaf(p, v[e], acc[h][e]);
    }
  }
  if (lane == 0)
#pragma unroll
    for (int h = 0; h < HP; ++h) {
      m_s[warp][h] = m[h];
      s_s[warp][h] = s[h];
    }
#pragma unroll
  for (int h = 0; h < HP; ++h) {
    if (h >= nh) break;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) acc_s[warp][lane * E + e] = acc[h][e];
    __syncthreads();
    if (threadIdx.x >= D) continue;
    float M = -INFINITY, sum = 0.f, o = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, m_s[w][h]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      // a warp without a token has a maximum of -inf, a sum of 0 and weighs nothing
      const float f = m_s[w][h] == -INFINITY ? (s_s[w][h] == 0.f ? 0.f : qnan())
                                             : exp2f(m_s[w][h] - M);
      sum = fmaf(s_s[w][h], f, sum);
      o = fmaf(acc_s[w][threadIdx.x], f, o);
    }
    kv4_finish(a, b, h0 + h, part, threadIdx.x, D, direct, L, bad_s, M, sum, o);
  }
  if (bad_s == 2 && threadIdx.x == 0) set_status(a.status, PA_ERR_BAD_BLOCK_ID);
}

template <typename T>
cudaError_t launch_kv4_generic(const Kv4Args& a, cudaStream_t s) {
  const dim3 grid(a.num_parts, a.num_kv_heads * a.head_groups, a.num_seqs);
  switch (a.head_dim) {
    case 64: pa_kv4_generic_kernel<T, 64><<<grid, 256, 0, s>>>(a); break;
    case 128: pa_kv4_generic_kernel<T, 128><<<grid, 256, 0, s>>>(a); break;
    default: pa_kv4_generic_kernel<T, 256><<<grid, 256, 0, s>>>(a); break;
  }
  return cudaGetLastError();
}

}  // namespace pa
