// pa_portable.cuh -- CUDA-core attention of one query row over a list of
// tokens, for the windowed and shared-prefix calls: every element type,
// head_dim, block size, group and cache layout that the decode calls take.
//
// One CTA handles one (row, KV head, part of the row's list): a row is a
// sequence (decode) or a token of a chunk (prefill).  The list is
//   kDecodeWindow   the sinks below the window, then the window's tokens;
//   kPrefillWindow  the same at the row's position, with tokens from ctx_lens
//                   on taken from the chunk's dense keys and values;
//   kPrefix         the tokens of the shared prefix.
// It is walked in chunks of 256 tokens as in pa_generic.cuh: the chunk's
// places first (block-table entries, one thread per token), then QK^T with
// lanes splitting head_dim, the running softmax with one warp per head, and
// P.V with warps splitting head_dim and lanes splitting tokens.  All G query
// heads of the KV head share each key and value, eight at a time.
//
// A row of one part writes its output; longer rows write partials
// (max in natural-log units, sum, normalised output) that pa_join.cu joins.
// Bound by instructions, 4 D operations a token and head on the CUDA cores, as
// the decode calls' portable kernel is.  Measured, bf16 on the cases that the
// tensor-core kernels serve: 256 sequences, 8 KV heads of 128, window 1024
// 757 us (tensor cores 125); a windowed chunk of 4096 tokens, 24 / 4 heads of
// 256, 15.8 ms (174 us).
#pragma once

#include "pa_generic.cuh"
#include "pa_span.cuh"

namespace pa {

struct ListSmem {
  int64_t slice[256];  // element offset of the token's (block, KV head) slice, or of its dense row
  int32_t slot[256];   // its place in the block; -1: dense row; -2: bad block, not read
};

template <typename T, int D>
__global__ void __launch_bounds__(256) pa_portable_kernel(const ListArgs a) {
  using C = GenericCfg<T, D>;
  __shared__ GenericSmem<D> sm;
  __shared__ ListSmem ls;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x;
  const int kvh = blockIdx.y, part = blockIdx.z;
  const int BS = a.block_size, G = a.group, Hq = a.num_heads;

  // ---- the row's list ------------------------------------------------------
  int seq = 0;                // block-table row
  int32_t n_low = 0, lo = 0;  // list token u is token u (u < n_low) or lo + u - n_low
  int32_t n = 0;              // tokens of the list
  int32_t ctx = INT32_MAX;    // tokens from here on are chunk rows
  int64_t chunk0 = 0;         //   chunk row of token ctx
  bool ok = true;
  if (a.mode == kPrefix) {
    n = a.lens[0];
    ok = n >= 0 && n <= a.max_len;
  } else {
    int32_t L;                // tokens up to and including the query
    if (a.mode == kDecodeWindow) {
      seq = static_cast<int>(row);
      L = a.lens[seq];
      ok = L >= 0 && L <= a.max_len;
    } else {
      int x = 0, z = a.num_seqs;  // last sequence that starts at or before the row
      while (z - x > 1) {
        const int m = (x + z) >> 1;
        if (a.query_start[m] <= row) x = m;
        else z = m;
      }
      seq = x;
      const int32_t s0 = a.query_start[seq], s1 = a.query_start[seq + 1];
      // rows of no sequence, or of a chunk that cannot be trusted, stay as they are
      if (s0 < 0 || row < s0 || row >= s1 || s1 > a.total_tokens || s1 - s0 > a.max_query_len)
        return;
      ctx = a.lens[seq];
      ok = ctx >= 0 && ctx <= a.max_len &&
           ctx <= static_cast<int64_t>(a.max_blocks_per_seq) * BS;
      chunk0 = s0;
      L = ok ? ctx + static_cast<int32_t>(row - s0) + 1 : 0;
    }
    if (ok) {
      lo = L > a.window ? L - a.window : 0;
      n_low = min(a.num_sinks, lo);
      n = L - lo + n_low;
    }
  }
  if (!ok) {
    if (tid == 0) set_status(a.status, PA_ERR_BAD_SEQ_LEN);
    n = 0;
  }
  const bool partial = a.num_parts > 1 || a.always_partial;
  const int32_t u0 = a.num_parts > 1 ? part * a.part_size : 0;
  const int32_t u1 = a.num_parts > 1 ? min(n, u0 + a.part_size) : n;
  if (u0 >= u1 && part > 0) return;  // no such part

  const T* __restrict__ kc = static_cast<const T*>(a.k_cache);
  const T* __restrict__ vc = static_cast<const T*>(a.v_cache);
  const T* __restrict__ kn = static_cast<const T*>(a.k_new);
  const T* __restrict__ vn = static_cast<const T*>(a.v_new);
  const T* __restrict__ qp = static_cast<const T*>(a.q);
  const int32_t* __restrict__ bt =
      a.block_tables + static_cast<int64_t>(seq) * a.max_blocks_per_seq;

  for (int hg = 0; hg * C::HP < G; ++hg) {
    const int nh = min(C::HP, G - hg * C::HP);
    const int h0 = kvh * G + hg * C::HP;
    for (int i = tid; i < C::HP * D; i += C::NT) {
      const int hh = i / D, d = i % D;
      sm.q[hh][d] = hh < nh ? to_float(qp[(row * Hq + h0 + hh) * D + d]) * a.scale_log2 : 0.f;
      sm.acc[hh][d] = 0.f;
    }
    if (tid < C::HP) {
      sm.m_run[tid] = -INFINITY;
      sm.s_run[tid] = 0.f;
    }
    if (tid == 0) sm.bad = ok ? 0 : 1;
    __syncthreads();

    for (int32_t c0 = u0; c0 < u1; c0 += C::CH) {
      const int nt = min(C::CH, u1 - c0);
      if (tid < nt) {
        const int32_t u = c0 + tid;
        const int32_t t = u < n_low ? u : lo + (u - n_low);
        if (t >= ctx) {
          ls.slice[tid] = ((chunk0 + (t - ctx)) * a.num_kv_heads + kvh) * D;
          ls.slot[tid] = -1;
        } else {
          const int32_t id = bt[t / BS];
          if (id < 0 || id >= a.num_blocks) {
            sm.bad = 1;
            set_status(a.status, PA_ERR_BAD_BLOCK_ID);
            ls.slot[tid] = -2;
          } else {
            ls.slice[tid] = (static_cast<int64_t>(id) * a.num_kv_heads + kvh) * BS * D;
            ls.slot[tid] = t % BS;
          }
        }
      }
      __syncthreads();

      // ---- QK^T ------------------------------------------------------------
      for (int base = warp * C::U; base < nt; base += C::NW * C::U) {
        float kf[C::U][C::EPL];
#pragma unroll
        for (int u = 0; u < C::U; ++u) {
          const int tt = base + u;
          const int32_t slot = tt < nt ? ls.slot[tt] : -2;
          if (slot == -2) {
#pragma unroll
            for (int e = 0; e < C::EPL; ++e) kf[u][e] = 0.f;
          } else if (slot == -1) {
            load_row<T, C::EPL>(kn + ls.slice[tt] + lane * C::EPL, kf[u]);
          } else if (!a.split_x) {
            load_row<T, C::EPL>(kc + ls.slice[tt] + static_cast<int64_t>(slot) * D + lane * C::EPL,
                                kf[u]);
          } else {
#pragma unroll
            for (int g = 0; g < C::EPL / C::KG; ++g) {
              const int d = lane * C::EPL + g * C::KG;
              float f[C::KG];
              load_row<T, C::KG>(kc + ls.slice[tt] +
                                     (static_cast<int64_t>(d / C::X) * BS + slot) * C::X + d % C::X,
                                 f);
#pragma unroll
              for (int e = 0; e < C::KG; ++e) kf[u][g * C::KG + e] = f[e];
            }
          }
        }
        float part_sum[32];
#pragma unroll
        for (int h = 0; h < C::HP; ++h) {
          float qv[C::EPL];
#pragma unroll
          for (int e = 0; e < C::EPL; ++e) qv[e] = sm.q[h][lane * C::EPL + e];
#pragma unroll
          for (int u = 0; u < C::U; ++u) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < C::EPL; ++e) s = fmaf(qv[e], kf[u][e], s);
            part_sum[u * C::HP + h] = s;
          }
        }
        const float logit = reduce_scatter32(part_sum, lane);
        const int tt = base + lane / C::HP;
        if (tt < nt) sm.p[tt][lane % C::HP] = ls.slot[tt] == -2 ? -INFINITY : logit;
      }
      __syncthreads();

      // ---- running softmax: warp h owns head h -------------------------------
      {
        const int h = warp;
        float mx = -INFINITY;
        for (int tt = lane; tt < nt; tt += 32) mx = fmaxf(mx, sm.p[tt][h]);
        mx = warp_max(mx);
        const float m_old = sm.m_run[h];
        const float m_new = fmaxf(m_old, mx);
        float sum = 0.f;
        for (int tt = lane; tt < nt; tt += 32) {
          // a NaN logit goes on into the sum, also where none is above -inf
          const float l = sm.p[tt][h];
          const float pv =
              l == -INFINITY ? 0.f : exp2f(l - (m_new == -INFINITY ? 0.f : m_new));
          sm.p[tt][h] = pv;
          sum += pv;
        }
        sum = warp_sum(sum);
        if (lane == 0) {
          const float f = m_new == -INFINITY ? 1.f : exp2f(m_old - m_new);
          sm.factor[h] = f;
          sm.s_run[h] = sm.s_run[h] * f + sum;
          sm.m_run[h] = m_new;
        }
      }
      __syncthreads();

      // ---- P.V: warp owns a head_dim slice, lanes split tokens ----------------
      {
        const int tl = lane / C::LPT, vi = lane % C::LPT;
        const int d0 = warp * C::WSLICE + vi * C::VEC;
        float acc[C::HP][C::VEC];
#pragma unroll
        for (int h = 0; h < C::HP; ++h)
#pragma unroll
          for (int e = 0; e < C::VEC; ++e) acc[h][e] = 0.f;
        for (int tt = tl; tt < nt; tt += C::TPS) {
          const int32_t slot = ls.slot[tt];
          if (slot == -2) continue;
          float vf[C::VEC];
          if (slot == -1) {
            load_row<T, C::VEC>(vn + ls.slice[tt] + d0, vf);
          } else if (!a.split_x) {
            load_row<T, C::VEC>(vc + ls.slice[tt] + static_cast<int64_t>(slot) * D + d0, vf);
          } else {
#pragma unroll
            for (int e = 0; e < C::VEC; ++e)
              vf[e] = to_float(vc[ls.slice[tt] + static_cast<int64_t>(d0 + e) * BS + slot]);
          }
          const float4 pa4 = *reinterpret_cast<const float4*>(&sm.p[tt][0]);
          const float4 pb4 = *reinterpret_cast<const float4*>(&sm.p[tt][4]);
          const float pp[8] = {pa4.x, pa4.y, pa4.z, pa4.w, pb4.x, pb4.y, pb4.z, pb4.w};
#pragma unroll
          for (int h = 0; h < C::HP; ++h)
#pragma unroll
            for (int e = 0; e < C::VEC; ++e) acc[h][e] = fmaf(pp[h], vf[e], acc[h][e]);
        }
#pragma unroll
        for (int o = C::LPT; o < 32; o <<= 1)
#pragma unroll
          for (int h = 0; h < C::HP; ++h)
#pragma unroll
            for (int e = 0; e < C::VEC; ++e)
              acc[h][e] += __shfl_xor_sync(0xffffffffu, acc[h][e], o);
        if (tl == 0) {
#pragma unroll
          for (int h = 0; h < C::HP; ++h)
#pragma unroll
            for (int e = 0; e < C::VEC; ++e)
              sm.acc[h][d0 + e] = sm.acc[h][d0 + e] * sm.factor[h] + acc[h][e];
        }
      }
      __syncthreads();
    }

    // ---- epilogue ---------------------------------------------------------
    const bool bad = sm.bad != 0;
    for (int i = tid; i < nh * D; i += C::NT) {
      const int hh = i / D, d = i % D;
      const float s = sm.s_run[hh];
      const float o = bad ? qnan() : (s == 0.f ? 0.f : sm.acc[hh][d] / s);
      const int64_t r = row * Hq + h0 + hh;
      if (partial)
        a.part_out[(r * a.num_parts + part) * D + d] = o;
      else
        store_out(a.out, r * D + d, a.out_dtype, o);
    }
    if (partial && tid < nh) {
      const int64_t w = (row * Hq + h0 + tid) * a.num_parts + part;
      a.part_max[w] = bad ? qnan() : sm.m_run[tid] * kLn2;
      a.part_sum[w] = sm.s_run[tid];
    }
    __syncthreads();
  }
}

template <typename T, int D>
cudaError_t launch_portable_d(const ListArgs& a, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.rows), a.num_kv_heads, a.num_parts);
  pa_portable_kernel<T, D><<<grid, GenericCfg<T, D>::NT, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_portable_t(const ListArgs& a, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  switch (a.head_dim) {
    case 64: return launch_portable_d<T, 64>(a, s);
    case 128: return launch_portable_d<T, 128>(a, s);
    case 256: return launch_portable_d<T, 256>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pa
