// pa_own.cu -- the last kernel of pa_decode_prefix where the sequences' own
// lists are short: attention over the own tokens and the join with the prefix
// pass's partials in one launch.
//
// One CTA per (sequence, KV head), four warps (eight for head_dim 256: two per
// token group, each with half of the values' columns).  Lists of a few hundred
// tokens are bound by latency, not by bandwidth: so there is no staging, no
// pipeline between roles and no barrier until the end -- each warp takes every
// fourth group of 16 tokens with 16-byte loads straight into the operands of
// warp-level MMAs, and thousands of such warps keep the memory busy.
//   S[h, t]  = sum_d q[h, d] K[t, d]   m16n8k16: the G <= 8 heads are rows 0..7;
//              a thread's 16-byte piece of a row is the operand of two MMAs (the
//              order of d within the sum is free, and the same for q and K);
//   O[h, d] += sum_t p[h, t] V[t, d]   rows 0..7 of A hold p's 16-bit part, rows
//              8..15 the rounded remainder, so p keeps ~16 significant bits; B's
//              column of 8 output elements is spread over threads that hold 8
//              neighbouring d each, and pairs of tokens are put together by byte
//              permutation.
// The reference maximum of a warp moves as in pa_rows.cuh.  At the end the
// warps' and the prefix's partials are joined by log-sum-exp in shared memory.
#include <cstdint>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_span.cuh"

namespace pa {

namespace {

constexpr int kGroups = 4;           // token groups: warps, or pairs of warps
constexpr float kRescaleLog2 = 8.f;  // the reference maximum moves past 2^8 only

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two probabilities as a 16-bit pair and the pair of rounded remainders.
template <typename T>
__device__ __forceinline__ void split_pair(float p0, float p1, uint32_t& hi, uint32_t& lo) {
  const T h0 = round16(p0, static_cast<T*>(nullptr)), h1 = round16(p1, static_cast<T*>(nullptr));
  const T l0 = round16(p0 - to_float(h0), static_cast<T*>(nullptr));
  const T l1 = round16(p1 - to_float(h1), static_cast<T*>(nullptr));
  hi = bits16(h0) | (static_cast<uint32_t>(bits16(h1)) << 16);
  lo = bits16(l0) | (static_cast<uint32_t>(bits16(l1)) << 16);
}

template <typename T, int D>
__global__ void __launch_bounds__(D, 512 / D)
    pa_own_kernel(const KernelArgs a, const JoinList pre) {
  constexpr int kPieces = D / 32;             // 16-byte pieces of a row per thread (QK^T)
  __shared__ float o_s[kGroups][8][D];
  __shared__ float m_s[kGroups][8], s_s[kGroups][8];
  __shared__ int bad_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int grp = warp % kGroups, half = warp / kGroups;
  const int G = a.group, Hq = a.num_heads, BS = a.block_size;
  const int kvh = blockIdx.x % a.num_kv_heads, b = blockIdx.x / a.num_kv_heads;
  const int row = lane >> 2, c = lane & 3;
  if (tid == 0) bad_s = 0;
  __syncthreads();

  const int32_t L = __ldg(a.seq_lens + b);
  const bool ok = seq_len_ok(a, L);
  const int32_t n = ok ? L : 0;
  const T* __restrict__ kc = static_cast<const T*>(a.k_cache);
  const T* __restrict__ vc = static_cast<const T*>(a.v_cache);
  const int32_t* __restrict__ bt = a.block_tables + static_cast<int64_t>(b) * a.max_blocks_per_seq;

  // q of the heads (rows from G on are zero): in shared memory, since how many
  // warps there are decides more than how long each takes (128 registers: with
  // q in them, or both halves of the values in flight, 30 % fewer warps fit and
  // 256 sequences of 32 own tokens took 49 us for 42)
  __shared__ uint4 q_s[8][D / 8];
  for (int i = tid; i < 8 * (D / 8); i += D)
    q_s[i / (D / 8)][i % (D / 8)] =
        i / (D / 8) < G
            ? __ldg(reinterpret_cast<const uint4*>(
                        static_cast<const T*>(a.q) +
                        (static_cast<int64_t>(b) * Hq + kvh * G + i / (D / 8)) * D) +
                    i % (D / 8))
            : make_uint4(0, 0, 0, 0);
  __syncthreads();
  float m = -INFINITY, sum = 0.f;             // of this thread's head (all four c alike for m)
  float o[2][8][4];                           // [64 columns][element of 8][MMA accumulator]
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[j][e][x] = 0.f;
  bool bad = false;

  for (int t0 = grp * 16; t0 < n; t0 += kGroups * 16) {
    const int32_t id = __ldg(bt + t0 / BS);
    if (id < 0 || id >= a.num_blocks) {
      bad = true;
      continue;
    }
    const int64_t base =
        ((static_cast<int64_t>(id) * a.num_kv_heads + kvh) * BS + t0 % BS) * D;
    const int left = n - t0;                  // tokens of the group
    // keys: token `row` and `row + 8`; values: tokens 2c, 2c + 1, 2c + 8, 2c + 9
    uint4 k[2][kPieces];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        k[u][i] = row + 8 * u < left
                      ? __ldg(reinterpret_cast<const uint4*>(kc + base + (row + 8 * u) * D + 8 * c +
                                                             32 * i))
                      : make_uint4(0, 0, 0, 0);
    uint4 v[2][4];
    auto load_v = [&](int j) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int t = 2 * c + (x & 1) + 8 * (x >> 1);
        v[j][x] = t < left ? __ldg(reinterpret_cast<const uint4*>(vc + base + t * D + half * 128 +
                                                                  64 * j + 8 * row))
                           : make_uint4(0, 0, 0, 0);
      }
    };
    load_v(0);
    float s[2][4] = {};
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint4 q = q_s[row][4 * i + c];
        mma16816<T>(s[u], q.x, 0u, q.y, 0u, k[u][i].x, k[u][i].y);
        mma16816<T>(s[u], q.z, 0u, q.w, 0u, k[u][i].z, k[u][i].w);
      }
    load_v(1);  // into the keys' registers
    // logits of head `row`: tokens 2c, 2c + 1 (u = 0) and + 8 (u = 1)
    float l[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int t = 2 * c + (x & 1) + 8 * (x >> 1);
      l[x] = t < left ? s[x >> 1][x & 1] * a.scale_log2 : -INFINITY;
    }
    float mt = fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3]));
    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
    const bool move = mt > m + kRescaleLog2;  // also from -inf
    if (__any_sync(0xffffffffu, move)) {
      const float f = !move ? 1.f : m == -INFINITY ? 0.f : exp2f(m - mt);
      if (move) m = mt;
      sum *= f;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int x = 0; x < 4; ++x) o[j][e][x] *= f;
    }
    float p[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) p[x] = l[x] == -INFINITY ? 0.f : exp2f(l[x] - m);
    sum += (p[0] + p[1]) + (p[2] + p[3]);
    uint32_t h0, h1, l0, l1;
    split_pair<T>(p[0], p[1], h0, l0);
    split_pair<T>(p[2], p[3], h1, l1);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t* v0 = &v[j][0].x;
      const uint32_t* v1 = &v[j][1].x;
      const uint32_t* v2 = &v[j][2].x;
      const uint32_t* v3 = &v[j][3].x;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t sel = e & 1 ? 0x7632 : 0x5410;
        mma16816<T>(o[j][e], h0, l0, h1, l1, __byte_perm(v0[e / 2], v1[e / 2], sel),
                    __byte_perm(v2[e / 2], v3[e / 2], sel));
      }
    }
  }
  // ---- the warps' partials into shared memory ------------------------------------
  sum += __shfl_xor_sync(0xffffffffu, sum, 1);
  sum += __shfl_xor_sync(0xffffffffu, sum, 2);
  // element e of columns 64 j + 16 c (+ 8): accumulators 0 and 1, remainders 2 and 3
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int e = 0; e < 8; e += 4)
        *reinterpret_cast<float4*>(&o_s[grp][row][half * 128 + 64 * j + 16 * c + 8 * g + e]) =
            make_float4(o[j][e][g] + o[j][e][2 + g], o[j][e + 1][g] + o[j][e + 1][2 + g],
                        o[j][e + 2][g] + o[j][e + 2][2 + g], o[j][e + 3][g] + o[j][e + 3][2 + g]);
  if (half == 0 && c == 0) {
    m_s[grp][row] = m;
    s_s[grp][row] = sum;
  }
  if (bad && lane == 0) bad_s = 1;
  if (tid == 0) {
    if (!ok) set_status(a.status, PA_ERR_BAD_SEQ_LEN);
  }
  __syncthreads();
  if (tid == 0 && bad_s) set_status(a.status, PA_ERR_BAD_BLOCK_ID);

  // ---- the join: a thread takes four columns of a head ------------------------------
  int parts = 0;
  bool poison = !ok || bad_s != 0;
  if (pre.lens) {
    const int32_t P = __ldg(pre.lens);
    if (P < 0 || P > pre.max_len) {
      poison = true;
      if (!pre.m && tid == 0) set_status(a.status, PA_ERR_BAD_SEQ_LEN);  // no prefix pass ran
    } else if (pre.m) {
      parts = prefix_split(P, a.num_kv_heads, pre.key_blocks).segments(kvh) * pre.lanes;
    }
  }
  // the partials were written while this kernel ran: coherent loads, no __ldg
  cudaGridDependencySynchronize();
  for (int i = tid; i < G * (D / 4); i += D) {
    const int h = i / (D / 4), d = i % (D / 4) * 4;
    const int64_t r = static_cast<int64_t>(b) * Hq + kvh * G + h;
    float M = -INFINITY, w = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    bool nan_seen = poison;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) M = fmaxf(M, m_s[g][h]);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float f = m_s[g][h] == -INFINITY ? 0.f : exp2f(m_s[g][h] - M);
      const float4 v = *reinterpret_cast<const float4*>(&o_s[g][h][d]);
      w = fmaf(s_s[g][h], f, w);
      acc.x = fmaf(v.x, f, acc.x);
      acc.y = fmaf(v.y, f, acc.y);
      acc.z = fmaf(v.z, f, acc.z);
      acc.w = fmaf(v.w, f, acc.w);
    }
    M *= kLn2;                                // the partials' unit
    constexpr int kBatch = 8;
    for (int base = 0; base < parts; base += kBatch) {
      float mp[kBatch], sp[kBatch];
      float4 v[kBatch];
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        mp[x] = -INFINITY;
        sp[x] = 0.f;
        v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (base + x < parts) {
          const int64_t at = r * pre.stride + base + x;
          mp[x] = __ldcg(pre.m + at);
          sp[x] = __ldcg(pre.s + at);
          v[x] = __ldcg(reinterpret_cast<const float4*>(pre.o + at * D + d));
        }
      }
      float mb = M;
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        nan_seen |= isnan(mp[x]) || isnan(sp[x]);  // a bad block, or a NaN logit
        mb = fmaxf(mb, mp[x]);
      }
      if (mb > M) {
        const float f = expf(M - mb);         // 0 when M is -inf
        w *= f;
        acc.x *= f;
        acc.y *= f;
        acc.z *= f;
        acc.w *= f;
        M = mb;
      }
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        if (mp[x] == -INFINITY) continue;
        const float f = sp[x] * expf(mp[x] - M);
        w += f;
        acc.x = fmaf(v[x].x, f, acc.x);
        acc.y = fmaf(v[x].y, f, acc.y);
        acc.z = fmaf(v[x].z, f, acc.z);
        acc.w = fmaf(v[x].w, f, acc.w);
      }
    }
    const float inv = nan_seen ? qnan() : w > 0.f ? 1.f / w : 0.f;
    store_out4(a.out, r * D + d, a.out_dtype,
               make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
  }
}

template <typename T, int D>
cudaError_t launch_own_d(const KernelArgs& a, const JoinList& pre, bool pdl, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.num_seqs) * a.num_kv_heads, 1, 1);
  cfg.blockDim = dim3(D, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, pa_own_kernel<T, D>, a, pre);
}

}  // namespace

// Measured against pass 1 + join in kernels of their own (prefix of 4096, own
// lists of n / 2 .. n; us, this kernel / those): 32 heads over 8 of 128: 64
// sequences, n = 32: 19 / 31, 128: 25 / 33, 256: 33 / 36, 512: 47 / 42; 256
// sequences: 42 / 60, 56 / 63, 77 / 74, 115 / 100; 8 sequences: 15 / 17, 18 / 17.
// 24 over 4 of 256: 64 sequences 24 / 30, 30 / 33, 38 / 34; 256: 65 / 70, 84 / 72.
bool own_applicable(const pa_params_t* p) {
  const int64_t pairs = static_cast<int64_t>(p->num_seqs) * p->num_kv_heads;
  return tc_applicable(p) && p->block_size % 16 == 0 && pairs >= 128 &&
         pairs < (int64_t(1) << 31) && p->max_seq_len <= (p->head_dim == 128 ? 256 : 128);
}

cudaError_t launch_own(const KernelArgs& a, const JoinList& prefix, pa_dtype_t t, bool pdl,
                       cudaStream_t s) {
  if (t == PA_BF16)
    return a.head_dim == 256 ? launch_own_d<__nv_bfloat16, 256>(a, prefix, pdl, s)
                             : launch_own_d<__nv_bfloat16, 128>(a, prefix, pdl, s);
  return a.head_dim == 256 ? launch_own_d<__half, 256>(a, prefix, pdl, s)
                           : launch_own_d<__half, 128>(a, prefix, pdl, s);
}

}  // namespace pa
