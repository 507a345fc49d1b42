// pa_kv4.cuh -- the paged cache held in 4 bits: its format, the work list of its
// kernels, and what they share.
//
// A head row of D elements is D / 2 bytes of codes (element 2i in the low half of
// byte i) and D / group pairs (scale, minimum) of the model's element type; code
// c stands for c * scale + minimum.  Row r of a pool, r = (block * Hkv + head) *
// block_size + place, has its codes at r * D / 2 and its pairs at r * D / group.
#pragma once

#include <type_traits>

#include "pa_device.cuh"

namespace pa {

// ---- a scale and a minimum ------------------------------------------------------

template <typename T>
__device__ __forceinline__ float2 widen_pair(uint32_t w) {
  float2 p;
  widen2(static_cast<const T*>(nullptr), w, p.x, p.y);
  return p;
}
// Pair i of a pool's pairs.
template <typename T>
__device__ __forceinline__ float2 load_pair(const void* pairs, int64_t i) {
  if constexpr (std::is_same<T, float>::value)
    return __ldg(static_cast<const float2*>(pairs) + i);
  else
    return widen_pair<T>(__ldg(static_cast<const uint32_t*>(pairs) + i));
}

// ---- two floats as one operand of the packed instructions -------------------------

using F2 = unsigned long long;
__device__ __forceinline__ F2 pair(float x, float y) {
  F2 v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  return v;
}
__device__ __forceinline__ float2 unpair(F2 v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ F2 add2(F2 x, F2 y) {
  F2 v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(x), "l"(y));
  return v;
}
__device__ __forceinline__ F2 mul2(F2 x, F2 y) {
  F2 v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(x), "l"(y));
  return v;
}
__device__ __forceinline__ F2 fma2(F2 x, F2 y, F2 z) {
  F2 v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(x), "l"(y), "l"(z));
  return v;
}

// ---- decode -------------------------------------------------------------------------

// Whether the call can serve this sequence length.
__device__ __forceinline__ bool kv4_len_ok(const Kv4Args& a, int32_t L) {
  return L >= 0 && L <= a.max_len &&
         L <= static_cast<int64_t>(a.max_blocks_per_seq) * a.block_size;
}

// Element d of the joined result of a part of head h: maximum M (base 2), sum and
// weighted sum o, into the output or the part's partial.  `bad`: a length or a
// block id that cannot be trusted.
__device__ __forceinline__ void kv4_finish(const Kv4Args& a, int b, int h, int part, int d, int D,
                                           bool direct, int32_t L, int bad, float M, float sum,
                                           float o) {
  const int64_t row = static_cast<int64_t>(b) * a.num_heads + h;
  const float r = bad ? qnan() : L == 0 ? 0.f : o / sum;
  if (direct) {
    store_out(a.out, row * D + d, a.out_dtype, r);
    return;
  }
  const int64_t at = row * a.num_parts + part;
  a.part_out[at * D + d] = r;
  if (d == 0) {
    a.part_max[at] = bad ? qnan() : M;
    a.part_sum[at] = bad ? qnan() : sum;
  }
}

// ---- the work list ----------------------------------------------------------------
//
// Sequence b has n_b work items (parts of its tokens, pages); the list is all of
// them, sequence after sequence, and CTAs take items from it, so that nothing is
// spent on what a short sequence does not have.  Every CTA sums the counts of 32
// sequences at a time into shared memory; an item's sequence is found by a binary
// search there and a scan of 32 counts by the warp that asks.  `Count` gives n_b
// (its lengths are inputs of the call).
constexpr int kListSpan = 32;
inline __host__ __device__ int list_chunks(int num_seqs) {
  return (num_seqs + kListSpan - 1) / kListSpan;
}
inline size_t list_bytes(int num_seqs) { return (list_chunks(num_seqs) + 1) * sizeof(uint32_t); }

// All threads of the CTA; returns the length of the list.  `start` holds
// list_chunks() + 1 words.
template <typename Count>
__device__ uint32_t list_build(uint32_t* start, int num_seqs, const Count& count) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int chunks = list_chunks(num_seqs);
  for (int c = warp; c < chunks; c += warps) {
    const int b = c * kListSpan + lane;
    uint32_t n = b < num_seqs ? count(b) : 0;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (lane == 0) start[c] = n;
  }
  __syncthreads();
  if (warp == 0) {
    uint32_t sum = 0;
    for (int c0 = 0; c0 < chunks; c0 += 32) {
      const uint32_t own = c0 + lane < chunks ? start[c0 + lane] : 0;
      uint32_t x = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (c0 + lane < chunks) start[c0 + lane] = sum + x - own;
      sum += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) start[chunks] = sum;
  }
  __syncthreads();
  return start[chunks];
}

// All lanes of a warp: the sequence of item i, and which of its items it is.
template <typename Count>
__device__ __forceinline__ void list_find(const uint32_t* start, int num_seqs, const Count& count,
                                          uint32_t i, int& seq, uint32_t& index) {
  int lo = 0, hi = list_chunks(num_seqs);  // start[lo] <= i < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= i) lo = mid;
    else hi = mid;
  }
  const int lane = threadIdx.x & 31, b = lo * kListSpan + lane;
  const uint32_t own = b < num_seqs ? count(b) : 0;
  uint32_t x = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  const uint32_t at = i - (lo > 0 ? start[lo] : 0);  // one span needs no list
  const int who = __ffs(__ballot_sync(0xffffffffu, at < x)) - 1;  // the first sum past it
  seq = lo * kListSpan + who;
  index = at - __shfl_sync(0xffffffffu, x - own, who);
}

}  // namespace pa
