// pa_kv4_tc.cuh -- tensor-core decode over the 4-bit cache, bf16 and f16.
//
// A work item is a part of a sequence, a KV head and up to eight of its query
// heads.  The warps of a CTA take its tiles of 16 (head_dim 256) or 32 tokens in
// turn, each with a ring of its own (cp.async, no barrier between warps) and running
// statistics of its own; they are joined at the end of the item.
//
// Codes never become values.  With k = s c + m,
//   q . k = sum_g s_g (sum_g q c) + m_g (sum_g q),
// so the MMA multiplies q by codes, and a group's scale enters in float32, once per
// token, group and head.  With v = s (c - 8) + (m + 8 s),
//   sum_t p v = sum_t (p s) c - 8 sum_t (p s) + sum_t p (m + 8 s),
// so p s is what the second MMA multiplies by codes; its own sum comes from an MMA
// with rows of eights, and the last sum from one of scales and minima by p.  That one
// takes p in two parts of 16 bits, and the keys' minima the sums of q in two or three.
//   * A code in the low half of a byte, masked, is the f16 subnormal c 2^-24, in the
//     high half c 2^-20: one mask makes two operands of a 32-bit word, and the powers
//     of two leave with the scales.
//   * Keys are the 16 x 16 operand A (16 tokens), q is B (8 heads), scaled per head by
//     a power of two to below 2^15: exact, but for elements 2^-24 below the largest.
//     The 16 elements of an MMA are those a lane finds in its words (LDSM), q in that
//     order.
//   * Values are A with rows d and columns t: LDSM's transpose brings two tokens' 16
//     bits into one word.  B is p s, multiplied in float32 (with a power of two per group
//     that follows the largest scale seen) and rounded to f16 once: half a step, 2^-11 of
//     it, on c - 8 and not on c, since the eights are multiplied by the rounded products
//     too.  What is 2^-35 of the largest scale, for a weight of 1, is the least step: a token
//     of the largest weight keeps all its bits while its scale is above 2^-24 of the largest.
//     (The product in f16 instead, of both rounded, took 0 to 2 % less time, 3 to 5 % with
//     groups of 32 of bf16, and lost what was below 2^-17 of the largest scale.  What the
//     rounding leaves, multiplied too, takes 10 to 17 % more, 256 sequences up to 100K 627 to
//     691 us; without it f16 outputs are off by 1.05 times what float32 sums with one rounding
//     to f16 are, 1.3 times at most of 250 batches, bf16 outputs by as much as those.)
//   * The reference of the softmax moves when a logit passes it by 2^4, the scales'
//     power when a scale passes it: one vote a tile, no reduction otherwise.
// All sums are float32.
//
// Bound by instructions and by what waits on them, not by memory: a tile of 16 tokens of
// 128 elements is some 290 warp instructions, 130 of them on the ALU pipe (64 masks and
// 16 shifts), 22 MMAs.  Measured: 76 sequences of 8192, 32 / 8 heads of 128, one group a
// row: 141 us = 4.8 TB/s, 71 % of the copy rate; the same kernel's copies alone take 124 us,
// its arithmetic alone 121.  114 of 4096, 24 / 4 of 256: 101 us = 5.3 TB/s.  One sequence of
// 100K 32 us with the join (5 us before the first stage, 20 of streaming, 2.5 to join the
// warps), 256 sequences up to 100K 627 us, 33 of f16 with groups of 32 161 us.
#pragma once

#include <atomic>

#include "pa_kv4.cuh"

namespace pa {
namespace kv4 {

constexpr unsigned kAll = 0xffffffffu;

template <int D, int GS, bool kWide>
struct Cfg {
  // warps of a CTA, and CTAs that are resident on an SM
  static constexpr int kWarps = kWide ? (D == 256 ? 12 : 16) : 4;
  static constexpr int kCtas = kWide ? 1 : D == 256 ? 3 : 4;
  static constexpr int kNT = kWarps * 32;
  static constexpr int kLeast = 128;  // tokens of a part that pay for its join
  static constexpr int NB = D / 32;             // blocks of 32 elements: a word of keys a lane
  static constexpr int NP = D / GS;             // pairs of a head row
  static constexpr int SB = NP * 4;             //   and their bytes
  static constexpr int MT = D == 256 ? 1 : 2;   // 16-token tiles of a stage
  static constexpr int ROWS = 16 * MT;
  static constexpr int KP = D / 2 + 16;         // pitch of codes: rows of LDSM in other banks
  static constexpr int kV = ROWS * KP;
  static constexpr int kKs = kV + ROWS * KP;
  static constexpr int kVs = kKs + ROWS * SB;
  static constexpr int kStage = kVs + ROWS * SB;
  static constexpr int kStages = !kWide && D == 64 ? 3 : 2;
  static constexpr int PP = ROWS + 4;           // pitch of the weights' transposition
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kQ = D / 32 * 512;       // q fragments
  static constexpr int kOffQ = kRing;
  static constexpr int kOffQs = kOffQ + kQ;                  // sums of q: [D / 32][8]
  static constexpr int kOffP = kOffQs + D / 32 * 8 * 4;      // weights: [warp][8][PP]
  static constexpr int kOffW = kOffP + kWarps * 8 * PP * 4;  // statistics: [2][warp][8]
  static constexpr int kOffList = kOffW + 2 * kWarps * 8 * 4;
  static_assert((kOffList + 1024 + 128) * kCtas <= 228 * 1024, "resident CTAs");
  static_assert(kStages * kStage >= 8 * D * 4, "a warp's results take its ring's place");
  static_assert(kStage % 16 == 0 && KP % 16 == 0, "16-byte copies");
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// `bytes` of 16 from src, the rest zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes));
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src));
}
template <int N>
__device__ __forceinline__ void copy_small(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N),
               "r"(bytes));
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// c (16 x 8, f32) += a (16 x 16) * b (16 x 8), f16 or bf16
template <typename T>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same from zero.
template <typename T>
__device__ __forceinline__ void mma0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                     uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^k, k in -126..127
__device__ __forceinline__ float pow2(int k) { return __int_as_float((k + 127) << 23); }
__device__ __forceinline__ int exponent(float x) {
  return (__float_as_int(x) >> 23 & 255) - 127;
}
// Two floats rounded to T, and what the rounding left, rounded too.
template <typename T>
__device__ __forceinline__ uint32_t pack(float x, float y) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <typename T>
__device__ __forceinline__ uint32_t split(float& x, float& y) {
  const uint32_t h = pack<T>(x, y);
  const float2 f = widen_pair<T>(h);
  x -= f.x;
  y -= f.y;
  return h;
}
__device__ __forceinline__ float low_half(const __nv_bfloat16*, uint32_t w) {
  return __uint_as_float(w << 16);
}
__device__ __forceinline__ float low_half(const __half*, uint32_t w) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(w)));
}
// Two float32 products, rounded to f16.
__device__ __forceinline__ uint32_t products(float2 x, float2 y) {
  const float2 z = unpair(mul2(pair(x.x, x.y), pair(y.x, y.y)));
  return pack<__half>(z.x, z.y);
}
// The scale of a pair.
template <typename T>
__device__ __forceinline__ float scale_of(uint32_t w) {
  return low_half(static_cast<const T*>(nullptr), w);
}

// The N pairs of a row in shared memory (N words, a power of two).
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
}

// Four 8 x 8 matrices of 16-bit units, lane's row at `addr`; kTrans: their transposes.
template <bool kTrans>
__device__ __forceinline__ void ldsm(uint32_t (&w)[4], uint32_t addr) {
  if constexpr (kTrans)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr)
                 : "memory");
}

// Parts of sequence b: those with a token; one for a row that the item itself has to
// finish (no join follows).
struct Parts {
  const Kv4Args& a;
  int32_t size;
  __device__ __forceinline__ uint32_t of(int32_t L) const {
    return kv4_len_ok(a, L) && L > 0 ? (static_cast<uint32_t>(L) + size - 1) / size
                                     : a.num_parts == 1;
  }
  __device__ __forceinline__ uint32_t operator()(int b) const { return of(__ldg(a.lens + b)); }
};

// Tokens of a part, from the lengths of the call: all CTAs come to the same.
//   * Few (sequence, KV head) pairs for the CTAs that are resident: one round, as even as
//     parts of one size are: the least size that makes no more items than CTAs (32
//     sequences or fewer), or one that does whatever the lengths are.
//   * Many, of different lengths: a CTA's share of the work is w tokens; parts of n tokens cost
//     it w / n starts, each worth some kStart tokens, and leave it waiting for about half a part
//     at the end: n = sqrt(2 kStart w).
//   * Many, most of them nearly as long as the longest: of 1 to 32 even parts of that, the number
//     with the least rounds of items, the last one counted 0.7 (a CTA that has an SM for itself)
//     to 1.  Measured, us, by w alone and so: 76 sequences of 8192, 32 / 8 heads of 128, 166 and
//     141; 100 of 4000 116 and 113; 300 of 2000, 24 / 4 of 256, 169 and 137; 60 of 2000 50 and 44;
//     114 of 4096 132 and 101 (but 128 of 2500, 32 / 8 of 128, 94 and 96; 40 of 4000 60.0 and 60.6).
// Never below `least` (nor below what the workspace has slots for, part_floor, which is at most
// kKv4Longest), nor above kKv4Longest.  In float32: nothing else depends on the size but speed.
constexpr float kStart = 200.f, kJoin = 300.f;  // tokens that a start and the join are worth
constexpr float kEven = 0.8f;                   // mean over longest
__device__ __forceinline__ int32_t choose_part(const Kv4Args& a, float tokens, float longest,
                                               int32_t own, int32_t least) {
  if (a.num_parts == 1) return max((a.max_len + 63) / 64 * 64, 64);
  const float per = static_cast<float>(a.num_kv_heads * a.head_groups);
  const float pairs = per * a.num_seqs, room = a.room, share = tokens * per / room;
  least = max(least, a.part_floor);
  const int32_t most = max(min((a.max_len + 63) / 64 * 64, kKv4Longest), least);
  const auto within = [&](float n) {  // whole tiles
    return n >= static_cast<float>(most) ? most
                                         : max((static_cast<int32_t>(ceilf(n)) + 63) / 64 * 64, least);
  };
  if (2.f * pairs > room) {
    if (tokens < kEven * longest * a.num_seqs) return within(sqrtf(2.f * kStart * share));
    // a lane for every number of parts
    const int lane = threadIdx.x & 31;
    const int32_t n = within(__fdividef(longest, lane + 1.f));
    const float parts = ceilf(__fdividef(longest, static_cast<float>(n)));
    const float rounds = __fdividef(pairs * parts, room), x = rounds - floorf(rounds);
    const float cost = (floorf(rounds) + (x > 0.f ? 0.7f + 0.3f * x : 0.f)) * (n + kStart) +
                       (parts > 1.f ? kJoin : 0.f);
    const unsigned best = __reduce_min_sync(kAll, (__float_as_uint(cost) & ~31u) | lane);
    return __shfl_sync(kAll, n, best & 31);
  }
  if (a.num_seqs == 1) return within(__fdividef(tokens, floorf(__fdividef(room, per))));
  int32_t hi = within(tokens * per / (room - pairs));
  if (a.num_seqs > 32) return hi;
  // lanes hold the lengths: the fewest tokens, to some steps, with which all items have CTAs
  int32_t lo = within(share) - 64;
  const float fits = room / per;
#pragma unroll 1
  for (int i = 0; i < 5 && hi - lo > 64; ++i) {
    const int32_t mid = lo + (hi - lo) / 128 * 64;
    float n = ceilf(__fdividef(static_cast<float>(own), static_cast<float>(mid)));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) n += __shfl_xor_sync(kAll, n, o);
    if (n <= fits) hi = mid;
    else lo = mid;
  }
  return hi;
}

// The queue of items, in the workspace's control block: CTAs take their first item by
// number, further ones here.  The CTA that is done last leaves it as it was found, zeros.
struct Queue {
  uint32_t next, done;
};

template <typename T, int D, int GS, bool kWide>
__global__ void __launch_bounds__(Cfg<D, GS, kWide>::kNT, Cfg<D, GS, kWide>::kCtas)
    pa_kv4_tc_kernel(const Kv4Args a) {
  using C = Cfg<D, GS, kWide>;
  constexpr int NB = C::NB, MT = C::MT, NP = C::NP, kWarps = C::kWarps, kNT = C::kNT;
  constexpr bool kHalf = std::is_same<T, __half>::value;
  constexpr int kParts = kHalf ? 2 : 3;                  // of the sums of q
  constexpr float kMinUp = kHalf ? 0x1p16f : 1.f;        // keeps f16 operands in range
  // Weights are taken times 2^kUp, and the reference moves when a logit passes it by 2^kBar;
  // scales are taken times a power of two that leaves the largest below 2^kTop.  The weights are
  // split into two of T, and the products, at most 2^15, rounded to f16.
  constexpr float kUp = 8.f, kBar = 4.f;
  constexpr int kTop = 3;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int bad_s;
  __shared__ uint32_t next_s, next_part_s;
  __shared__ int next_b_s, next_len_s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, c = lane & 3;  // row of A, or head of B; column pair
  uint8_t* ring = smem + warp * (C::kStages * C::kStage);
  uint4* qf = reinterpret_cast<uint4*>(smem + C::kOffQ);
  float* qs = reinterpret_cast<float*>(smem + C::kOffQs);
  float* pt = reinterpret_cast<float*>(smem + C::kOffP) + warp * (8 * C::PP);
  float* stat = reinterpret_cast<float*>(smem + C::kOffW);  // [2][kWarps][8]
  uint32_t* list = reinterpret_cast<uint32_t*>(smem + C::kOffList);

  cudaTriggerProgrammaticLaunchCompletion();  // the join waits for this grid's end itself
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.num_seqs; b += kNT)
      if (!kv4_len_ok(a, __ldg(a.lens + b))) set_status(a.status, PA_ERR_BAD_SEQ_LEN);
  const uint32_t per = a.num_kv_heads * a.head_groups;
  Parts parts{a, 0};
  uint32_t items;
  // the item at hand: sequence, part, length; the first is found from registers where a lane
  // has a sequence
  int b = 0;
  uint32_t part = 0;
  int32_t L = 0;
  bool found = a.num_seqs <= kListSpan;
  if (found) {
    const int32_t given = lane < a.num_seqs ? __ldg(a.lens + lane) : 0;
    const int32_t own = kv4_len_ok(a, given) ? given : 0;
    float tokens = own;
    int32_t longest = own;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      tokens += __shfl_xor_sync(kAll, tokens, o);
      longest = max(longest, __shfl_xor_sync(kAll, longest, o));
    }
    parts.size = choose_part(a, tokens, longest, own, C::kLeast);
    const uint32_t n = lane < a.num_seqs ? parts.of(own) : 0;
    uint32_t sums = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(kAll, sums, o);
      if (lane >= o) sums += y;
    }
    items = __shfl_sync(kAll, sums, 31);
    const uint32_t sp = blockIdx.x / per;
    if (sp < items) {
      b = __ffs(__ballot_sync(kAll, sp < sums)) - 1;
      part = sp - __shfl_sync(kAll, sums - n, b);
      L = __shfl_sync(kAll, given, b);
    }
  } else {
    // whole numbers: the sum has one order of addition
    unsigned long long* all = reinterpret_cast<unsigned long long*>(stat);
    if (threadIdx.x == 0) all[0] = all[1] = 0;
    __syncthreads();
    unsigned long long tokens = 0;
    int32_t longest = 0;
    for (int i = threadIdx.x; i < a.num_seqs; i += kNT) {
      const int32_t one = __ldg(a.lens + i);
      if (!kv4_len_ok(a, one)) continue;
      tokens += one;
      longest = max(longest, one);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      tokens += __shfl_xor_sync(kAll, tokens, o);
      longest = max(longest, __shfl_xor_sync(kAll, longest, o));
    }
    if (lane == 0) {
      atomicAdd(all, tokens);
      atomicMax(all + 1, static_cast<unsigned long long>(longest));
    }
    __syncthreads();
    parts.size = choose_part(a, static_cast<float>(all[0]), static_cast<float>(all[1]), 0,
                             C::kLeast);
    items = list_build(list, a.num_seqs, parts);
  }
  items *= per;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.part_at = parts.size;  // for the join

  // without the marker the control block may hold anything: items by number then
  Queue* queue = reinterpret_cast<Queue*>(a.part_at + 1);
  const bool queued = items > gridDim.x &&
                      __ldg(a.status + kMarkerOffset / 4) == kMarker;

  for (uint32_t item = blockIdx.x; item < items;) {
    if (threadIdx.x == 0)  // for the next turn; read after barriers
      next_s = queued ? gridDim.x + atomicAdd(&queue->next, 1u) : item + gridDim.x;
    const uint32_t sp = item / per, x = item - sp * per;
    if (!found) {
      list_find(list, a.num_seqs, parts, sp, b, part);
      L = __ldg(a.lens + b);
    }
    found = false;
    const int kvh = x / a.head_groups, hg = x - kvh * a.head_groups;
    const int nh = min(kKv4Heads, a.group - hg * kKv4Heads);
    const int h0 = kvh * a.group + hg * kKv4Heads;
    if (!kv4_len_ok(a, L) || L == 0) {
      const int64_t row = static_cast<int64_t>(b) * a.num_heads + h0;
      for (int i = threadIdx.x; i < nh * D; i += kNT)
        store_out(a.out, row * D + i, a.out_dtype, L == 0 ? 0.f : qnan());
      __syncthreads();
      item = next_s;
      __syncthreads();
      continue;
    }
    const bool direct = L <= parts.size;  // the only part: no join
    const int32_t t0 = part * parts.size;
    const int32_t t1 = L - t0 > parts.size ? t0 + parts.size : L;
    const int32_t* table = a.block_tables + static_cast<int64_t>(b) * a.max_blocks_per_seq;
    const int BS = a.block_size;

    // ---- copies: stage i of this warp is tokens t0 + (i * kWarps + warp) * ROWS ... ----
    const int stages = (t1 - t0 + C::ROWS * kWarps - 1 - warp * C::ROWS) / (C::ROWS * kWarps);
    bool bad = false;
    // Pages of 16-token multiples: a tile is in one page, one run of memory.  The page
    // ids are loaded a stage ahead.
    int32_t page[MT];
    const auto load_pages = [&](int i) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int32_t t = t0 + (i * kWarps + warp) * C::ROWS + 16 * mt;
        page[mt] = -1;
        if (a.paged16 && t < t1)
          page[mt] = __ldg(table + (a.block_shift >= 0 ? t >> a.block_shift : t / BS));
      }
    };
    // bytes of a page in the pools, and this lane's 16 in a head's part and in a stage
    const uint32_t page_rows = static_cast<uint32_t>(a.num_kv_heads) * BS;
    const uint32_t page_codes = page_rows * (D / 2), page_pairs = page_rows * C::SB;
    const uint32_t head_codes = kvh * BS * (D / 2) + lane * 16;
    const uint32_t head_pairs = kvh * BS * C::SB + lane * 16;
    const uint32_t copy_k = lane / (D / 32) * C::KP + lane % (D / 32) * 16;
    const uint32_t copy_v = C::kV + lane / (D / 32) * C::KP + lane % (D / 32) * 16;
    const auto issue = [&](int i, uint32_t dst) {
      const int32_t ts = t0 + (i * kWarps + warp) * C::ROWS;
      bool whole = a.paged16 && ts + C::ROWS <= t1;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        whole = whole && static_cast<uint32_t>(page[mt]) < static_cast<uint32_t>(a.num_blocks);
      if (whole) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const int32_t t = ts + 16 * mt;
          const uint32_t at = a.block_shift >= 0 ? t & (BS - 1) : t % BS;
          // a page's part of a pool is below 2^32 bytes (paged16)
          const uint64_t codes = static_cast<uint64_t>(static_cast<uint32_t>(page[mt])) *
                                     page_codes + (at * (D / 2) + head_codes);
          const uint8_t* kc = a.k_codes + codes;
          const uint8_t* vc = a.v_codes + codes;
          const uint32_t to = dst + copy_k + 16 * mt * C::KP;
          const uint32_t vto = dst + copy_v + 16 * mt * C::KP;
#pragma unroll
          for (int u = 0; u < D / 64; ++u) {
            copy16(to + u * (1024 / D) * C::KP, kc + u * 512);
            copy16(vto + u * (1024 / D) * C::KP, vc + u * 512);
          }
          if (lane < C::SB) {
            const uint64_t pairs = static_cast<uint64_t>(static_cast<uint32_t>(page[mt])) *
                                       page_pairs + (at * C::SB + head_pairs);
            const uint32_t pto = dst + C::kKs + 16 * mt * C::SB + lane * 16;
            copy16(pto, static_cast<const uint8_t*>(a.k_pairs) + pairs);
            copy16(pto + (C::kVs - C::kKs), static_cast<const uint8_t*>(a.v_pairs) + pairs);
          }
        }
      } else if (a.paged16) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const int32_t t = ts + 16 * mt;
          int n = min(max(t1 - t, 0), 16);  // tokens of the tile
          int64_t row = 0;
          if (n > 0) {
            if (page[mt] < 0 || page[mt] >= a.num_blocks) {
              bad = true;
              n = 0;
            } else {
              const int at = a.block_shift >= 0 ? t & (BS - 1) : t % BS;
              row = (static_cast<int64_t>(page[mt]) * a.num_kv_heads + kvh) * BS + at;
            }
          }
          const uint8_t* kc = a.k_codes + row * (D / 2);
          const uint8_t* vc = a.v_codes + row * (D / 2);
#pragma unroll
          for (int u = 0; u < D / 64; ++u) {
            const int idx = u * 32 + lane, rr = idx / (D / 32), piece = idx % (D / 32);
            const int bytes = rr < n ? 16 : 0;
            copy16(dst + (16 * mt + rr) * C::KP + piece * 16, kc + idx * 16, bytes);
            copy16(dst + C::kV + (16 * mt + rr) * C::KP + piece * 16, vc + idx * 16, bytes);
          }
          if (lane < C::SB) {  // SB pieces of 16 bytes are 16 rows of SB bytes
            const int bytes = min(max(n * C::SB - lane * 16, 0), 16);
            const uint32_t to = dst + C::kKs + 16 * mt * C::SB + lane * 16;
            copy16(to, static_cast<const uint8_t*>(a.k_pairs) + row * C::SB + lane * 16, bytes);
            copy16(to + (C::kVs - C::kKs),
                   static_cast<const uint8_t*>(a.v_pairs) + row * C::SB + lane * 16, bytes);
          }
        }
      } else {  // any page size: a row at a time
        const auto place = [&](int rr, bool& ok) -> int64_t {
          const int32_t t = ts + rr;
          ok = t < t1;
          if (!ok) return 0;
          const int32_t j = t / BS, id = __ldg(table + j);
          if (id < 0 || id >= a.num_blocks) {
            bad = true;
            ok = false;
            return 0;
          }
          return (static_cast<int64_t>(id) * a.num_kv_heads + kvh) * BS + (t - j * BS);
        };
        for (int idx = lane; idx < C::ROWS * (D / 32); idx += 32) {
          const int rr = idx / (D / 32), piece = idx % (D / 32);
          bool ok;
          const int64_t at = place(rr, ok) * (D / 2) + piece * 16;
          copy16(dst + rr * C::KP + piece * 16, a.k_codes + at, ok ? 16 : 0);
          copy16(dst + C::kV + rr * C::KP + piece * 16, a.v_codes + at, ok ? 16 : 0);
        }
        constexpr int kPiece = C::SB < 16 ? C::SB : 16;
        for (int idx = lane; idx < C::ROWS * (C::SB / kPiece); idx += 32) {
          const int rr = idx / (C::SB / kPiece), piece = idx % (C::SB / kPiece);
          bool ok;
          const int64_t at = place(rr, ok) * C::SB + piece * kPiece;
          const uint32_t to = dst + C::kKs + rr * C::SB + piece * kPiece;
          copy_small<kPiece>(to, static_cast<const uint8_t*>(a.k_pairs) + at, ok ? kPiece : 0);
          copy_small<kPiece>(to + (C::kVs - C::kKs), static_cast<const uint8_t*>(a.v_pairs) + at,
                             ok ? kPiece : 0);
        }
      }
    };
    // ---- q: a lane has eight elements of each block of head r; warps take blocks in turn ---
    constexpr int kOwn = (NB + kWarps - 1) / kWarps;
    const T* qrow = static_cast<const T*>(a.q) +
                    (static_cast<int64_t>(b) * a.num_heads + h0 + min(r, nh - 1)) * D + 8 * c;
    float f[kOwn][8];
    load_pages(0);
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      if (warp + i * kWarps < NB) load_row<T, 8>(qrow + 32 * (warp + i * kWarps), f[i]);
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) {
      if (i < stages) {
        issue(i, smem_addr(ring + i * C::kStage));
        load_pages(i + 1);
      }
      copies_commit();
    }
    // the largest |q| of each head; fragments; sums over blocks
    float largest = 0.f;
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      if (warp + i * kWarps < NB)
#pragma unroll
        for (int e = 0; e < 8; ++e) largest = fmaxf(largest, fabsf(f[i][e]));
    largest = fmaxf(largest, __shfl_xor_sync(kAll, largest, 1));
    largest = fmaxf(largest, __shfl_xor_sync(kAll, largest, 2));
    if (c == 0 && warp < NB) stat[warp * 8 + r] = largest;
    if (threadIdx.x == 0) bad_s = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < (kWarps < NB ? kWarps : NB); ++w)
      largest = fmaxf(largest, stat[w * 8 + r]);
    // queries of 2^116 and more become infinite in f16, and their rows NaN
    const int shift = min(max(14 - exponent(largest), -100), 126);
    // the sign of the logits' scale goes with q, so that larger products are larger logits
    const float by = a.scale_log2 > 0.f   ? pow2(shift)
                     : a.scale_log2 < 0.f ? -pow2(shift)
                                          : a.scale_log2 * pow2(shift);
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int u = warp + i * kWarps;
      if (u >= NB) break;
      float total = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[i][e] = r < nh ? f[i][e] * by : 0.f;
        total += f[i][e];
      }
      // the high halves' elements meet codes 2^4 as large
      constexpr float k16 = 1.f / 16;
      qf[u * 32 + lane] = make_uint4(pack<__half>(f[i][0], f[i][4]), pack<__half>(f[i][2], f[i][6]),
                                     pack<__half>(f[i][1] * k16, f[i][5] * k16),
                                     pack<__half>(f[i][3] * k16, f[i][7] * k16));
      total += __shfl_xor_sync(kAll, total, 1);
      total += __shfl_xor_sync(kAll, total, 2);
      if (c == 0) qs[u * 8 + r] = total;
    }
    // the factor of a logit of this lane's heads 2c, 2c + 1
    float lf[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      lf[e] = fminf(fmaxf(fabsf(a.scale_log2) * pow2(min(24 - __shfl_sync(kAll, shift, (2 * c + e) * 4),
                                                  127)), 0x1p-126f), 0x1p127f);
    __syncthreads();
    // The warp with the fewest tiles looks the next item up (256 sequences up to 100K 640 to 628
    // us, 500 up to 2000 107 to 105; with its pages' ids as well 632).  Wide CTAs have one, mostly.
    if (!kWide && warp == kWarps - 1 && next_s < items) {
      int nb;
      uint32_t np;
      list_find(list, a.num_seqs, parts, next_s / per, nb, np);
      const int32_t nl = __ldg(a.lens + nb);
      if (lane == 0) next_b_s = nb, next_part_s = np, next_len_s = nl;
    }
    // The sums of q over groups 2c and 2c + 1 of head r, as B of the product with the
    // minima: three bf16 or two f16 parts.  f16: times 2^16, at most 2^14.
    uint32_t qb[kParts];
    {
      float g[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        g[e] = 0.f;
        if (2 * c + e < NP)
#pragma unroll
          for (int u = 0; u < GS / 32; ++u) g[e] += qs[((2 * c + e) * (GS / 32) + u) * 8 + r];
        g[e] *= 0x1p-24f * kMinUp;
      }
#pragma unroll
      for (int i = 0; i < kParts; ++i) qb[i] = split<T>(g[0], g[1]);
    }

    // ---- the part -----------------------------------------------------------------------
    // o: tiles of a block, rows r and r + 8 the elements 4 r + 2 t and 4 r + 2 t + 1.  eights: row
    // r is group r.  sums: rows r are the minima of group r, r + 8 its scales.
    // lim, up: of group lane % NP, the bound of its scales and what they are taken times.
    float o[NB][2][4], eights[4], sums[4], lim = 0.f, up = 0.f;
    float ref[2] = {-INFINITY, -INFINITY}, bar[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][t][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) eights[e] = sums[e] = 0.f;

    // this lane's row and 16 bytes for LDSM: two blocks of 16 tokens
    const uint32_t ldsm_at = (lane & 15) * C::KP + (lane >> 4) * 16;
    // where this lane's scales go: token lane / NP (and on), group lane % NP
    const int scale_at = (lane / (2 * NP) * NP + lane % NP) * 2 + lane / NP % 2;
    uint8_t* st = ring;                                     // this stage, and
    uint8_t* refill = ring + (C::kStages - 1) * C::kStage;  // the one before it
    for (int i = 0; i < stages; ++i) {
      copies_wait<C::kStages - 2>();
      __syncwarp();  // this stage has landed for all lanes, and the one to refill is read
      if (i + C::kStages - 1 < stages) {
        issue(i + C::kStages - 1, smem_addr(refill));
        load_pages(i + C::kStages);
      }
      copies_commit();
      const int n = t1 - (t0 + (i * kWarps + warp) * C::ROWS);  // tokens, if fewer than ROWS

      // logits of rows r, r + 8 and heads 2c, 2c + 1
      float l[MT][4];
      {
        uint32_t kw[MT][2][NP];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const uint8_t* at = st + C::kKs + (16 * mt + r) * C::SB;
          load_words(at, kw[mt][0]);
          load_words(at + 8 * C::SB, kw[mt][1]);
          // minima times the sums of q; groups past the last meet zeros
          uint32_t m0, m1;
          if constexpr (NP == 1) {
            m0 = __byte_perm(kw[mt][0][0], 0, 0x3232);
            m1 = __byte_perm(kw[mt][1][0], 0, 0x3232);
          } else {
            uint32_t w0[2], w1[2];
            const int g = 2 * c % NP * 4;
            load_words(at + g, w0);
            load_words(at + 8 * C::SB + g, w1);
            m0 = __byte_perm(w0[0], w0[1], 0x7632);
            m1 = __byte_perm(w1[0], w1[1], 0x7632);
          }
          mma0<T>(l[mt], m0, m1, 0, 0, qb[0], 0);
#pragma unroll
          for (int i = 1; i < kParts; ++i) mma<T>(l[mt], m0, m1, 0, 0, qb[i], 0);
          if constexpr (kMinUp != 1.f)
#pragma unroll
            for (int e = 0; e < 4; ++e) l[mt][e] *= 1.f / kMinUp;
        }
        constexpr int kPer = GS < 64 ? 1 : 2;  // blocks that an accumulator sums
#pragma unroll
        for (int j = 0; j < NB; j += 2) {
          const uint4 q0 = qf[j * 32 + lane], q1 = qf[(j + 1) * 32 + lane];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            // words of blocks j (rows r, r + 8) and j + 1
            uint32_t w[4];
            ldsm<false>(w, smem_addr(st) + 16 * mt * C::KP + ldsm_at + 16 * j);
            float acc[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t lo = w[2 * h], hi = w[2 * h + 1], lo8 = lo >> 8, hi8 = hi >> 8;
              const uint4 q = h ? q1 : q0;
              float (&x)[4] = acc[kPer == 2 ? 0 : h];
              if (h == 0 || kPer == 1)
                mma0<__half>(x, lo & kLow, hi & kLow, lo8 & kLow, hi8 & kLow, q.x, q.y);
              else
                mma<__half>(x, lo & kLow, hi & kLow, lo8 & kLow, hi8 & kLow, q.x, q.y);
              mma<__half>(x, lo & kHigh, hi & kHigh, lo8 & kHigh, hi8 & kHigh, q.z, q.w);
            }
#pragma unroll
            for (int h = 0; h < 2 / kPer; ++h) {
              const float s0 = scale_of<T>(kw[mt][0][(j + h) * 32 / GS]);
              const float s1 = scale_of<T>(kw[mt][1][(j + h) * 32 / GS]);
              l[mt][0] = fmaf(s0, acc[h][0], l[mt][0]);
              l[mt][1] = fmaf(s0, acc[h][1], l[mt][1]);
              l[mt][2] = fmaf(s1, acc[h][2], l[mt][2]);
              l[mt][3] = fmaf(s1, acc[h][3], l[mt][3]);
            }
          }
        }
      }
      if (n < C::ROWS) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (16 * mt + r + (e & 2) * 4 >= n) l[mt][e] = -INFINITY;
      }

      // does a logit pass the reference, or a scale its power?
      bool moves = false;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) moves = moves || l[mt][e] > bar[e & 1];
      constexpr int kScales = C::ROWS * NP / 32;  // of the stage, a lane's; of group lane % NP
      const uint32_t* vpairs = reinterpret_cast<const uint32_t*>(st + C::kVs);
      float vs[kScales];
#pragma unroll
      for (int u = 0; u < kScales; ++u) {
        vs[u] = scale_of<T>(vpairs[u * 32 + lane]);
        moves = moves || fabsf(vs[u]) > lim;
      }
      if (__any_sync(kAll, moves)) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = ref[e];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) top = fmaxf(top, fmaxf(l[mt][e], l[mt][e + 2]) * lf[e]);
#pragma unroll
          for (int s = 4; s <= 16; s <<= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, s));
          const bool m = top > ref[e] + kBar;
          f[e] = m ? ex2(ref[e] - top) : 1.f;  // 0 where nothing has been seen
          if (m) ref[e] = top;
          bar[e] = (ref[e] + kBar) / lf[e];
          sum[e] *= f[e];
        }
        // the groups' powers
        float most = 0.f;
#pragma unroll
        for (int u = 0; u < kScales; ++u) most = fmaxf(most, fabsf(vs[u]));
#pragma unroll
        for (int s = NP; s <= 16; s <<= 1) most = fmaxf(most, __shfl_xor_sync(kAll, most, s));
        float g = 1.f;
        if (most > lim) {
          const float to = pow2(min(max(exponent(most) + 1, -120), 127));
          if (lim > 0.f) g = lim / to;
          lim = to;
          up = pow2(kTop - exponent(to));
        }
        // The first stage has zeros to scale.  Passing them by, us: 64 sequences of 6000, 24 / 4
        // heads of 256, 105.5 to 102.9; 33 sequences of bf16, groups of 32, 169.2 to 163.4, of f16
        // 160.6 to 161.1.
        if (i > 0) {
          float ge = 1.f;
#pragma unroll
          for (int j = 0; j < NP; ++j) {
            const float gj = __shfl_sync(kAll, g, j);
            if (j == r) ge = gj;
#pragma unroll
            for (int i = j * (GS / 32); i < (j + 1) * (GS / 32); ++i)
#pragma unroll
              for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][t][e] *= f[e & 1] * gj;
          }
          eights[0] *= f[0] * ge;
          eights[1] *= f[1] * ge;
#pragma unroll
          for (int e = 0; e < 4; ++e) sums[e] *= f[e & 1];
        }
      }

      // weights, and their transposition: heads as rows, tokens as columns
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = ex2(fmaf(l[mt][e], lf[e & 1], kUp - ref[e & 1]));
          sum[e & 1] += p;
          pt[(2 * c + (e & 1)) * C::PP + 16 * mt + r + (e & 2) * 4] = p;
        }
      // the scales, tokens side by side: [token pair][group][2], where the keys' pairs were
      __syncwarp();  // that all lanes have read
      float* ts = reinterpret_cast<float*>(st + C::kKs);
#pragma unroll
      for (int u = 0; u < kScales; ++u) ts[scale_at + u * 32] = vs[u] * up;
      __syncwarp();

#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const float2 pa = *reinterpret_cast<const float2*>(pt + r * C::PP + 16 * mt + 2 * c);
        const float2 pb = *reinterpret_cast<const float2*>(pt + r * C::PP + 16 * mt + 2 * c + 8);
        const uint32_t at = smem_addr(st) + C::kV + 16 * mt * C::KP + ldsm_at;
        const uint8_t* sc = st + C::kVs + (16 * mt + 2 * c) * C::SB;
        // scales of tokens 2c, 2c + 1 and 2c + 8, 2c + 9
        const float2* sa = reinterpret_cast<const float2*>(ts) + (8 * mt + c) * NP;
        const float2* sb = sa + 4 * NP;
        {
          // weights, in two parts of 16 bits, times minima and scales: group r % NP
          uint32_t w[4];
          const int g = r % NP;
          const uint32_t* x = reinterpret_cast<const uint32_t*>(sc) + g;
          w[0] = x[0], w[1] = x[NP], w[2] = x[8 * NP], w[3] = x[9 * NP];
          const uint32_t m0 = __byte_perm(w[0], w[1], 0x7632);
          const uint32_t m1 = __byte_perm(w[0], w[1], 0x5410);
          const uint32_t m2 = __byte_perm(w[2], w[3], 0x7632);
          const uint32_t m3 = __byte_perm(w[2], w[3], 0x5410);
          float2 la = pa, lb = pb;
          const uint32_t h0 = split<T>(la.x, la.y), h1 = split<T>(lb.x, lb.y);
          mma<T>(sums, m0, m1, m2, m3, h0, h1);
          mma<T>(sums, m0, m1, m2, m3, pack<T>(la.x, la.y), pack<T>(lb.x, lb.y));
        }
        uint32_t b0 = 0, b1 = 0;  // p s of the group, by MMA columns
#pragma unroll
        for (int j = 0; j < NB; j += 2) {
          // two tokens' 16 bits of blocks j and j + 1: the transpose weaves them
          uint32_t w[4];
          ldsm<true>(w, at + 16 * j);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if ((j + h) * 32 % GS == 0) {
              const int g = (j + h) * 32 / GS;
              b0 = products(pa, sa[g]);
              b1 = products(pb, sb[g]);
              const uint32_t eight = g == r ? 0x00080008u : 0u;
              mma<__half>(eights, eight, 0, eight, 0, b0, b1);
            }
            const uint32_t x0 = w[2 * h], x1 = w[2 * h + 1], y0 = x0 >> 8, y1 = x1 >> 8;
            mma<__half>(o[j + h][0], x0 & kLow, x0 & kHigh, x1 & kLow, x1 & kHigh, b0, b1);
            mma<__half>(o[j + h][1], y0 & kLow, y0 & kHigh, y1 & kLow, y1 & kHigh, b0, b1);
          }
        }
      }
      __syncwarp();  // pt is written again
      refill = st;
      st = st == ring + (C::kStages - 1) * C::kStage ? ring : st + C::kStage;
    }
    copies_wait<0>();

    // ---- join of the warps ------------------------------------------------------------------
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int s = 4; s <= 16; s <<= 1) sum[e] += __shfl_xor_sync(kAll, sum[e], s);
    if (bad) bad_s = 1;
    if (r == 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        stat[warp * 8 + 2 * c + e] = ref[e];
        stat[(kWarps + warp) * 8 + 2 * c + e] = sum[e];
      }
    }
    __syncwarp();
    float* mine = reinterpret_cast<float*>(ring);  // [8][D]: the warp is done with its ring
#pragma unroll
    for (int g = 0; g < NP; ++g) {
      const float u = __shfl_sync(kAll, up, g), down = u > 0.f ? 1.f / u : 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float ex = fmaf(8.f, __shfl_sync(kAll, sums[e + 2], g * 4 + c),
                              __shfl_sync(kAll, sums[e], g * 4 + c));
        const float ei = __shfl_sync(kAll, eights[e], g * 4 + c) * 0x1p24f;
#pragma unroll
        for (int j = g * (GS / 32); j < (g + 1) * (GS / 32); ++j)
          *reinterpret_cast<float4*>(mine + (2 * c + e) * D + 32 * j + 4 * r) =
              make_float4(fmaf(o[j][0][e] * 0x1p24f - ei, down, ex),
                          fmaf(o[j][0][e + 2] * 0x1p20f - ei, down, ex),
                          fmaf(o[j][1][e] * 0x1p24f - ei, down, ex),
                          fmaf(o[j][1][e + 2] * 0x1p20f - ei, down, ex));
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nh * (D / 4); i += kNT) {
      const int h = i / (D / 4), d = i % (D / 4);
      float M = -INFINITY, total = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, stat[w * 8 + h]);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        // a warp's weight beside the largest reference; one without a token weighs nothing
        const float m = stat[w * 8 + h], s = stat[(kWarps + w) * 8 + h];
        const float x = m == -INFINITY ? (s == 0.f ? 0.f : qnan()) : ex2(m - M);
        const float4 y = *reinterpret_cast<const float4*>(
            smem + w * (C::kStages * C::kStage) + (h * D + 4 * d) * 4);
        total = fmaf(s, x, total);
        v.x = fmaf(y.x, x, v.x);
        v.y = fmaf(y.y, x, v.y);
        v.z = fmaf(y.z, x, v.z);
        v.w = fmaf(y.w, x, v.w);
      }
      const float inv = bad_s ? qnan() : 1.f / total;
      v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
      const int64_t row = static_cast<int64_t>(b) * a.num_heads + h0 + h;
      if (direct) {
        store_out4(a.out, row * D + 4 * d, a.out_dtype, v);
      } else {
        const int64_t at = row * a.num_parts + part;
        reinterpret_cast<float4*>(a.part_out)[at * (D / 4) + d] = v;
        if (d == 0) {
          a.part_max[at] = bad_s ? qnan() : M;
          a.part_sum[at] = total * 0x1p-8f;  // 2^-kUp
        }
      }
    }
    if (bad_s && threadIdx.x == 0) set_status(a.status, PA_ERR_BAD_BLOCK_ID);
    item = next_s;
    if (!kWide) b = next_b_s, part = next_part_s, L = next_len_s;
    found = !kWide;
    __syncthreads();  // the ring, the statistics and q are written again
  }
  if (queued && threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(&queue->done, 1u) == gridDim.x - 1) {
      queue->next = 0;
      queue->done = 0;
    }
  }
}

template <typename T, int D, int GS, bool kWide>
cudaError_t launch_w(Kv4Args a, int64_t items, int dev, int sms, cudaStream_t s) {
  using C = Cfg<D, GS, kWide>;
  static std::atomic<bool> configured[128];
  const auto kern = pa_kv4_tc_kernel<T, D, GS, kWide>;
  constexpr int kMost = C::kOffList + (65536 / kListSpan + 1) * 4;  // the longest list
  static_assert(kMost <= 227 * 1024, "shared memory of a CTA");
  if (dev >= 128 || !configured[dev].load(std::memory_order_acquire)) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
    if (dev < 128) configured[dev].store(true, std::memory_order_release);
  }
  a.room = sms * C::kCtas;
  kern<<<static_cast<unsigned>(items < a.room ? items : a.room), C::kNT,
         C::kOffList + list_bytes(a.num_seqs), s>>>(a);
  return cudaGetLastError();
}

template <typename T, int D, int GS>
cudaError_t launch_d(const Kv4Args& a, int64_t items, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t pairs = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads * a.head_groups;
  // Wide CTAs: fewer, larger parts and one join of their warps, where a pair is one part or
  // the pairs are few and long.  Measured, us, wide and narrow: one part, 32 / 8 heads of 128,
  // eight sequences of 128 tokens 6.9 and 5.5, 256 7.3 and 6.6, 320 7.6 and 7.7, 400 8.3 and
  // 8.9, 1000 11.3 and 13.2; in parts, 24 / 4 of 256, one of 4000 11.1 and 10.3, 6000 11.8 and
  // 12.0, 100K 32.3 and 34.0; two of 100K 50.9 and 51.6, four of 32000 (16 pairs) 38.7 and 37.1,
  // eight of 20000 49.9 and 44.2.
  const bool wide = a.num_parts == 1 ? 2 * pairs <= sms && a.max_len > 320
                                     : 16 * pairs <= sms && a.max_len > 6000;
  return wide ? launch_w<T, D, GS, true>(a, items, dev, sms, s)
              : launch_w<T, D, GS, false>(a, items, dev, sms, s);
}

template <typename T>
cudaError_t launch(const Kv4Args& a, int64_t items, cudaStream_t s) {
  switch (a.head_dim * 256 + a.group_size) {
    case 64 * 256 + 32: return launch_d<T, 64, 32>(a, items, s);
    case 64 * 256 + 64: return launch_d<T, 64, 64>(a, items, s);
    case 128 * 256 + 32: return launch_d<T, 128, 32>(a, items, s);
    case 128 * 256 + 64: return launch_d<T, 128, 64>(a, items, s);
    case 128 * 256 + 128: return launch_d<T, 128, 128>(a, items, s);
    case 256 * 256 + 32: return launch_d<T, 256, 32>(a, items, s);
    case 256 * 256 + 64: return launch_d<T, 256, 64>(a, items, s);
    default: return launch_d<T, 256, 128>(a, items, s);
  }
}

}  // namespace kv4
}  // namespace pa
