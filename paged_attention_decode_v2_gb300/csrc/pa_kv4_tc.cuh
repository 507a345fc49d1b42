// pa_kv4_tc.cuh -- tensor-core decode over the 4-bit cache, bf16 and f16.
//
// A work item is a part of a sequence, a KV head and up to eight of its query
// heads.  The four warps of a CTA take its tiles of 16 (head_dim 256) or 32 tokens
// in turn, each with a ring of its own (cp.async, no barrier between warps) and
// running statistics of its own; they are joined at the end of the item.
//
// Codes never become values.  With k = s c + m,
//   q . k = sum_g s_g (sum_g q c) + m_g (sum_g q),
// so the MMA multiplies q by codes, and a group's scale and minimum enter in
// float32, once per token, group and head.  With v = s (c - 8) + (m + 8 s),
//   sum_t p v = sum_t (p s) c - 8 sum_t (p s) + sum_t p (m + 8 s),
// so p s is what the second MMA multiplies by codes; its own sum comes from an MMA
// with rows of eights, the last sum is float32 on the CUDA cores.
//   * A code in the low half of a byte, masked, is the f16 subnormal c 2^-24, in the
//     high half c 2^-20: one mask makes two operands of a 32-bit word, and the powers
//     of two leave with the scales.
//   * Keys are the 16 x 16 operand A (16 tokens), q is B (8 heads), scaled per head by
//     a power of two to below 2^15: exact, but for elements 2^-24 below the largest.
//     The 16 elements of an MMA are those a lane finds in its words, q in that order.
//   * Values are A with rows d and columns t: two tokens' words are woven by PRMT.
//     B is p s, rounded to f16: a half step, 2^-11 of each weight, on c - 8 and not on
//     c, since the eights are multiplied by the rounded weights too.  p s is scaled by
//     a power of two per group that follows the largest scale seen.
//   * The reference of the softmax moves when a logit passes it by 2^8, the scales'
//     power when a scale passes it: one vote a tile, no reduction otherwise.
// All sums are float32.
//
// Bound by instructions rather than memory: of 16 tokens x 64 elements a lane has 32
// codes of each kind, about 40 instructions for keys and 50 for values.
#pragma once

#include <atomic>

#include "pa_kv4.cuh"

namespace pa {
namespace kv4 {

constexpr int kWarps = 4;
constexpr int kNT = kWarps * 32;
constexpr unsigned kAll = 0xffffffffu;

template <int D, int GS>
struct Cfg {
  static constexpr int CH = GS < 64 ? GS : 64;  // elements that an accumulator sums
  static constexpr int NCH = D / CH;
  static constexpr int W = CH / 32;             // words of a chunk that a lane has
  static constexpr int NP = D / GS;             // pairs of a head row
  static constexpr int SB = NP * 4;             //   and their bytes
  static constexpr int MT = D >= 128 ? 1 : 2;   // 16-token tiles of a stage
  static constexpr int ROWS = 16 * MT;
  // Pitches that spread a warp's reads over the banks: keys by 8-byte (4-byte for
  // groups of 32) reads of 8 rows, values by 4-byte reads of rows 2 apart.
  static constexpr int KP = CH == 32 ? D / 2 + 16 : D == 64 ? 32 : D / 2 + 32;
  static constexpr int VP = D / 2 + 16;
  static constexpr int kV = ROWS * KP;
  static constexpr int kKs = kV + ROWS * VP;
  static constexpr int kVs = kKs + ROWS * SB;
  static constexpr int kStage = kVs + ROWS * SB;
  static constexpr int kStages = D == 128 ? 4 : 3;
  static constexpr int PP = ROWS + 4;           // pitch of the weights' transposition
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kQ = D / 32 * 512;       // q fragments
  static constexpr int kOffQ = kRing;
  static constexpr int kOffQs = kOffQ + kQ;                  // sums of q: [NCH][8]
  static constexpr int kOffP = kOffQs + NCH * 8 * 4;         // weights: [warp][8][PP]
  static constexpr int kOffW = kOffP + kWarps * 8 * PP * 4;  // statistics: [4][warp][8]
  static constexpr int kOffList = kOffW + 4 * kWarps * 8 * 4;
  static constexpr int kCtas = kv4_tc_ctas(D);  // resident on an SM
  static_assert((kOffList + 1024 + 1024) * kCtas <= 228 * 1024, "resident CTAs");
  static_assert(kRing >= kWarps * 8 * D * 4, "the join uses the ring");
  static_assert(kStage % 16 == 0 && KP % 16 == 0 && VP % 16 == 0, "16-byte copies");
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// `bytes` of 16 from src, the rest zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes));
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

// c (16 x 8, f32) += a (16 x 16) * b (16 x 8), f16
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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
__device__ __forceinline__ uint32_t f16x2(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
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

// Parts of sequence b: those with a token; one for a row that the item itself has to
// finish (direct: no join follows).
struct Parts {
  const Kv4Args& a;
  __device__ __forceinline__ uint32_t operator()(int b) const {
    const int32_t L = __ldg(a.lens + b);
    const bool some = kv4_len_ok(a, L) && L > 0;
    return some ? (L + a.part_size - 1) / a.part_size : a.num_parts == 1;
  }
};

template <typename T, int D, int GS>
__global__ void __launch_bounds__(kNT, Cfg<D, GS>::kCtas) pa_kv4_tc_kernel(const Kv4Args a) {
  using C = Cfg<D, GS>;
  constexpr int NCH = C::NCH, MT = C::MT, W = C::W, NP = C::NP, CH = C::CH;
  constexpr int kTiles = CH / 16;  // MMA tiles of a chunk's values
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int bad_s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, c = lane & 3;  // row of A, or head of B; column pair
  uint8_t* ring = smem + warp * (C::kStages * C::kStage);
  uint4* qf = reinterpret_cast<uint4*>(smem + C::kOffQ);
  float* qs = reinterpret_cast<float*>(smem + C::kOffQs);
  float* pt = reinterpret_cast<float*>(smem + C::kOffP) + warp * (8 * C::PP);
  float* stat = reinterpret_cast<float*>(smem + C::kOffW);  // [4][kWarps][8]
  uint32_t* list = reinterpret_cast<uint32_t*>(smem + C::kOffList);

  cudaTriggerProgrammaticLaunchCompletion();  // the join waits for this grid's end itself
  const Parts parts{a};
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.num_seqs; b += kNT)
      if (!kv4_len_ok(a, __ldg(a.lens + b))) set_status(a.status, PA_ERR_BAD_SEQ_LEN);
  const uint32_t per = a.num_kv_heads * a.head_groups;
  const uint32_t items = list_build(list, a.num_seqs, parts) * per;
  const bool direct = a.num_parts == 1;

  for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
    int b;
    uint32_t part;
    const uint32_t sp = item / per, x = item - sp * per;
    list_find(list, a.num_seqs, parts, sp, b, part);
    const int kvh = x / a.head_groups, hg = x - kvh * a.head_groups;
    const int nh = min(kKv4Heads, a.group - hg * kKv4Heads);
    const int h0 = kvh * a.group + hg * kKv4Heads;
    const int32_t L = __ldg(a.lens + b);
    if (!kv4_len_ok(a, L) || L == 0) {
      for (int i = threadIdx.x; i < nh * D; i += kNT)
        kv4_finish(a, b, h0 + i / D, 0, i % D, D, true, L, L != 0, 0.f, 1.f, 0.f);
      continue;
    }
    const int32_t t0 = part * a.part_size, t1 = min(L, t0 + a.part_size);
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
    const auto issue = [&](int i) {
      const uint32_t dst = smem_addr(ring + i % C::kStages * C::kStage);
      const int32_t ts = t0 + (i * kWarps + warp) * C::ROWS;
      if (a.paged16) {
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
            copy16(dst + C::kV + (16 * mt + rr) * C::VP + piece * 16, vc + idx * 16, bytes);
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
          copy16(dst + C::kV + rr * C::VP + piece * 16, a.v_codes + at, ok ? 16 : 0);
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
    load_pages(0);
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) {
      if (i < stages) {
        issue(i);
        load_pages(i + 1);
      }
      copies_commit();
    }

    // ---- q: fragments, and its sums over chunks ---------------------------------------
    // Unit u = (chunk j, word i) holds a lane's elements d0 .. d0 + 7; warps take units in
    // turn.  The largest |q| of each head first.
    const T* qrow = static_cast<const T*>(a.q) +
                    (static_cast<int64_t>(b) * a.num_heads + h0 + min(r, nh - 1)) * D;
    const auto first = [&](int u) { return u / W * CH + c * (CH / 4) + u % W * 8; };
    constexpr int kUnits = D / 32;
    float largest = 0.f;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      if (u % kWarps != warp) continue;
      float f[8];
      load_row<T, 8>(qrow + first(u), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) largest = fmaxf(largest, fabsf(f[e]));
    }
    largest = fmaxf(largest, __shfl_xor_sync(kAll, largest, 1));
    largest = fmaxf(largest, __shfl_xor_sync(kAll, largest, 2));
    if (c == 0) stat[warp * 8 + r] = largest;
    if (threadIdx.x == 0) bad_s = 0;
    for (int i = threadIdx.x; i < NCH * 8; i += kNT) qs[i] = 0.f;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) largest = fmaxf(largest, stat[w * 8 + r]);
    const int shift = min(14 - exponent(largest), 126);
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      if (u % kWarps != warp) continue;
      float f[8], sum = 0.f;
      load_row<T, 8>(qrow + first(u), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[e] = r < nh ? f[e] * pow2(shift) : 0.f;
        sum += f[e];
      }
      // the high halves' elements meet codes 2^4 as large
      constexpr float k16 = 1.f / 16;
      qf[u * 32 + lane] = make_uint4(f16x2(f[0], f[4]), f16x2(f[2], f[6]),
                                     f16x2(f[1] * k16, f[5] * k16), f16x2(f[3] * k16, f[7] * k16));
      sum += __shfl_xor_sync(kAll, sum, 1);
      sum += __shfl_xor_sync(kAll, sum, 2);
      if constexpr (W == 1) {
        if (c == 0) qs[u * 8 + r] = sum * 0x1p-24f;
      } else {
        if (c == 0) atomicAdd(&qs[u / W * 8 + r], sum * 0x1p-24f);  // two terms: any order
      }
    }
    // the factor of a logit of this lane's heads 2c, 2c + 1
    float lf[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      lf[e] = a.scale_log2 * pow2(min(24 - __shfl_sync(kAll, shift, (2 * c + e) * 4), 127));
    __syncthreads();

    // ---- the part -----------------------------------------------------------------------
    float o[NCH][kTiles][4], eights[4], extra[NCH], lim = 0.f, up[NCH];
    float ref[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      extra[j] = up[j] = 0.f;
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][t][e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) eights[e] = 0.f;

    for (int i = 0; i < stages; ++i) {
      copies_wait<C::kStages - 2>();
      __syncwarp();  // this stage has landed for all lanes, and the one to refill is read
      if (i + C::kStages - 1 < stages) {
        issue(i + C::kStages - 1);
        load_pages(i + C::kStages);
      }
      copies_commit();
      const uint8_t* st = ring + i % C::kStages * C::kStage;
      const int n = t1 - (t0 + (i * kWarps + warp) * C::ROWS);  // tokens, if fewer than ROWS

      // logits of rows r, r + 8 and heads 2c, 2c + 1
      float l[MT][4];
      {
        uint32_t kw[MT][2][NP];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          load_words(st + C::kKs + (16 * mt + r) * C::SB, kw[mt][0]);
          load_words(st + C::kKs + (16 * mt + r + 8) * C::SB, kw[mt][1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) l[mt][e] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
          uint4 qv[W];
#pragma unroll
          for (int w = 0; w < W; ++w) qv[w] = qf[(j * W + w) * 32 + lane];
          const float2 s2 = *reinterpret_cast<const float2*>(qs + j * 8 + 2 * c);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const uint8_t* at = st + (16 * mt + r) * C::KP + j * (CH / 2) + c * (4 * W);
            uint32_t lo[W], hi[W];
            load_words(at, lo);
            load_words(at + 8 * C::KP, hi);
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < W; ++w) {
              const uint32_t lo8 = lo[w] >> 8, hi8 = hi[w] >> 8;
              mma(acc, lo[w] & kLow, hi[w] & kLow, lo8 & kLow, hi8 & kLow, qv[w].x, qv[w].y);
              mma(acc, lo[w] & kHigh, hi[w] & kHigh, lo8 & kHigh, hi8 & kHigh, qv[w].z, qv[w].w);
            }
            const float2 p0 = widen_pair<T>(kw[mt][0][j * CH / GS]);
            const float2 p1 = widen_pair<T>(kw[mt][1][j * CH / GS]);
            l[mt][0] = fmaf(p0.y, s2.x, fmaf(p0.x, acc[0], l[mt][0]));
            l[mt][1] = fmaf(p0.y, s2.y, fmaf(p0.x, acc[1], l[mt][1]));
            l[mt][2] = fmaf(p1.y, s2.x, fmaf(p1.x, acc[2], l[mt][2]));
            l[mt][3] = fmaf(p1.y, s2.y, fmaf(p1.x, acc[3], l[mt][3]));
          }
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) l[mt][e] *= lf[e & 1];
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
        for (int e = 0; e < 4; ++e) moves = moves || l[mt][e] > ref[e & 1] + 8.f;
      constexpr int kScales = C::ROWS * NP;  // pairs of the stage; lane's are of group lane % NP
      const uint32_t* vpairs = reinterpret_cast<const uint32_t*>(st + C::kVs);
#pragma unroll
      for (int u = 0; u < (kScales + 31) / 32; ++u)
        if (kScales % 32 == 0 || u * 32 + lane < kScales)
          moves = moves || fabsf(widen_pair<T>(vpairs[u * 32 + lane]).x) > lim;
      if (__any_sync(kAll, moves)) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = ref[e];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) top = fmaxf(top, fmaxf(l[mt][e], l[mt][e + 2]));
#pragma unroll
          for (int s = 4; s <= 16; s <<= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, s));
          const bool m = top > ref[e] + 8.f;
          f[e] = m ? ex2(ref[e] - top) : 1.f;  // 0 where nothing has been seen
          if (m) ref[e] = top;
          sum[e] *= f[e];
        }
        // head r's factor, for the sums that lie by head
        const float f0 = __shfl_sync(kAll, f[0], r >> 1), f1 = __shfl_sync(kAll, f[1], r >> 1);
        const float fr = r & 1 ? f1 : f0;
        // the groups' powers
        float most = 0.f;
#pragma unroll
        for (int u = 0; u < (kScales + 31) / 32; ++u)
          if (kScales % 32 == 0 || u * 32 + lane < kScales)
            most = fmaxf(most, fabsf(widen_pair<T>(vpairs[u * 32 + lane]).x));
#pragma unroll
        for (int s = NP; s <= 16; s <<= 1) most = fmaxf(most, __shfl_xor_sync(kAll, most, s));
        float g = 1.f;
        if (most > lim) {
          const float to = pow2(min(max(exponent(most) + 1, -119), 127));
          if (lim > 0.f) g = lim / to;
          lim = to;
        }
        float ge = 1.f;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
          const float gj = __shfl_sync(kAll, g, j * CH / GS);
          const float lj = __shfl_sync(kAll, lim, j * CH / GS);
          up[j] = lj > 0.f ? pow2(7 - exponent(lj)) : 0.f;
          if (j == r) ge = gj;
          extra[j] *= fr;
#pragma unroll
          for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][t][e] *= f[e & 1] * gj;
        }
        eights[0] *= f[0] * ge;
        eights[1] *= f[1] * ge;
      }

      // weights, and their transposition: heads as rows, tokens as columns
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = ex2(l[mt][e] - ref[e & 1]);
          sum[e & 1] += p;
          pt[(2 * c + (e & 1)) * C::PP + 16 * mt + r + (e & 2) * 4] = p;
        }
      __syncwarp();

#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const float2 pa = *reinterpret_cast<const float2*>(pt + r * C::PP + 16 * mt + 2 * c);
        const float2 pb = *reinterpret_cast<const float2*>(pt + r * C::PP + 16 * mt + 2 * c + 8);
        const uint8_t* at = st + C::kV + (16 * mt + 2 * c) * C::VP;
        const uint8_t* sc = st + C::kVs + (16 * mt + 2 * c) * C::SB;
        uint32_t vw[4][NP];
        load_words(sc, vw[0]);
        load_words(sc + C::SB, vw[1]);
        load_words(sc + 8 * C::SB, vw[2]);
        load_words(sc + 9 * C::SB, vw[3]);
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
          const float2 p0 = widen_pair<T>(vw[0][j * CH / GS]);
          const float2 p1 = widen_pair<T>(vw[1][j * CH / GS]);
          const float2 p2 = widen_pair<T>(vw[2][j * CH / GS]);
          const float2 p3 = widen_pair<T>(vw[3][j * CH / GS]);
          extra[j] = fmaf(pa.x, fmaf(8.f, p0.x, p0.y), extra[j]);
          extra[j] = fmaf(pa.y, fmaf(8.f, p1.x, p1.y), extra[j]);
          extra[j] = fmaf(pb.x, fmaf(8.f, p2.x, p2.y), extra[j]);
          extra[j] = fmaf(pb.y, fmaf(8.f, p3.x, p3.y), extra[j]);
          const uint32_t b0 = f16x2(pa.x * (p0.x * up[j]), pa.y * (p1.x * up[j]));
          const uint32_t b1 = f16x2(pb.x * (p2.x * up[j]), pb.y * (p3.x * up[j]));
          const uint32_t eight = j == r ? 0x00080008u : 0u;
          mma(eights, eight, 0, eight, 0, b0, b1);
          // a lane's word of the chunk, and for groups of 32 its half of it
          const int word = j * (CH / 8) + (W == 2 ? r : r >> 1);
          const uint32_t w0 = *reinterpret_cast<const uint32_t*>(at + 4 * word);
          const uint32_t w1 = *reinterpret_cast<const uint32_t*>(at + C::VP + 4 * word);
          const uint32_t w2 = *reinterpret_cast<const uint32_t*>(at + 8 * C::VP + 4 * word);
          const uint32_t w3 = *reinterpret_cast<const uint32_t*>(at + 9 * C::VP + 4 * word);
#pragma unroll
          for (int h = 0; h < W; ++h) {
            const uint32_t pick = (W == 2 ? h : r & 1) ? 0x7632u : 0x5410u;
            const uint32_t x0 = __byte_perm(w0, w1, pick), x1 = __byte_perm(w2, w3, pick);
            mma(o[j][2 * h], x0 & kLow, x0 & kHigh, x1 & kLow, x1 & kHigh, b0, b1);
            mma(o[j][2 * h + 1], x0 >> 8 & kLow, x0 >> 8 & kHigh, x1 >> 8 & kLow,
                x1 >> 8 & kHigh, b0, b1);
          }
        }
      }
      __syncwarp();  // pt is written again
    }
    copies_wait<0>();

    // ---- join of the warps ------------------------------------------------------------------
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int s = 4; s <= 16; s <<= 1) sum[e] += __shfl_xor_sync(kAll, sum[e], s);
    if (bad) bad_s = 1;
    __syncthreads();  // all warps are done with the ring; bad_s
    if (r == 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        stat[warp * 8 + 2 * c + e] = ref[e];
        stat[(kWarps + warp) * 8 + 2 * c + e] = sum[e];
      }
    }
    float* mine = reinterpret_cast<float*>(smem) + warp * (8 * D);  // [8][D]
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      extra[j] += __shfl_xor_sync(kAll, extra[j], 1);
      extra[j] += __shfl_xor_sync(kAll, extra[j], 2);
      const float down = up[j] > 0.f ? 1.f / up[j] : 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float ex = __shfl_sync(kAll, extra[j], (2 * c + e) * 4);
        const float ei = __shfl_sync(kAll, eights[e], j * 4 + c) * 0x1p24f;
        float* to = mine + (2 * c + e) * D + j * CH + r * (CH / 8);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          // rows r and r + 8 of the MMA: elements 2t and 2t + 1 of the lane's run
          to[2 * t] = fmaf(o[j][t][e] * 0x1p24f - ei, down, ex);
          to[2 * t + 1] = fmaf(o[j][t][e + 2] * 0x1p20f - ei, down, ex);
        }
      }
    }
    __syncthreads();
    // a warp's weight beside the largest reference; a warp without a token weighs nothing
    if (threadIdx.x < kWarps * 8) {
      const int h = threadIdx.x & 7;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, stat[w * 8 + h]);
      const float m = stat[threadIdx.x], s = stat[kWarps * 8 + threadIdx.x];
      stat[2 * kWarps * 8 + threadIdx.x] =
          m == -INFINITY ? (s == 0.f ? 0.f : qnan()) : ex2(m - M);
      if (threadIdx.x < 8) stat[3 * kWarps * 8 + h] = M;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nh * D; i += kNT) {
      const int h = i / D, d = i % D;
      float total = 0.f, v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = stat[(2 * kWarps + w) * 8 + h];
        total = fmaf(stat[(kWarps + w) * 8 + h], f, total);
        v = fmaf(reinterpret_cast<const float*>(smem)[(w * 8 + h) * D + d], f, v);
      }
      kv4_finish(a, b, h0 + h, part, d, D, direct, L, bad_s, stat[3 * kWarps * 8 + h], total, v);
    }
    if (bad_s && threadIdx.x == 0) set_status(a.status, PA_ERR_BAD_BLOCK_ID);
    __syncthreads();  // the ring, the statistics and q are written again
  }
}

template <typename T, int D, int GS>
cudaError_t launch_d(const Kv4Args& a, int64_t items, cudaStream_t s) {
  using C = Cfg<D, GS>;
  static std::atomic<bool> configured[128];
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const auto kern = pa_kv4_tc_kernel<T, D, GS>;
  // room for the longest list
  constexpr int kMost = C::kOffList + (65536 / kListSpan + 1) * 4;
  if (dev >= 128 || !configured[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
    if (dev < 128) configured[dev].store(true, std::memory_order_release);
  }
  const int64_t room = static_cast<int64_t>(sms) * C::kCtas;
  kern<<<static_cast<unsigned>(items < room ? items : room), kNT,
         C::kOffList + list_bytes(a.num_seqs), s>>>(a);
  return cudaGetLastError();
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
