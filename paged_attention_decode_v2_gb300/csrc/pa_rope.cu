// pa_rope.cu -- pa_qk_norm_rope and pa_qk_norm_rope_axes: norm of each query and
// key head, rotation by position, and the write of keys and values into the paged
// cache.
//
// Row t has R = Hq + 2 Hkv head rows of D elements: queries, keys, values.  D / 8
// lanes hold a head row in registers, each lane four pairs of the rotation:
// elements (j, j + rot / 2) or (2j, 2j + 1), and runs of the tail where
// rotary_dim < D, so a pair never leaves its lane.  The sum of squares is a
// shuffle reduction; y = x * r * w in float32, the rotation, one rounding, one
// store: queries to q_out, keys and values to their slot (and k_out / v_out).
//
// Bound by memory where there are many rows: every element is read and written
// once.  What stands in the way is issuing instructions and waiting: so the
// arithmetic is in pairs of floats (one instruction for two), and a warp takes
// a run of head rows of one kind and one row t (two or four side by side where
// D < 256), everything that does not depend on the head -- the slot's place,
// the angles, the weights -- done once per run, kUnroll rows loaded before the
// first is used.  Measured on the device, bf16: 8192 rows of 24 / 4 heads of 256
// (277 MB) 47.5 us = 5.8 TB/s, 87 % of the copy rate (115 us with one lane per 16
// bytes, pairs in two lanes and the set-up per head row); 32 rows of 32 / 8
// heads of 128 2.5 us, a launch's latency.
//
// With several axes (time, height, width) pair j turns by the angle of its own
// axis' position: a lane's four pairs read their cosines and sines in up to four
// rows of the table, once per run.  Two bits a pair say which axis it has; they
// are kernel parameters, a byte a lane.  It costs nothing that shows: 8192 rows of 24 / 4
// heads of 256 with three axes in turn 47.1 us, 32 rows 3.0 us.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include <cuda_runtime_api.h>

#include "pa_device.cuh"

namespace pa {

namespace {

// A CTA is one warp: its registers are free for the next as soon as it is done,
// and nothing waits for a slower neighbour.  Measured, 8192 rows of 24 / 4 heads of
// 256, bf16: CTAs of 256 threads 54 us, 128 51, 64 49, 32 47.5.
constexpr int kNT = 32;

struct RopeArgs {
  const void* q;
  const void* k;
  const void* v;
  const void* qw;
  const void* kw;
  const float* cos_sin;
  const int32_t* positions;
  const int64_t* slots;
  void* q_out;
  void* k_out;
  void* v_out;
  void* k_cache;
  void* v_cache;
  int32_t* status;
  int64_t q_stride, k_stride, v_stride;
  int64_t pool;  // slots of the pool
  int32_t num_tokens, num_heads, num_kv_heads, block_size, rot, max_position;
  int32_t interleaved, split_x;
  int32_t block_shift;         // log2 of block_size, or -1
  int32_t run;                 // head rows of a run
  int32_t q_runs, kv_runs;     // runs of a row t: queries; keys, and as many values
  int64_t items;
  float eps, weight_offset;
};

// Several axes: a row of positions for each, and the axes of the pairs, two bits
// a pair, four pairs a byte.
struct RopeAxesArgs : RopeArgs {
  int32_t num_axes;
  uint8_t axes[PA_ROPE_MAX_PAIRS / 4];
};

// Two floats in one 64-bit register, for the packed float32 instructions.
using F2 = unsigned long long;
__device__ __forceinline__ F2 pair(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair(F2 v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 swapped(F2 v) {
  float x, y;
  unpair(v, x, y);
  return pair(y, x);
}

// Four elements as they are in memory, and widened.
template <typename T>
struct Raw4 {
  uint2 v;
  __device__ __forceinline__ void load(const T* p) {
    v = __ldcs(reinterpret_cast<const uint2*>(p));
  }
  __device__ __forceinline__ void widen(F2* f) const {
    float x, y;
    widen2(static_cast<const T*>(nullptr), v.x, x, y);
    f[0] = pair(x, y);
    widen2(static_cast<const T*>(nullptr), v.y, x, y);
    f[1] = pair(x, y);
  }
};
template <>
struct Raw4<float> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) {
    v = __ldcs(reinterpret_cast<const float4*>(p));
  }
  __device__ __forceinline__ void widen(F2* f) const {
    f[0] = pair(v.x, v.y);
    f[1] = pair(v.z, v.w);
  }
};

// Round four values to the element type and store them at p.
__device__ __forceinline__ void store4(float* p, const F2* f) {
  float4 v;
  unpair(f[0], v.x, v.y);
  unpair(f[1], v.z, v.w);
  __stcs(reinterpret_cast<float4*>(p), v);
}
__device__ __forceinline__ uint32_t round2(F2 f, __nv_bfloat16*) {
  float x, y;
  unpair(f, x, y);
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t round2(F2 f, __half*) {
  float x, y;
  unpair(f, x, y);
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ void store4(T* p, const F2* f) {
  __stcs(reinterpret_cast<uint2*>(p), make_uint2(round2(f[0], p), round2(f[1], p)));
}

__device__ __forceinline__ float round_elem(float x, float*) { return x; }
__device__ __forceinline__ __nv_bfloat16 round_elem(float x, __nv_bfloat16* p) {
  return round16(x, p);
}
__device__ __forceinline__ __half round_elem(float x, __half* p) { return round16(x, p); }

// What a lane needs to norm and rotate its eight elements of any head row.
// Element pairs y[0..3] hold elements oa .. oa + 3 and ob .. ob + 3; out =
// y * c + other * s with `other` the pairs' other sides: y[2], y[3], y[0], y[1]
// (halves), or each pair swapped (interleaved).  Lanes that do not rotate leave
// y alone: with c = 1 and s = 0 an infinite `other` would make y NaN, and -0
// would become +0.
struct Lane {
  F2 w[4], c[4], s[4];
  bool turns;
};

template <int LPR, bool kInter>
__device__ __forceinline__ void norm_rotate(F2 (&y)[4], const Lane& l, bool norm, float eps,
                                            unsigned mask) {
  constexpr int D = LPR * 8;
  if (norm) {
    F2 q = mul2(y[0], y[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) q = fma2(y[i], y[i], q);
    float x, z;
    unpair(q, x, z);
    float ss = x + z;
#pragma unroll
    for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
    const float rn = rsqrtf(fmaf(ss, 1.f / D, eps));
    const F2 r2 = pair(rn, rn);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = mul2(mul2(y[i], r2), l.w[i]);
  }
  if (!l.turns) return;
  const F2 t[4] = {kInter ? swapped(y[0]) : y[2], kInter ? swapped(y[1]) : y[3],
                   kInter ? swapped(y[2]) : y[0], kInter ? swapped(y[3]) : y[1]};
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = fma2(y[i], l.c[i], mul2(t[i], l.s[i]));
}

// Head rows loaded at once, per side of the warp, and CTAs per SM that the
// register budget is set for (64 registers: two spilled at most for 16-bit
// types, up to 40 for float32).  Measured on the same rows with CTAs of 64
// threads: 4 rows and 16 CTAs 48.6 us, 4 and 12 51.2 us, 2 and 20 50.7 us, 6
// and 12 53.3 us.
constexpr int kUnroll = 4;
constexpr int kCtas = 32;

template <typename T, int D, bool kInter, typename Args>
__global__ void __launch_bounds__(kNT, kCtas) pa_rope_kernel(const Args a) {
  constexpr bool kAxes = std::is_same<Args, RopeAxesArgs>::value;
  constexpr int X = 16 / sizeof(T);                   // elements of a split-x key group
  constexpr int LPR = D / 8;                          // lanes of a head row
  constexpr int kSide = 32 / LPR;                     // head rows side by side in a warp
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x % LPR, side = threadIdx.x % 32 / LPR;
  const uint32_t item = blockIdx.x * (kNT / 32) + threadIdx.x / 32;
  if (item >= a.items) return;
  const uint32_t per_row = a.q_runs + 2 * a.kv_runs;
  const int32_t t = static_cast<int32_t>(item / per_row);
  // the runs of a row t in an order that turns with t, or, where 152 is a multiple
  // of per_row, some SMs would get all the runs of one kind (1001 rows, split-x
  // values: 10.0 us, so 6.6)
  const int k = static_cast<int>((item - t * per_row + t) % per_row);
  const int64_t slot = __ldg(a.slots + t);
  const int32_t pos = a.rot ? __ldg(a.positions + t) : 0;
  int32_t other[3] = {0, 0, 0};                       // the positions on further axes
  if constexpr (kAxes) {
#pragma unroll
    for (int x = 0; x < 3; ++x)
      if (a.rot && x + 1 < a.num_axes)
        other[x] = __ldg(a.positions + static_cast<int64_t>(x + 1) * a.num_tokens + t);
  }
  const int kind = k < a.q_runs ? 0 : k < a.q_runs + a.kv_runs ? 1 : 2;
  const int h0 = (kind == 0 ? k : kind == 1 ? k - a.q_runs : k - a.q_runs - a.kv_runs) * a.run;
  const int heads = kind == 0 ? a.num_heads : a.num_kv_heads;
  const int h1 = min(h0 + a.run, heads);
  // this lane's two runs of four elements
  const int half = a.rot / 2, j0 = lane * 4;
  const bool rotates = j0 < half;                     // half is a multiple of 8
  const int oa = kInter ? lane * 8 : rotates ? j0 : half + j0;
  const int ob = kInter ? lane * 8 + 4 : rotates ? j0 + half : D / 2 + j0;

  const T* src = (kind == 0   ? static_cast<const T*>(a.q) + t * a.q_stride
                  : kind == 1 ? static_cast<const T*>(a.k) + t * a.k_stride
                              : static_cast<const T*>(a.v) + t * a.v_stride) +
                 (h0 + side) * D;
  Raw4<T> raw[kUnroll][2];
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (h + side + u * kSide < h1) {
        raw[u][0].load(src + u * kSide * D + oa);
        raw[u][1].load(src + u * kSide * D + ob);
      }
    src += kUnroll * kSide * D;
  };
  load(h0);
  if (slot == -1) return;                             // padding
  bool pos_ok = !a.rot || (pos >= 0 && pos < a.max_position);
  if constexpr (kAxes) {
#pragma unroll
    for (int x = 0; x < 3; ++x)
      pos_ok = pos_ok && (!a.rot || (other[x] >= 0 && other[x] < a.max_position));
  }
  const bool slot_ok = !a.k_cache || (slot >= 0 && slot < a.pool);
  if (k == 0 && threadIdx.x % 32 == 0) {
    if (!slot_ok) set_status(a.status, PA_ERR_BAD_SLOT);
    if (!pos_ok) set_status(a.status, PA_ERR_BAD_POSITION);
  }
  Lane l;
  const bool norm = a.qw != nullptr;
  if (kind < 2) {
    float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (kAxes && rotates && pos_ok) {
      if constexpr (kAxes) {
        // pairs j0 .. j0 + 3, each on its axis' row
        const unsigned of = a.axes[lane];
        const float* at[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const unsigned x = of >> (2 * i) & 3;
          const int32_t p = x == 0 ? pos : x == 1 ? other[0] : x == 2 ? other[1] : other[2];
          at[i] = a.cos_sin + static_cast<int64_t>(p) * a.rot + j0 + i;
        }
        c = make_float4(__ldg(at[0]), __ldg(at[1]), __ldg(at[2]), __ldg(at[3]));
        s = make_float4(__ldg(at[0] + half), __ldg(at[1] + half), __ldg(at[2] + half),
                        __ldg(at[3] + half));
      }
    } else if (rotates && pos_ok) {
      const float* row = a.cos_sin + static_cast<int64_t>(pos) * a.rot + j0;
      c = __ldg(reinterpret_cast<const float4*>(row));
      s = __ldg(reinterpret_cast<const float4*>(row + half));
    }
    if (!pos_ok) c.x = c.y = c.z = c.w = qnan();      // the rows come out NaN
    l.turns = rotates || !pos_ok;
    if (kInter) {
      l.c[0] = pair(c.x, c.x), l.c[1] = pair(c.y, c.y);
      l.c[2] = pair(c.z, c.z), l.c[3] = pair(c.w, c.w);
      l.s[0] = pair(-s.x, s.x), l.s[1] = pair(-s.y, s.y);
      l.s[2] = pair(-s.z, s.z), l.s[3] = pair(-s.w, s.w);
    } else {
      l.c[0] = l.c[2] = pair(c.x, c.y);
      l.c[1] = l.c[3] = pair(c.z, c.w);
      l.s[0] = pair(-s.x, -s.y), l.s[1] = pair(-s.z, -s.w);
      l.s[2] = pair(s.x, s.y), l.s[3] = pair(s.z, s.w);
    }
    if (norm) {
      const T* w = static_cast<const T*>(kind == 0 ? a.qw : a.kw);
      float f[8];
      load_row<T, 4>(w + oa, *reinterpret_cast<float(*)[4]>(&f[0]));
      load_row<T, 4>(w + ob, *reinterpret_cast<float(*)[4]>(&f[4]));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        l.w[i] = pair(f[2 * i] + a.weight_offset, f[2 * i + 1] + a.weight_offset);
    }
  }
  // where the rows go: q_out, or dense and the slot's place in the pool
  const bool cache = kind > 0 && a.k_cache && slot_ok && pos_ok;
  T* dense = static_cast<T*>(kind == 0 ? a.q_out : kind == 1 ? a.k_out : a.v_out);
  if (dense) dense += static_cast<int64_t>(t) * heads * D;
  T* pool = nullptr;
  const int64_t head = static_cast<int64_t>(a.block_size) * D;  // a head's part of a block
  int64_t pa = 0, pb = 0;
  if (cache) {
    const int64_t block = a.block_shift >= 0 ? slot >> a.block_shift : slot / a.block_size;
    const int at = static_cast<int>(slot - block * a.block_size);
    pool = static_cast<T*>(kind == 1 ? a.k_cache : a.v_cache) + block * heads * head;
    if (!a.split_x) {
      pa = static_cast<int64_t>(at) * D + oa;
      pb = static_cast<int64_t>(at) * D + ob;
    } else if (kind == 1) {  // 16-byte groups [D / X][block_size][X]
      pa = (static_cast<int64_t>(oa / X) * a.block_size + at) * X + oa % X;
      pb = (static_cast<int64_t>(ob / X) * a.block_size + at) * X + ob % X;
    } else {                 // [D][block_size]
      pa = static_cast<int64_t>(oa) * a.block_size + at;
      pb = static_cast<int64_t>(ob) * a.block_size + at;
    }
  }
  for (int h = h0;;) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int x = h + side + u * kSide;
      if (h + u * kSide >= h1) break;
      F2 y[4];
      raw[u][0].widen(&y[0]);
      raw[u][1].widen(&y[2]);
      if (kind < 2) norm_rotate<LPR, kInter>(y, l, norm, a.eps, kAll);
      if (x >= h1) continue;
      if (dense) {
        store4(dense + x * D + oa, y);
        store4(dense + x * D + ob, y + 2);
      }
      if (!cache) continue;
      if (!a.split_x || kind == 1) {
        store4(pool + x * head + pa, y);
        store4(pool + x * head + pb, y + 2);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float f[2];
          unpair(y[e / 2], f[0], f[1]);
          pool[x * head + (e < 4 ? pa : pb) + static_cast<int64_t>(e % 4) * a.block_size] =
              round_elem(f[e % 2], static_cast<T*>(nullptr));
        }
      }
    }
    h += kUnroll * kSide;
    if (h >= h1) break;
    load(h);
  }
}

template <typename T, int D, bool kInter, typename Args>
cudaError_t launch_i(Args a, int sms, cudaStream_t s) {
  constexpr int kWarps = kNT / 32;
  constexpr int kSide = 32 / (D / 8);
  // two loads' worth of head rows a run, fewer while the runs do not fill the
  // GPU twice (16 warps an SM)
  a.run = 2 * kUnroll * kSide;
  while (a.run > kSide &&
         static_cast<int64_t>(a.num_tokens) * (a.num_heads + 2 * a.num_kv_heads) / a.run <
             static_cast<int64_t>(sms > 0 ? sms : 152) * 16)
    a.run = a.run / 2 > kSide ? a.run / 2 : kSide;
  a.q_runs = (a.num_heads + a.run - 1) / a.run;
  a.kv_runs = (a.num_kv_heads + a.run - 1) / a.run;
  a.items = static_cast<int64_t>(a.num_tokens) * (a.q_runs + 2 * a.kv_runs);
  if (a.items + kWarps >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  pa_rope_kernel<T, D, kInter, Args>
      <<<static_cast<unsigned>((a.items + kWarps - 1) / kWarps), kNT, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int D, typename Args>
cudaError_t launch_d(const Args& a, int sms, cudaStream_t s) {
  return a.interleaved ? launch_i<T, D, true>(a, sms, s) : launch_i<T, D, false>(a, sms, s);
}

template <typename T, typename Args>
cudaError_t launch_t(const Args& a, int D, int sms, cudaStream_t s) {
  switch (D) {
    case 64: return launch_d<T, 64>(a, sms, s);
    case 128: return launch_d<T, 128>(a, sms, s);
    default: return launch_d<T, 256>(a, sms, s);
  }
}

template <typename Args>
cudaError_t launch(const Args& a, pa_dtype_t dtype, int D, int sms, cudaStream_t s) {
  switch (dtype) {
    case PA_F32: return launch_t<float>(a, D, sms, s);
    case PA_BF16: return launch_t<__nv_bfloat16>(a, D, sms, s);
    default: return launch_t<__half>(a, D, sms, s);
  }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// Both calls; `axes` null: one position a row.
pa_status_t norm_rope(const pa_rope_params_t* p, const pa_rope_axes_t* axes, const void* q,
                      const void* k, const void* v, const void* q_weight, const void* k_weight,
                      const float* cos_sin, const int32_t* positions, const int64_t* slots,
                      void* q_out, void* k_out, void* v_out, void* k_cache, void* v_cache,
                      int32_t* status, cudaStream_t stream) {
  if (!p || p->num_tokens < 0 || p->num_heads < 1 || p->num_kv_heads < 1) return PA_ERR_INVALID_ARG;
  if (p->block_size < 1 || p->num_blocks < 1) return PA_ERR_INVALID_ARG;
  if (p->flags & ~(PA_ROPE_INTERLEAVED | PA_FLAG_SPLIT_X)) return PA_ERR_INVALID_ARG;
  if (p->dtype != PA_F32 && p->dtype != PA_BF16 && p->dtype != PA_F16) return PA_ERR_UNSUPPORTED;
  if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (p->rotary_dim < 0 || p->rotary_dim > p->head_dim || p->rotary_dim % 16)
    return PA_ERR_INVALID_ARG;
  if (p->rotary_dim && p->max_position < 1) return PA_ERR_INVALID_ARG;
  if (axes) {
    if (axes->num_axes < 1 || axes->num_axes > PA_ROPE_MAX_AXES) return PA_ERR_INVALID_ARG;
    for (int j = 0; j < p->rotary_dim / 2; ++j)
      if (axes->axis_of[j] >= axes->num_axes) return PA_ERR_INVALID_ARG;
  }
  if (p->num_heads > 65535 || p->num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
  if (!(p->eps >= 0.f)) return PA_ERR_INVALID_ARG;
  const int64_t D = p->head_dim, esz = p->dtype == PA_F32 ? 4 : 2;
  if (p->num_tokens > 1 &&
      (p->q_stride < p->num_heads * D || p->k_stride < p->num_kv_heads * D ||
       p->v_stride < p->num_kv_heads * D))
    return PA_ERR_INVALID_ARG;
  if (p->num_tokens == 0) return PA_OK;
  if (!q || !k || !v || !slots || !q_out) return PA_ERR_INVALID_ARG;
  if (p->rotary_dim && (!cos_sin || !positions)) return PA_ERR_INVALID_ARG;
  if (!q_weight != !k_weight || !k_cache != !v_cache) return PA_ERR_INVALID_ARG;
  if (p->num_tokens > 1 &&
      ((p->q_stride * esz) % 16 || (p->k_stride * esz) % 16 || (p->v_stride * esz) % 16))
    return PA_ERR_MISALIGNED;
  for (const void* x : {q, k, v, q_weight, k_weight, static_cast<const void*>(cos_sin),
                        static_cast<const void*>(q_out), static_cast<const void*>(k_out),
                        static_cast<const void*>(v_out), static_cast<const void*>(k_cache),
                        static_cast<const void*>(v_cache)})
    if (!aligned(x, 16)) return PA_ERR_MISALIGNED;
  if (!aligned(positions, 4) || !aligned(slots, 8) || !aligned(status, 4))
    return PA_ERR_MISALIGNED;
  {
    // No output over an input or over another output: other CTAs may still read
    // the one, or write the other.  q, k and v may be replaced in place where the
    // rows coincide: a lane stores the elements that it has loaded.
    const int64_t T = p->num_tokens, nq = p->num_heads * D, nk = p->num_kv_heads * D;
    const double most = 4e18;  // past any address space: sizes of wild parameters end here
    const auto size = [&](double elements) {
      return static_cast<size_t>(std::min(elements * esz, most));
    };
    const auto rows = [&](int64_t stride, int64_t n) {
      return size(static_cast<double>(T - 1) * stride + n);
    };
    const auto in = [&](const void* x, int64_t stride, int64_t n, const void* out) {
      const bool replaced = x == out && (T == 1 || stride == n);
      return Range{replaced ? nullptr : x, rows(T > 1 ? stride : n, n), false};
    };
    const size_t pool = size(static_cast<double>(p->num_blocks) * p->block_size * nk);
    const size_t D1 = static_cast<size_t>(D * esz);
    const Range r[] = {
        in(q, p->q_stride, nq, q_out),
        in(k, p->k_stride, nk, k_out),
        in(v, p->v_stride, nk, v_out),
        {q_weight, D1, false},
        {k_weight, D1, false},
        {p->rotary_dim ? cos_sin : nullptr,
         static_cast<size_t>(p->max_position) * p->rotary_dim * 4, false},
        {p->rotary_dim ? positions : nullptr, static_cast<size_t>(T) * 4 * (axes ? axes->num_axes : 1),
         false},
        {slots, static_cast<size_t>(T) * 8, false},
        {q_out, rows(nq, nq), true},
        {k_out, rows(nk, nk), true},
        {v_out, rows(nk, nk), true},
        {k_cache, pool, true},
        {v_cache, pool, true},
        {status, 4, true}};
    if (outputs_overlap(r, sizeof r / sizeof r[0])) return PA_ERR_INVALID_ARG;
  }
  RopeArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.qw = q_weight;
  a.kw = k_weight;
  a.cos_sin = cos_sin;
  a.positions = positions;
  a.slots = slots;
  a.q_out = q_out;
  a.k_out = k_out;
  a.v_out = v_out;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.status = status;
  a.q_stride = p->q_stride;
  a.k_stride = p->k_stride;
  a.v_stride = p->v_stride;
  a.pool = static_cast<int64_t>(p->num_blocks) * p->block_size;
  a.num_tokens = p->num_tokens;
  a.num_heads = p->num_heads;
  a.num_kv_heads = p->num_kv_heads;
  a.block_size = p->block_size;
  a.block_shift = (p->block_size & (p->block_size - 1)) ? -1 : __builtin_ctz(p->block_size);
  a.rot = p->rotary_dim;
  a.max_position = p->max_position;
  a.interleaved = (p->flags & PA_ROPE_INTERLEAVED) ? 1 : 0;
  a.split_x = (p->flags & PA_FLAG_SPLIT_X) ? 1 : 0;
  a.eps = p->eps;
  a.weight_offset = p->weight_offset;
  const int sms = sm100_num_sms();
  cudaError_t e;
  if (axes) {
    RopeAxesArgs x{};
    static_cast<RopeArgs&>(x) = a;
    x.num_axes = axes->num_axes;
    for (int i = 0; i < p->rotary_dim / 2; ++i)
      x.axes[i / 4] = static_cast<uint8_t>(x.axes[i / 4] | axes->axis_of[i] << (2 * (i % 4)));
    e = launch(x, p->dtype, p->head_dim, sms, stream);
  } else {
    e = launch(a, p->dtype, p->head_dim, sms, stream);
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace
}  // namespace pa

extern "C" {

pa_status_t pa_qk_norm_rope(const pa_rope_params_t* p, const void* q, const void* k,
                            const void* v, const void* q_weight, const void* k_weight,
                            const float* cos_sin, const int32_t* positions, const int64_t* slots,
                            void* q_out, void* k_out, void* v_out, void* k_cache, void* v_cache,
                            int32_t* status, cudaStream_t stream) {
  return pa::norm_rope(p, nullptr, q, k, v, q_weight, k_weight, cos_sin, positions, slots, q_out,
                       k_out, v_out, k_cache, v_cache, status, stream);
}

pa_status_t pa_qk_norm_rope_axes(const pa_rope_params_t* p, const pa_rope_axes_t* axes,
                                 const void* q, const void* k, const void* v,
                                 const void* q_weight, const void* k_weight, const float* cos_sin,
                                 const int32_t* positions, const int64_t* slots, void* q_out,
                                 void* k_out, void* v_out, void* k_cache, void* v_cache,
                                 int32_t* status, cudaStream_t stream) {
  if (!axes) return PA_ERR_INVALID_ARG;
  return pa::norm_rope(p, axes, q, k, v, q_weight, k_weight, cos_sin, positions, slots, q_out,
                       k_out, v_out, k_cache, v_cache, status, stream);
}

}  // extern "C"
