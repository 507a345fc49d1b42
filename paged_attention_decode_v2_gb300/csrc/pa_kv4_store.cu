// pa_kv4_store.cu -- pa_store_kv4: keys and values into the 4-bit paged cache.
//
// For each group of a head row: m = min x, s = (max x - m) / 15 rounded to the
// element type, c = min(15, round((x - m) / s)), to even where it is halfway (0
// where s is 0).  x - m is float32, rounded once (exact for 16-bit rows of ordinary
// spread); the code is that of its exact quotient by s, below s = 2^-100 of the quotient
// rounded to float32.  m is an x, so the scale is all that is rounded to fewer bits, before
// the codes are made with it.  A group with a value that is not finite, or whose range is not, gets
// NaN for both and reads back as NaN.
//
// D / 16 lanes hold a head row, sixteen elements each; a group's extremes are a
// shuffle reduction over group / 16 of them.  One pass: 32 bytes a lane are read, 8
// bytes of codes written, and with k_out and v_out the values that the codes stand
// for.  Bound by instructions as much as by memory: some 200 a row of 256.  Measured on
// the device, bf16: 8192 rows of 4 heads of 256 with k_out and v_out (77 MB) 16.1 us = 4.8
// TB/s (36 us with a division per element and eight elements a lane); 32 rows 2.3 us, a
// launch.  Halves of a row as a lane's two eights, for stores of whole sectors, cost more
// than they gave (18.1 us).
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include <cuda_runtime_api.h>

#include "pa_kv4.cuh"

namespace pa {

namespace {

constexpr int kNT = 128;

struct StoreArgs {
  const void* k;
  const void* v;
  const int64_t* slots;
  uint8_t* k_codes;
  uint8_t* v_codes;
  void* k_pairs;
  void* v_pairs;
  void* k_out;        // may be null, and
  void* v_out;
  int32_t* status;
  int64_t k_stride, v_stride;
  int64_t pool;       // slots of the pool
  uint32_t rows;      // head rows of the call: keys and values
  int32_t num_kv_heads, block_size;
  int32_t span_shift;               // log2 of the lanes of a group, group_size / 16
  int32_t head_shift, block_shift;  // log2, or -1
};

// Minimum and maximum that are NaN where an operand is.
__device__ __forceinline__ float min_nan(float x, float y) {
  float z;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}
__device__ __forceinline__ float max_nan(float x, float y) {
  float z;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}
__device__ __forceinline__ uint32_t min2(uint32_t x, uint32_t y, const __nv_bfloat16*) {
  const __nv_bfloat162 z = __hmin2_nan(*reinterpret_cast<__nv_bfloat162*>(&x),
                                       *reinterpret_cast<__nv_bfloat162*>(&y));
  return *reinterpret_cast<const uint32_t*>(&z);
}
__device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y, const __nv_bfloat16*) {
  const __nv_bfloat162 z = __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&x),
                                       *reinterpret_cast<__nv_bfloat162*>(&y));
  return *reinterpret_cast<const uint32_t*>(&z);
}
__device__ __forceinline__ uint32_t min2(uint32_t x, uint32_t y, const __half*) {
  const __half2 z = __hmin2_nan(*reinterpret_cast<__half2*>(&x), *reinterpret_cast<__half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&z);
}
__device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y, const __half*) {
  const __half2 z = __hmax2_nan(*reinterpret_cast<__half2*>(&x), *reinterpret_cast<__half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&z);
}

// Eight elements as they are in memory, widened, and their extremes.
template <typename T>
struct Raw8 {
  uint4 v;
  __device__ __forceinline__ void load(const T* p) {
    v = __ldcs(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void widen(float (&f)[8]) const {
    const T* t = nullptr;
    widen2(t, v.x, f[0], f[1]);
    widen2(t, v.y, f[2], f[3]);
    widen2(t, v.z, f[4], f[5]);
    widen2(t, v.w, f[6], f[7]);
  }
  __device__ __forceinline__ void extremes(float& lo, float& hi) const {
    const T* t = nullptr;
    float x, y;
    widen2(t, min2(min2(v.x, v.y, t), min2(v.z, v.w, t), t), x, y);
    lo = min_nan(x, y);
    widen2(t, max2(max2(v.x, v.y, t), max2(v.z, v.w, t), t), x, y);
    hi = max_nan(x, y);
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void widen(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  __device__ __forceinline__ void extremes(float& lo, float& hi) const {
    lo = min_nan(min_nan(min_nan(a.x, a.y), min_nan(a.z, a.w)),
                 min_nan(min_nan(b.x, b.y), min_nan(b.z, b.w)));
    hi = max_nan(max_nan(max_nan(a.x, a.y), max_nan(a.z, a.w)),
                 max_nan(max_nan(b.x, b.y), max_nan(b.z, b.w)));
  }
};

// range / 15, rounded to nearest: the quotient's remainder corrects the product with
// 1 / 15.  (What float32 keeps less than whole, below 2^-100, takes the division.)
__device__ __forceinline__ float fifteenth(float range) {
  if (range < 0x1p-100f) return __fdiv_rn(range, 15.f);
  const float q = range * (1.f / 15);
  return fmaf(fmaf(-15.f, q, range), 1.f / 15, q);
}

// A code by the division.
__device__ __noinline__ float divided(float d, float s) {
  return s > 0.f ? fminf(rintf(__fdiv_rn(d, s)), 15.f) : 0.f;
}

// c = min(15, round(d / s)) of the eight d = x - lo, and the codes packed.  By the approximate
// reciprocal the quotients are off by less than 2^-18 (15 times 2^-23, the reciprocal's and the
// product's error), so a rounded one may differ only within that of a half; there d - c s, which
// is exact, says on which side of the half d is.  (Rows of 16 bits come to a half often: some 1
// in 500 elements.)  Scales that are subnormal or nearly so take the division.
__device__ __forceinline__ uint32_t make_codes(const float (&x)[8], float lo, float s,
                                               F2 (&c)[4]) {
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  if (!(s > 0.f)) inv = 0.f;  // no range: 0; NaN: the codes do not matter
  constexpr float kMagic = 0x1.8p23f;  // adding it rounds to a whole number, to even
  const F2 low = pair(-lo, -lo), by = pair(inv, inv), up = pair(kMagic, kMagic),
           down = pair(-kMagic, -kMagic), minus = pair(-1.f, -1.f);
  float far = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 q = unpair(mul2(add2(pair(x[2 * e], x[2 * e + 1]), low), by));
    const F2 y = pair(fminf(q.x, 15.f), fminf(q.y, 15.f));
    c[e] = add2(add2(y, up), down);
    const float2 r = unpair(fma2(c[e], minus, y));
    far = fmaxf(far, fmaxf(fabsf(r.x), fabsf(r.y)));
  }
  if (far > 0.5f - 0x1p-17f) {
    const float half = 0.5f * s;
    const auto settle = [&](float d, float k) {
      const float r = fmaf(-k, s, d), other = k + copysignf(1.f, r);
      const bool odd = (static_cast<int>(k) & 1) != 0;
      return fabsf(r) > half || (fabsf(r) == half && odd) ? fminf(other, 15.f) : k;
    };
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 k = unpair(c[e]);
      c[e] = pair(settle(x[2 * e] - lo, k.x), settle(x[2 * e + 1] - lo, k.y));
    }
  }
  if (s < 0x1p-100f) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c[e] = pair(divided(x[2 * e] - lo, s), divided(x[2 * e + 1] - lo, s));
  }
  // four codes are 16 bits of a float's whole number
  const float2 c0 = unpair(c[0]), c1 = unpair(c[1]), c2 = unpair(c[2]), c3 = unpair(c[3]);
  const float a = fmaf(16.f, fmaf(16.f, fmaf(16.f, c1.y, c1.x), c0.y), c0.x) + 0x1p23f;
  const float b = fmaf(16.f, fmaf(16.f, fmaf(16.f, c3.y, c3.x), c2.y), c2.x) + 0x1p23f;
  return s >= 0.f ? __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x5410) : 0u;
}

template <typename T>
__device__ __forceinline__ float rounded(float x) {
  if constexpr (std::is_same<T, float>::value) return x;
  else return to_float(round16(x, static_cast<T*>(nullptr)));
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  return bits16(round16(x, static_cast<T*>(nullptr))) |
         static_cast<uint32_t>(bits16(round16(y, static_cast<T*>(nullptr)))) << 16;
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
  if constexpr (std::is_same<T, float>::value) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
  } else {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]),
                                                   pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7])));
  }
}

// kRows: head rows that a lane has in flight.
template <typename T, int D, int kRows>
__global__ void __launch_bounds__(kNT) pa_store_kv4_kernel(const StoreArgs a) {
  constexpr int LPR = D / 16;       // lanes of a head row
  constexpr int kSide = 32 / LPR;   // head rows side by side in a warp
  const int lane = threadIdx.x % LPR, side = threadIdx.x % 32 / LPR;
  const uint32_t warp = blockIdx.x * (kNT / 32) + threadIdx.x / 32;
  const uint32_t r0 = warp * (kRows * kSide) + side;
  const uint32_t H = a.num_kv_heads;
  const int span = 1 << a.span_shift;  // lanes of a group

  Raw8<T> raw[kRows][2];
  int64_t slot[kRows];
  uint32_t t[kRows], head[kRows];
  int kind[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const uint32_t r = r0 + u * kSide;
    slot[u] = -1;
    if (r >= a.rows) continue;
    const uint32_t x = a.head_shift >= 0 ? r >> a.head_shift : r / H;  // 2 t + kind
    t[u] = x / 2;
    kind[u] = x & 1;
    head[u] = r - x * H;
    slot[u] = __ldg(a.slots + t[u]);
    const T* src = (kind[u] ? static_cast<const T*>(a.v) + t[u] * a.v_stride
                            : static_cast<const T*>(a.k) + t[u] * a.k_stride) +
                   head[u] * D + lane * 16;
    raw[u][0].load(src);
    raw[u][1].load(src + 8);
  }
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    // every lane of the warp takes part in the reductions
    float lo, hi, x, y;
    raw[u][0].extremes(lo, hi);
    raw[u][1].extremes(x, y);
    lo = min_nan(lo, x);
    hi = max_nan(hi, y);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      if (o >= span) break;
      lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    if (slot[u] == -1) continue;    // padding, or no such row
    float range = hi - lo;
    if (!isfinite(range)) lo = range = qnan();
    const float s = rounded<T>(std::is_same<T, float>::value ? __fdiv_rn(range, 15.f)
                                                             : fifteenth(range));
    T* out = static_cast<T*>(kind[u] ? a.v_out : a.k_out);
    if (out) out += (static_cast<uint64_t>(t[u]) * H + head[u]) * D + lane * 16;
    uint2 codes;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float f[8];
      F2 c[4];
      raw[u][h].widen(f);
      (h ? codes.y : codes.x) = make_codes(f, lo, s, c);
      if (out) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 v = unpair(fma2(c[e], pair(s, s), pair(lo, lo)));
          f[2 * e] = v.x;
          f[2 * e + 1] = v.y;
        }
        store8(out + 8 * h, f);
      }
    }
    if (slot[u] < 0 || slot[u] >= a.pool) {
      if (lane == 0) set_status(a.status, PA_ERR_BAD_SLOT);
      continue;
    }
    // block ids and rows of a page are 31 bits
    const uint32_t block = static_cast<uint32_t>(
        a.block_shift >= 0 ? slot[u] >> a.block_shift : slot[u] / a.block_size);
    const uint32_t at = static_cast<uint32_t>(slot[u]) - block * a.block_size;
    const uint64_t row = static_cast<uint64_t>(block) * (H * a.block_size) +
                         (head[u] * a.block_size + at);
    *reinterpret_cast<uint2*>((kind[u] ? a.v_codes : a.k_codes) + row * (D / 2) + lane * 8) =
        codes;
    if ((lane & (span - 1)) == 0) {
      const uint64_t i = row * (LPR >> a.span_shift) + (lane >> a.span_shift);
      void* pairs = kind[u] ? a.v_pairs : a.k_pairs;
      if constexpr (std::is_same<T, float>::value)
        static_cast<float2*>(pairs)[i] = make_float2(s, lo);
      else
        static_cast<uint32_t*>(pairs)[i] = pack2<T>(s, lo);
    }
  }
}

template <typename T, int D, int kRows>
cudaError_t launch_r(const StoreArgs& a, cudaStream_t s) {
  constexpr uint32_t kPer = kNT / 32 * kRows * (32 / (D / 16));
  pa_store_kv4_kernel<T, D, kRows><<<(a.rows + kPer - 1) / kPer, kNT, 0, s>>>(a);
  return cudaGetLastError();
}

// Rows in flight for each lane: two, or one while two leave the GPU's SMs without some warps
// each.
template <typename T, int D>
cudaError_t launch_d(const StoreArgs& a, cudaStream_t s) {
  return a.rows / (32 / (D / 16)) < 152 * 32 ? launch_r<T, D, 1>(a, s) : launch_r<T, D, 2>(a, s);
}

template <typename T>
cudaError_t launch(const StoreArgs& a, int D, cudaStream_t s) {
  switch (D) {
    case 64: return launch_d<T, 64>(a, s);
    case 128: return launch_d<T, 128>(a, s);
    default: return launch_d<T, 256>(a, s);
  }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

}  // namespace
}  // namespace pa

extern "C" pa_status_t pa_store_kv4(const pa_store_kv4_params_t* p, const void* k, const void* v,
                                    const int64_t* slots, void* k_codes, void* v_codes,
                                    void* k_scales, void* v_scales, void* k_out, void* v_out,
                                    int32_t* status, cudaStream_t stream) {
  using namespace pa;
  if (!p || p->num_tokens < 0 || p->num_kv_heads < 1) return PA_ERR_INVALID_ARG;
  if (p->block_size < 1 || p->num_blocks < 1) return PA_ERR_INVALID_ARG;
  if (pa_status_t st = check_kv4(p->dtype, p->head_dim, p->group_size)) return st;
  if (p->num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(p->num_kv_heads) * p->block_size >= (int64_t(1) << 31))
    return PA_ERR_UNSUPPORTED;
  // head rows, and those of a CTA past the last, are counted in 31 bits
  if (static_cast<int64_t>(p->num_tokens) * p->num_kv_heads * 2 + 1024 >= (int64_t(1) << 31))
    return PA_ERR_UNSUPPORTED;
  const int64_t D = p->head_dim, T = p->num_tokens, n = p->num_kv_heads * D;
  const int64_t esz = p->dtype == PA_F32 ? 4 : 2;
  if (T > 1 && (p->k_stride < n || p->v_stride < n)) return PA_ERR_INVALID_ARG;
  if (T == 0) return PA_OK;
  if (!k || !v || !slots || !k_codes || !v_codes || !k_scales || !v_scales)
    return PA_ERR_INVALID_ARG;
  if (T > 1 && ((p->k_stride * esz) % 16 || (p->v_stride * esz) % 16)) return PA_ERR_MISALIGNED;
  for (const void* x : {k, v, static_cast<const void*>(k_codes), static_cast<const void*>(v_codes),
                        static_cast<const void*>(k_scales), static_cast<const void*>(v_scales),
                        static_cast<const void*>(k_out), static_cast<const void*>(v_out)})
    if (!aligned(x, 16)) return PA_ERR_MISALIGNED;
  if (!aligned(slots, 8) || !aligned(status, 4)) return PA_ERR_MISALIGNED;
  {
    // No output over an input or another output; k and v may be replaced in place
    // where the rows coincide: a lane stores the elements that it has loaded.
    const double most = 4e18;  // past any address space: sizes of wild parameters end here
    const auto size = [&](double bytes) { return static_cast<size_t>(std::min(bytes, most)); };
    const auto in = [&](const void* x, int64_t stride, const void* out) {
      const bool replaced = x == out && (T == 1 || stride == n);
      return Range{replaced ? nullptr : x,
                   size((static_cast<double>(T - 1) * (T > 1 ? stride : 0) + n) * esz), false};
    };
    const double rows = static_cast<double>(p->num_blocks) * p->block_size * p->num_kv_heads;
    const size_t codes = size(rows * (D / 2)), pairs = size(rows * (D / p->group_size) * 2 * esz);
    const size_t dense = size(static_cast<double>(T) * n * esz);
    const Range r[] = {in(k, p->k_stride, k_out), in(v, p->v_stride, v_out),
                       {slots, static_cast<size_t>(T) * 8, false},
                       {k_codes, codes, true}, {v_codes, codes, true},
                       {k_scales, pairs, true}, {v_scales, pairs, true},
                       {k_out, dense, true}, {v_out, dense, true}, {status, 4, true}};
    if (outputs_overlap(r, sizeof r / sizeof r[0])) return PA_ERR_INVALID_ARG;
  }
  StoreArgs a{};
  a.k = k;
  a.v = v;
  a.slots = slots;
  a.k_codes = static_cast<uint8_t*>(k_codes);
  a.v_codes = static_cast<uint8_t*>(v_codes);
  a.k_pairs = k_scales;
  a.v_pairs = v_scales;
  a.k_out = k_out;
  a.v_out = v_out;
  a.status = status;
  a.k_stride = p->k_stride;
  a.v_stride = p->v_stride;
  a.pool = static_cast<int64_t>(p->num_blocks) * p->block_size;
  a.rows = static_cast<uint32_t>(T * p->num_kv_heads * 2);
  a.num_kv_heads = p->num_kv_heads;
  a.block_size = p->block_size;
  const auto shift = [](int n) { return (n & (n - 1)) ? -1 : __builtin_ctz(n); };
  a.block_shift = shift(p->block_size);
  a.head_shift = shift(p->num_kv_heads);
  a.span_shift = shift(p->group_size / 16);
  cudaError_t e;
  switch (p->dtype) {
    case PA_F32: e = launch<float>(a, p->head_dim, stream); break;
    case PA_BF16: e = launch<__nv_bfloat16>(a, p->head_dim, stream); break;
    default: e = launch<__half>(a, p->head_dim, stream); break;
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
