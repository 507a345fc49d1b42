// pa_kv4_store.cu -- pa_store_kv4: keys and values into the 4-bit paged cache.
//
// For each group of a head row: m = min x, s = (max x - m) / 15 rounded to the
// element type, c = min(15, round((x - m) / s)), to even where it is halfway (0
// where s is 0).  x - m and the quotients are float32, each rounded once; m is an
// x, so the scale is all that is rounded to fewer bits, before the codes are made
// with it.  A group with a value that is not finite, or whose range is not, gets
// NaN for both and reads back as NaN.
//
// D / 8 lanes hold a head row, eight elements each; a group's extremes are a
// shuffle reduction over group / 8 of them.  One pass: 16 bytes a lane are read,
// 4 bytes of codes written, and with k_out and v_out the values that the codes
// stand for.
#include <algorithm>
#include <cstdint>

#include <cuda_runtime_api.h>

#include "pa_kv4.cuh"

namespace pa {

namespace {

constexpr int kNT = 128;

struct StoreArgs {
  const void* k;
  const void* v;
  const int64_t* slots;
  uint8_t* codes[2];  // k, v
  void* pairs[2];
  void* out[2];       // may be null
  int32_t* status;
  int64_t k_stride, v_stride;
  int64_t pool;       // slots of the pool
  int64_t rows;       // head rows of the call: keys and values
  int32_t num_kv_heads, block_size, block_shift, group;
};

// Eight elements as they are in memory, and widened.
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
};

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
  constexpr int LPR = D / 8;        // lanes of a head row
  constexpr int kSide = 32 / LPR;   // head rows side by side in a warp
  const int lane = threadIdx.x % LPR, side = threadIdx.x % 32 / LPR;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kNT + threadIdx.x) / 32;
  const int64_t r0 = warp * (kRows * kSide) + side;
  const int H = a.num_kv_heads, span = a.group / 8;  // lanes of a group

  Raw8<T> raw[kRows];
  int64_t slot[kRows];
  int32_t t[kRows];
  int kind[kRows], head[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int64_t r = r0 + u * kSide;
    slot[u] = -1;
    if (r >= a.rows) continue;
    t[u] = static_cast<int32_t>(r / (2 * H));
    const int x = static_cast<int>(r - static_cast<int64_t>(t[u]) * 2 * H);
    kind[u] = x >= H;
    head[u] = x - (kind[u] ? H : 0);
    slot[u] = __ldg(a.slots + t[u]);
    const T* src = kind[u] ? static_cast<const T*>(a.v) + t[u] * a.v_stride
                           : static_cast<const T*>(a.k) + t[u] * a.k_stride;
    raw[u].load(src + head[u] * D + lane * 8);
  }
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    // every lane of the warp takes part in the reductions
    float f[8];
    raw[u].widen(f);
    float lo = f[0], hi = f[0];
    bool finite = true;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo = fminf(lo, f[e]);
      hi = fmaxf(hi, f[e]);
      finite = finite && isfinite(f[e]);
    }
    for (int o = span / 2; o >= 1; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const unsigned lanes = (1u << span) - 1;  // group / 8 is 16 at most
    const unsigned all = __ballot_sync(0xffffffffu, finite) >> (threadIdx.x % 32 / span * span);
    if (slot[u] == -1) continue;              // padding, or no such row
    float range = hi - lo;
    if ((all & lanes) != lanes || !isfinite(range)) lo = range = qnan();
    const float s = rounded<T>(__fdiv_rn(range, 15.f));
    uint32_t codes = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float c = s > 0.f ? fminf(rintf(__fdiv_rn(f[e] - lo, s)), 15.f) : 0.f;
      codes |= static_cast<uint32_t>(c) << (4 * e);
      f[e] = fmaf(c, s, lo);
    }
    T* out = static_cast<T*>(a.out[kind[u]]);
    if (out) store8(out + (static_cast<int64_t>(t[u]) * H + head[u]) * D + lane * 8, f);
    if (slot[u] < 0 || slot[u] >= a.pool) {
      if (lane == 0) set_status(a.status, PA_ERR_BAD_SLOT);
      continue;
    }
    const int64_t block =
        a.block_shift >= 0 ? slot[u] >> a.block_shift : slot[u] / a.block_size;
    const int64_t row =
        (block * H + head[u]) * a.block_size + (slot[u] - block * a.block_size);
    *reinterpret_cast<uint32_t*>(a.codes[kind[u]] + row * (D / 2) + lane * 4) = codes;
    if (lane % span == 0) {
      const int64_t i = row * (D / a.group) + lane / span;
      if constexpr (std::is_same<T, float>::value)
        static_cast<float2*>(a.pairs[kind[u]])[i] = make_float2(s, lo);
      else
        static_cast<uint32_t*>(a.pairs[kind[u]])[i] = pack2<T>(s, lo);
    }
  }
}

template <typename T, int D, int kRows>
cudaError_t launch_r(const StoreArgs& a, cudaStream_t s) {
  constexpr int64_t kPer = kNT / 32 * kRows * (32 / (D / 8));
  const int64_t ctas = (a.rows + kPer - 1) / kPer;
  if (ctas >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  pa_store_kv4_kernel<T, D, kRows><<<static_cast<unsigned>(ctas), kNT, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch(const StoreArgs& a, int D, cudaStream_t s) {
  switch (D) {
    case 64: return launch_r<T, 64, 2>(a, s);
    case 128: return launch_r<T, 128, 2>(a, s);
    default: return launch_r<T, 256, 2>(a, s);
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
  a.codes[0] = static_cast<uint8_t*>(k_codes);
  a.codes[1] = static_cast<uint8_t*>(v_codes);
  a.pairs[0] = k_scales;
  a.pairs[1] = v_scales;
  a.out[0] = k_out;
  a.out[1] = v_out;
  a.status = status;
  a.k_stride = p->k_stride;
  a.v_stride = p->v_stride;
  a.pool = static_cast<int64_t>(p->num_blocks) * p->block_size;
  a.rows = T * p->num_kv_heads * 2;
  a.num_kv_heads = p->num_kv_heads;
  a.block_size = p->block_size;
  a.block_shift = (p->block_size & (p->block_size - 1)) ? -1 : __builtin_ctz(p->block_size);
  a.group = p->group_size;
  cudaError_t e;
  switch (p->dtype) {
    case PA_F32: e = launch<float>(a, p->head_dim, stream); break;
    case PA_BF16: e = launch<__nv_bfloat16>(a, p->head_dim, stream); break;
    default: e = launch<__half>(a, p->head_dim, stream); break;
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
