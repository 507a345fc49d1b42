// pa_rope.cu -- pa_qk_norm_rope: norm of each query and key head, rotation by
// position, and the write of keys and values into the paged cache.
//
// Row t has R = Hq + 2 Hkv head rows of D elements: queries, keys, values.  A
// group of LPR lanes (a row's 16-byte pieces, at most a warp) holds one head
// row in registers: sum of squares by shuffles, y = x * r * w in float32, the
// rotation of the pair (i, i + rot / 2) by one shuffle with the lane that
// holds the partner (pairs (2i, 2i + 1) are within a lane), one rounding, one
// store: queries to q_out, keys and values to their slot (and k_out / v_out).
//
// Bound by memory: every element is read and written once.  A group takes
// kHeads head rows of one row t, so the row's angles (4 bytes per rotated
// element, as many bytes as two 16-bit head rows) are loaded once for all of
// them and several 16-byte loads are in flight.
#include <cstdint>

#include <cuda_runtime_api.h>

#include "pa_device.cuh"

namespace pa {

namespace {

constexpr int kNT = 256;

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
  int32_t interleaved, split_x, head_groups;
  float eps, weight_offset;
};

// Round E values to T and store them at p (aligned to their size).
template <typename T, int E>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[E]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < E / 4; ++i)
      reinterpret_cast<float4*>(p)[i] =
          make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
  } else {
    static_assert(E == 8, "16-byte pieces");
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const T a = round16(f[2 * i], static_cast<T*>(nullptr));
      const T b = round16(f[2 * i + 1], static_cast<T*>(nullptr));
      w[i] = bits16(a) | (static_cast<uint32_t>(bits16(b)) << 16);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__device__ __forceinline__ float round_elem(float x, float*) { return x; }
__device__ __forceinline__ __nv_bfloat16 round_elem(float x, __nv_bfloat16* p) {
  return round16(x, p);
}
__device__ __forceinline__ __half round_elem(float x, __half* p) { return round16(x, p); }

template <typename T, int D, int kHeads>
__global__ void __launch_bounds__(kNT) pa_rope_kernel(const RopeArgs a) {
  constexpr int X = 16 / sizeof(T);                   // elements of a 16-byte piece
  constexpr int LPR = D / X < 32 ? D / X : 32;        // lanes of a head row
  constexpr int E = D / LPR;                          // elements a lane holds
  constexpr int kGroups = kNT / LPR;
  static_assert(E == X || E == 2 * X, "pieces of a lane");
  const int lane = threadIdx.x % LPR;                 // within the group
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kGroups + threadIdx.x / LPR;
  const int64_t t = item / a.head_groups;
  if (t >= a.num_tokens) return;                      // whole groups leave together
  const unsigned mask = (LPR == 32 ? 0xffffffffu : ((1u << LPR) - 1u))
                        << (threadIdx.x % 32 / LPR * LPR);
  const int Hq = a.num_heads, Hkv = a.num_kv_heads, R = Hq + 2 * Hkv;
  const int first = static_cast<int>(item % a.head_groups) * kHeads;
  const int64_t slot = __ldg(a.slots + t);
  const int32_t pos = a.rot ? __ldg(a.positions + t) : 0;
  if (slot == -1) return;                             // padding
  const bool pos_ok = !a.rot || (pos >= 0 && pos < a.max_position);
  const bool slot_ok = slot >= 0 && slot < a.pool;
  if (first == 0 && lane == 0) {
    if (!slot_ok) set_status(a.status, PA_ERR_BAD_SLOT);
    if (!pos_ok) set_status(a.status, PA_ERR_BAD_POSITION);
  }
  const bool cache = a.k_cache && slot_ok && pos_ok;
  const int64_t block = slot_ok ? slot / a.block_size : 0;
  const int at = slot_ok ? static_cast<int>(slot % a.block_size) : 0;

  float x[kHeads][E];
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    const int r = first + j;
    if (r >= R) break;
    const T* src = r < Hq ? static_cast<const T*>(a.q) + t * a.q_stride + r * D
                   : r < Hq + Hkv
                       ? static_cast<const T*>(a.k) + t * a.k_stride + (r - Hq) * D
                       : static_cast<const T*>(a.v) + t * a.v_stride + (r - Hq - Hkv) * D;
    load_row<T, E>(src + lane * E, x[j]);
  }
  // the angles of this lane's elements: pair j of the row at table column j
  const int half = a.rot / 2;
  const bool rotates = a.rot && lane * E < a.rot;     // rot is a multiple of 2 E
  float cs[E], sn[E];
  if (rotates && pos_ok) {
    const float* row = a.cos_sin + static_cast<int64_t>(pos) * a.rot;
    if (a.interleaved) {
      const int c0 = lane * E / 2;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        cs[e] = __ldg(row + c0 + e / 2);
        sn[e] = __ldg(row + half + c0 + e / 2);
        if (e % 2 == 0) sn[e] = -sn[e];
      }
    } else {
      const bool low = lane * E < half;
      const int c0 = lane * E - (low ? 0 : half);
      load_row<float, E>(row + c0, cs);
      load_row<float, E>(row + half + c0, sn);
#pragma unroll
      for (int e = 0; e < E; ++e) sn[e] = low ? -sn[e] : sn[e];
    }
  }
  const int base = threadIdx.x % 32 - lane;           // the group's first lane of the warp
  const int away = half / E;                          // lanes between a pair's halves
  const int partner = base + (!rotates || a.interleaved ? lane
                              : lane < away ? lane + away : lane - away);
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    const int r = first + j;
    if (r >= R) break;
    const bool value = r >= Hq + Hkv;
    if (!value) {
      const T* w = static_cast<const T*>(r < Hq ? a.qw : a.kw);
      if (w) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) ss = fmaf(x[j][e], x[j][e], ss);
#pragma unroll
        for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
        const float rn = rsqrtf(ss * (1.f / D) + a.eps);
        float wf[E];
        load_row<T, E>(w + lane * E, wf);
#pragma unroll
        for (int e = 0; e < E; ++e) x[j][e] = x[j][e] * rn * (wf[e] + a.weight_offset);
      }
      if (a.rot) {
        if (a.interleaved) {
          if (rotates) {
#pragma unroll
            for (int e = 0; e < E; e += 2) {
              const float p = x[j][e], b = x[j][e + 1];
              x[j][e] = fmaf(p, cs[e], b * sn[e]);
              x[j][e + 1] = fmaf(b, cs[e + 1], p * sn[e + 1]);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float o = __shfl_sync(mask, x[j][e], partner);
            if (rotates) x[j][e] = fmaf(x[j][e], cs[e], o * sn[e]);
          }
        }
        if (!pos_ok) {
#pragma unroll
          for (int e = 0; e < E; ++e) x[j][e] = qnan();
        }
      }
    }
    if (r < Hq) {
      store_vec<T, E>(static_cast<T*>(a.q_out) + (t * Hq + r) * D + lane * E, x[j]);
      continue;
    }
    const int h = value ? r - Hq - Hkv : r - Hq;
    T* dense = static_cast<T*>(value ? a.v_out : a.k_out);
    if (dense) store_vec<T, E>(dense + (t * Hkv + h) * D + lane * E, x[j]);
    if (!cache) continue;
    T* pool = static_cast<T*>(value ? a.v_cache : a.k_cache) +
              (block * Hkv + h) * static_cast<int64_t>(a.block_size) * D;
    if (!a.split_x) {
      store_vec<T, E>(pool + static_cast<int64_t>(at) * D + lane * E, x[j]);
    } else if (!value) {  // 16-byte pieces [D / X][block_size][X]
#pragma unroll
      for (int g = 0; g < E / X; ++g) {
        float f[X];
#pragma unroll
        for (int e = 0; e < X; ++e) f[e] = x[j][g * X + e];
        store_vec<T, X>(pool + (static_cast<int64_t>(lane * (E / X) + g) * a.block_size + at) * X,
                        f);
      }
    } else {              // [D][block_size]
#pragma unroll
      for (int e = 0; e < E; ++e)
        pool[static_cast<int64_t>(lane * E + e) * a.block_size + at] =
            round_elem(x[j][e], static_cast<T*>(nullptr));
    }
  }
}

template <typename T, int D>
cudaError_t launch_d(RopeArgs a, int sms, cudaStream_t s) {
  constexpr int X = 16 / sizeof(T);
  constexpr int LPR = D / X < 32 ? D / X : 32;
  const int R = a.num_heads + 2 * a.num_kv_heads;
  constexpr int kHeads = 4;
  (void)sms;
  a.head_groups = (R + kHeads - 1) / kHeads;
  const int64_t items = static_cast<int64_t>(a.num_tokens) * a.head_groups;
  const int64_t grid = (items + kNT / LPR - 1) / (kNT / LPR);
  if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  pa_rope_kernel<T, D, kHeads><<<static_cast<unsigned>(grid), kNT, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const RopeArgs& a, int D, int sms, cudaStream_t s) {
  switch (D) {
    case 64: return launch_d<T, 64>(a, sms, s);
    case 128: return launch_d<T, 128>(a, sms, s);
    default: return launch_d<T, 256>(a, sms, s);
  }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

}  // namespace
}  // namespace pa

extern "C" pa_status_t pa_qk_norm_rope(const pa_rope_params_t* p, const void* q, const void* k,
                                       const void* v, const void* q_weight, const void* k_weight,
                                       const float* cos_sin, const int32_t* positions,
                                       const int64_t* slots, void* q_out, void* k_out,
                                       void* v_out, void* k_cache, void* v_cache, int32_t* status,
                                       cudaStream_t stream) {
  using namespace pa;
  if (!p || p->num_tokens < 0 || p->num_heads < 1 || p->num_kv_heads < 1) return PA_ERR_INVALID_ARG;
  if (p->block_size < 1 || p->num_blocks < 1) return PA_ERR_INVALID_ARG;
  if (p->flags & ~(PA_ROPE_INTERLEAVED | PA_FLAG_SPLIT_X)) return PA_ERR_INVALID_ARG;
  if (p->dtype != PA_F32 && p->dtype != PA_BF16 && p->dtype != PA_F16) return PA_ERR_UNSUPPORTED;
  if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (p->rotary_dim < 0 || p->rotary_dim > p->head_dim || p->rotary_dim % 16)
    return PA_ERR_INVALID_ARG;
  if (p->rotary_dim && (p->max_position < 1 || !cos_sin || !positions)) return PA_ERR_INVALID_ARG;
  if (p->num_heads > 65535 || p->num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
  if (!(p->eps >= 0.f)) return PA_ERR_INVALID_ARG;
  const int64_t D = p->head_dim, esz = p->dtype == PA_F32 ? 4 : 2;
  if (p->num_tokens > 1 &&
      (p->q_stride < p->num_heads * D || p->k_stride < p->num_kv_heads * D ||
       p->v_stride < p->num_kv_heads * D))
    return PA_ERR_INVALID_ARG;
  if (p->num_tokens == 0) return PA_OK;
  if (!q || !k || !v || !slots || !q_out) return PA_ERR_INVALID_ARG;
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
  // q_out in place only where rows coincide
  if (q_out == q && p->num_tokens > 1 && p->q_stride != p->num_heads * D)
    return PA_ERR_INVALID_ARG;
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
  a.rot = p->rotary_dim;
  a.max_position = p->max_position;
  a.interleaved = (p->flags & PA_ROPE_INTERLEAVED) ? 1 : 0;
  a.split_x = (p->flags & PA_FLAG_SPLIT_X) ? 1 : 0;
  a.eps = p->eps;
  a.weight_offset = p->weight_offset;
  const int sms = sm100_num_sms();
  cudaError_t e;
  switch (p->dtype) {
    case PA_F32: e = launch_t<float>(a, p->head_dim, sms, stream); break;
    case PA_BF16: e = launch_t<__nv_bfloat16>(a, p->head_dim, sms, stream); break;
    default: e = launch_t<__half>(a, p->head_dim, sms, stream); break;
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
