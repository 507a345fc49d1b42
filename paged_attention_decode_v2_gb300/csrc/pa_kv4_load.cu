// pa_kv4_load.cu -- pa_load_kv4: pages of the 4-bit cache widened into pages of the
// element type, for the calls that take such pages (pa_prefill, pa_prefill_window).
//
// value = c * scale + minimum, one float32 operation, rounded once.  A lane takes
// eight codes (4 bytes) to eight elements (16 bytes, 32 in float32), so that a
// warp's loads and stores are whole lines; a page is one run of memory on both
// sides.  A CTA takes a run of the list of pages that the sequences have (pa_kv4.cuh),
// half of its threads the keys, half the values.
// Bound by memory, mostly by the 16-bit pages written.  Measured on the device, bf16:
// 24576 tokens, 4 heads of 256 (129 MB) 25.2 us = 5.1 TB/s; 33 ragged sequences, 16 heads of
// 128 (184 MB) 34.0 us = 5.4 TB/s, 80 % of the copy rate.  Sixteen codes a lane, in two
// stores of every other 16 bytes: 34 us and more.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include <cuda_runtime_api.h>

#include "pa_kv4.cuh"

namespace pa {

namespace {

constexpr int kNT = 256;
constexpr int kHalf = kNT / 2;
constexpr int kUnroll = 8;  // loads of a lane in flight
constexpr int kCtas = 4;    // resident on an SM

struct LoadArgs {
  const void* k_codes;
  const void* v_codes;
  const void* k_pairs;
  const void* v_pairs;
  void* k_out;
  void* v_out;
  const int32_t* tables;
  const int32_t* lens;
  const int32_t* out_tables;
  int32_t* status;
  int32_t num_seqs, block_size, num_blocks, num_out_blocks, width, out_width, max_len;
  int32_t page;         // elements of a page: Hkv * block_size * D
};

struct Pages {
  const LoadArgs& a;
  __device__ __forceinline__ bool ok(int32_t L) const {
    return L >= 0 && L <= a.max_len &&
           L <= static_cast<int64_t>(min(a.width, a.out_width)) * a.block_size;
  }
  __device__ __forceinline__ uint32_t operator()(int b) const {
    const int32_t L = __ldg(a.lens + b);
    return ok(L) ? (L + a.block_size - 1) / a.block_size : 0;
  }
};

template <typename T>
__device__ __forceinline__ void put8(T* p, const float (&f)[8]) {
  if constexpr (std::is_same<T, float>::value) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = bits16(round16(f[2 * i], static_cast<T*>(nullptr))) |
             static_cast<uint32_t>(bits16(round16(f[2 * i + 1], static_cast<T*>(nullptr)))) << 16;
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The values of eight codes.  Four bits at place 4e of a word are a whole number in the
// mantissa of a float of exponent 23 - 4e: no shift and no conversion, one subtraction.
__device__ __forceinline__ void widen_codes(uint32_t w, float2 p, float (&f)[8]) {
  constexpr uint32_t kOne[4] = {0x4b000000u, 0x49000000u, 0x47000000u, 0x45000000u};
  const F2 s = pair(p.x, p.x), m = pair(p.y, p.y);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const uint32_t x = h ? w >> 16 : w;
      const F2 c = add2(pair(__uint_as_float((x & (15u << 4 * e)) | kOne[e]),
                             __uint_as_float((x & (15u << 4 * (e + 1))) | kOne[e + 1])),
                        pair(-__uint_as_float(kOne[e]), -__uint_as_float(kOne[e + 1])));
      const float2 v = unpair(fma2(c, s, m));
      f[4 * h + e] = v.x;
      f[4 * h + e + 1] = v.y;
    }
  }
}

template <typename T, int GS>
__global__ void __launch_bounds__(kNT, kCtas) pa_load_kv4_kernel(const LoadArgs a) {
  extern __shared__ uint32_t start[];
  const Pages pages{a};
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.num_seqs; b += kNT)
      if (!pages.ok(__ldg(a.lens + b))) set_status(a.status, PA_ERR_BAD_SEQ_LEN);
  const uint32_t total = list_build(start, a.num_seqs, pages);
  // this CTA's run of the list; one half of it takes keys, the other values
  const uint32_t run = (total + gridDim.x - 1) / gridDim.x;
  uint32_t i = blockIdx.x * run;
  const uint32_t end = min(total, i + run);
  if (i >= end) return;
  const bool values = threadIdx.x >= kHalf;
  const int32_t units = a.page / 8;
  const uint32_t* pool = static_cast<const uint32_t*>(values ? a.v_codes : a.k_codes);
  const void* pairs = values ? a.v_pairs : a.k_pairs;
  T* wide = static_cast<T*>(values ? a.v_out : a.k_out);
  int b;
  uint32_t j;
  list_find(start, a.num_seqs, pages, i, b, j);
  uint32_t have = pages(b);
  int32_t from = __ldg(a.tables + static_cast<int64_t>(b) * a.width + j);
  int32_t to = __ldg(a.out_tables + static_cast<int64_t>(b) * a.out_width + j);
  for (;;) {
    const bool from_ok = from >= 0 && from < a.num_blocks;
    const bool to_ok = to >= 0 && to < a.num_out_blocks;
    if ((!from_ok || !to_ok) && threadIdx.x == 0) set_status(a.status, PA_ERR_BAD_BLOCK_ID);
    const int64_t unit0 = from_ok ? static_cast<int64_t>(from) * units : 0;
    const uint32_t* codes = pool + unit0;
    const int64_t pair0 = unit0 / (GS / 8);
    T* out = wide + (to_ok ? static_cast<int64_t>(to) * a.page : 0);
    // the next page's ids arrive while this page is widened
    if (++i < end) {
      if (++j >= have) {
        do have = pages(++b); while (have == 0);  // the list holds another page
        j = 0;
      }
      from = __ldg(a.tables + static_cast<int64_t>(b) * a.width + j);
      to = __ldg(a.out_tables + static_cast<int64_t>(b) * a.out_width + j);
    }
    // unit u has pair u / kPer; a lane's units are kHalf apart
    constexpr int kPer = GS / 8;
    const auto widen = [&](int32_t u0, auto whole) {
      uint32_t c[kUnroll];
      float2 p[kUnroll];
#pragma unroll
      for (int x = 0; x < kUnroll; ++x) {
        c[x] = 0;
        p[x] = make_float2(qnan(), qnan());
        if (whole.value || u0 + x * kHalf < units) {
          if (whole.value || from_ok) {
            c[x] = __ldcs(codes + u0 + x * kHalf);
            p[x] = load_pair<T>(pairs, pair0 + u0 / kPer + x * (kHalf / kPer));
          }
        }
      }
#pragma unroll
      for (int x = 0; x < kUnroll; ++x) {
        if (!whole.value && u0 + x * kHalf >= units) break;
        float f[8];
        widen_codes(c[x], p[x], f);
        put8(out + static_cast<int64_t>(u0 + x * kHalf) * 8, f);
      }
    };
    if (to_ok)
      for (int32_t u0 = threadIdx.x % kHalf; u0 < units; u0 += kHalf * kUnroll) {
        if (from_ok && u0 + (kUnroll - 1) * kHalf < units) widen(u0, std::true_type{});
        else widen(u0, std::false_type{});
      }
    if (i >= end) break;
  }
}

template <typename T>
cudaError_t launch(const LoadArgs& a, int64_t most, int group, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const unsigned grid =
      static_cast<unsigned>(std::min<int64_t>(most, static_cast<int64_t>(sms) * kCtas));
  const size_t smem = list_bytes(a.num_seqs);
  switch (group) {
    case 32: pa_load_kv4_kernel<T, 32><<<grid, kNT, smem, s>>>(a); break;
    case 64: pa_load_kv4_kernel<T, 64><<<grid, kNT, smem, s>>>(a); break;
    default: pa_load_kv4_kernel<T, 128><<<grid, kNT, smem, s>>>(a); break;
  }
  return cudaGetLastError();
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

}  // namespace
}  // namespace pa

extern "C" pa_status_t pa_load_kv4(const pa_load_kv4_params_t* p, const void* k_codes,
                                   const void* v_codes, const void* k_scales,
                                   const void* v_scales, const int32_t* block_tables,
                                   const int32_t* seq_lens, const int32_t* out_tables, void* k_out,
                                   void* v_out, int32_t* status, cudaStream_t stream) {
  using namespace pa;
  if (!p || p->num_seqs < 0 || p->num_kv_heads < 1 || p->max_seq_len < 0) return PA_ERR_INVALID_ARG;
  if (p->block_size < 1 || p->num_blocks < 1 || p->num_out_blocks < 1) return PA_ERR_INVALID_ARG;
  if (p->max_blocks_per_seq < 1 || p->max_out_blocks_per_seq < 1) return PA_ERR_INVALID_ARG;
  if (pa_status_t st = check_kv4(p->dtype, p->head_dim, p->group_size)) return st;
  if (p->num_seqs > 65535 || p->num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
  const int64_t pages = (static_cast<int64_t>(p->max_seq_len) + p->block_size - 1) / p->block_size;
  if (pages > p->max_blocks_per_seq || pages > p->max_out_blocks_per_seq) return PA_ERR_INVALID_ARG;
  // units of a page and pages of a call are counted in 31 bits
  const double page = static_cast<double>(p->num_kv_heads) * p->block_size * p->head_dim;
  const int64_t most = p->num_seqs * pages;
  if (page + 8.0 * kNT * kUnroll >= 2147483648.0 || 2 * most + 65536 >= (int64_t(1) << 31) ||
      static_cast<int64_t>(p->max_seq_len) + p->block_size >= (int64_t(1) << 31))
    return PA_ERR_UNSUPPORTED;
  if (p->num_seqs == 0) return PA_OK;
  if (!k_codes || !v_codes || !k_scales || !v_scales || !block_tables || !seq_lens ||
      !out_tables || !k_out || !v_out)
    return PA_ERR_INVALID_ARG;
  for (const void* x : {k_codes, v_codes, k_scales, v_scales, static_cast<const void*>(k_out),
                        static_cast<const void*>(v_out)})
    if (!aligned(x, 16)) return PA_ERR_MISALIGNED;
  if (!aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(out_tables, 4) ||
      !aligned(status, 4))
    return PA_ERR_MISALIGNED;
  {
    const double esz = p->dtype == PA_F32 ? 4 : 2, all = 4e18;
    const auto size = [&](double bytes) { return static_cast<size_t>(std::min(bytes, all)); };
    const size_t codes = size(page * p->num_blocks / 2);
    const size_t pairs = size(page * p->num_blocks / p->group_size * 2 * esz);
    const size_t wide = size(page * p->num_out_blocks * esz);
    const size_t B = static_cast<size_t>(p->num_seqs);
    const Range r[] = {{k_codes, codes, false}, {v_codes, codes, false}, {k_scales, pairs, false},
                       {v_scales, pairs, false},
                       {block_tables, B * p->max_blocks_per_seq * 4, false},
                       {seq_lens, B * 4, false},
                       {out_tables, B * p->max_out_blocks_per_seq * 4, false},
                       {k_out, wide, true}, {v_out, wide, true}, {status, 4, true}};
    if (outputs_overlap(r, sizeof r / sizeof r[0])) return PA_ERR_INVALID_ARG;
  }
  LoadArgs a{};
  a.k_codes = k_codes;
  a.v_codes = v_codes;
  a.k_pairs = k_scales;
  a.v_pairs = v_scales;
  a.k_out = k_out;
  a.v_out = v_out;
  a.tables = block_tables;
  a.lens = seq_lens;
  a.out_tables = out_tables;
  a.status = status;
  a.num_seqs = p->num_seqs;
  a.block_size = p->block_size;
  a.num_blocks = p->num_blocks;
  a.num_out_blocks = p->num_out_blocks;
  a.width = p->max_blocks_per_seq;
  a.out_width = p->max_out_blocks_per_seq;
  a.max_len = p->max_seq_len;
  a.page = static_cast<int32_t>(page);
  // no page at all: the lengths are still looked at
  const int64_t grid = std::max<int64_t>(most, 1);
  cudaError_t e;
  switch (p->dtype) {
    case PA_F32: e = launch<float>(a, grid, p->group_size, stream); break;
    case PA_BF16: e = launch<__nv_bfloat16>(a, grid, p->group_size, stream); break;
    default: e = launch<__half>(a, grid, p->group_size, stream); break;
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
