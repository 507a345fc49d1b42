// pa_rows.cuh -- attention of many query rows over a list of key tiles on the
// tensor cores (tcgen05): the windowed prefill and the shared-prefix pass.
//
// Rows.  The G query heads of one KV head share its keys, so a tile of up to
// 128 rows holds nq = 128 / G tokens (prefill) or sequences (prefix) times G
// heads: row r is token r / G, head r % G, and one TMA copy with box (64
// elements, G heads, nq tokens) brings a 64-element slice of all of them.
// Keys and values are read once for the G heads.
//
// Work unit: the rows of one or two tiles against a run of 128-key tiles.
//   * windowed prefill: (sequence, KV head, group of tokens); the key tiles
//     are those that hold a token some row sees: the sinks' tiles, then the
//     window's, context tiles from the paged cache and chunk tiles from the
//     dense tensors; rows are masked in the tiles that need it;
//   * prefix: (key block, row group): the key tiles of all KV heads are one
//     line cut into key blocks (pa_span.cuh); the row groups of one key block
//     run side by side on neighbouring CTAs, so a key tile comes from HBM once
//     and from L2 for the others.  Results are partials (max, sum, output)
//     that pa_join.cu joins.
//
// Steps.  A unit is a sequence of steps, each one product of a row tile with
// a key tile: QK^T into one of two tensor-memory buffers ("slots"), softmax
// of that slot by its own four warps, one thread per row, P written over the
// logits in 16 bits (keys 0-63 handed on before 64-127), and P.V from tensor
// memory.  The MMA warp issues QK^T(k), P.V(k - 1), so the tensor core works on
// one slot while the warps of the other run their softmax.  Twelve warps: 0-7
// softmax, 8 issues the MMAs, 9 and 10 stream keys and values through a ring of
// five 32 KB stages, 11 loads the next unit's rows.
//   head_dim 128, two row tiles ("dual"): slot s is row tile s, both against
//     the same key tile, which is read from shared memory twice and copied
//     once; each slot has its own output accumulator.
//   head_dim 128, one row tile (prefix of a small batch): slots take the key
//     tiles in turn, each with its own accumulator, maximum and sum: two
//     partials for the join.
//   head_dim 256: one row tile and one accumulator (256 of the 512 columns);
//     slots take the key tiles in turn and hand the row's reference maximum
//     from one to the other through shared memory as soon as it is known.
// The reference moves only when a tile's maximum exceeds it by more than 2^8
// (then the sum and the accumulator are rescaled), so p <= 2^8.  For f16, whose
// smallest step is 2^-24, it lies 2^7 below the maximum (p <= 2^15): with p <= 1
// at first, 20000 keys of weight 2^-25.2 next to one of weight 1 were lost.  Sums
// and accumulators are float32; p alone is rounded to 16 bits (the operand type
// of the MMA): by half a step of the type, in f16 also by 2^-32 of the largest p
// at most; the sum adds the unrounded p.
//
// Bound by the tensor core for many rows (4 * head_dim flops per row and key),
// and by latency for few.  Measured: prefix of 32000 tokens, 256 sequences, 32 / 8
// heads of 128: 81 us at full clocks = 1660 TFLOP/s, tensor pipe 82 % busy (in a
// loop the power cap holds 1.54 GHz: 93 us); windowed chunk of 4096 tokens,
// window 2048, 24 / 4 heads of 256: 174 us for 213 visible GFLOP, tensor pipe
// 68 % busy of the 86 % that 784 equal units leave on 152 SMs; 5 ragged chunks,
// window 512, 32 / 8 heads of 128: 31 us, 37 % busy (short units, masked tiles).
// What mattered: the MMA operands in uniform registers (an MMA was issued every
// 100 cycles instead of 64; 214 -> 165 us on the prefix), long stages and P in
// halves (165 -> 139), P against the reference in hand at head_dim 128
// (139 -> 127), and code that fits the instruction cache (119 -> 69 KB; windowed
// chunk 195 -> 176).  Pairs of CTAs with multicast keys gained 0-3 %, and a next
// unit's first QK^T ahead of the last P.V lost 2-4 %: neither is kept.
// Every wait is bounded; one that gives up makes the CTA's results NaN.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include <cuda.h>

#include "pa_device.cuh"
#include "pa_sm100.cuh"
#include "pa_span.cuh"

namespace pa {

namespace rw {

constexpr int kProducers = 2;        // warps that stream keys and values
constexpr int kMmaWarp = 8;          // warps 0-7 softmax, 9 and 10 producers, 11 the rows
constexpr int kRowWarp = kMmaWarp + 1 + kProducers;
constexpr int kThreads = 32 * (kRowWarp + 1);
constexpr int kTile = 128;           // rows of a row tile, keys of a key tile
constexpr int kStage = 32768;        // ring stage: two 64-element slices of a key tile, or values
constexpr int kSliceBytes = 16384;   // a 64-element slice of 128 rows
constexpr int kMaxStages = 5;
constexpr int kTmemCols = 512;       // S slot 0 | S slot 1 | O (two of 128, or one of 256)
constexpr int kOCol = 256;
constexpr float kRescaleLog2 = 8.f;
template <typename T>                // log2 of how far the reference lies below the maximum
constexpr float kBelowLog2 = std::is_same<T, __half>::value ? 7.f : 0.f;
constexpr long long kWaitBudget = 4000000000LL;    // cycles (about 2 s)
constexpr long long kSelftestBudget = 20000000LL;  // cycles (about 10 ms)
constexpr int kSmemLimit = 227 * 1024;
// register shares: the launch gives kThreads * 168; the softmax warps hold a
// row's 128 logits, the other warpgroup needs few (256 * 208 + 128 * 88)
constexpr int kSoftmaxRegs = 208;
constexpr int kOtherRegs = 88;

template <int D>
struct Layout {
  static constexpr int kSlices = D / 64;
  static constexpr int kKStages = kSlices / 2;         // ring stages of a key tile
  static constexpr int kVTokens = kStage / (D * 2);    // keys of a value stage
  static constexpr int kQBytes = 65536;                // D 128: two row tiles, D 256: one
  static constexpr int kStages = kMaxStages;
  static constexpr int kRingOff = kQBytes;
  static constexpr int kCtrlOff = kRingOff + kStages * kStage;
  static constexpr int kSmem = kCtrlOff + 2048 + 1024; // + room to align to 1024
  static_assert(kSmem <= kSmemLimit, "shared memory");
};

struct Ctrl {
  uint64_t full[kMaxStages];   // stage landed
  uint64_t empty[kMaxStages];  // stage consumed by its MMAs
  uint64_t qfull, qempty;      // row tiles landed / no longer read
  uint64_t s_full[2];          // a slot's logits ready
  uint64_t p_ready[2][2];      // a slot's P written, keys 0-63 and 64-127 (128 threads arrive)
  uint64_t o_done[2];          // the P.V of a slot's step (D 256), of its last step completed
  uint64_t m_next[2];          // D 256: the slot's step has published the reference maximum
  uint64_t o_free;             // D 256: the accumulator has been read (256 threads arrive)
  uint64_t tail[kProducers];   // producer-private: a value stage to be cleared landed
  uint64_t drain;              // abort path: all issued MMAs finished
  uint64_t never;              // self-test: nothing ever arrives here
  uint32_t tmem;
  int abort;
  int before[kRowsMaxCompact / 32 + 1];  // row groups before each 32 sequences (windowed prefill)
  float mref[kTile];           // D 256: a row's reference maximum, handed from slot to slot
  float lsum[2][kTile];        // D 256: the slots' sums at the end of a unit
};
static_assert(sizeof(Ctrl) <= 2048, "control block");

// One work unit, decoded the same way by every role.
struct Unit {
  int kvh;
  int seq;           // block-table row
  int32_t i0, n;     // first token (sequence of the batch), tokens of the sequence (batch)
  int64_t row0;      // tensor row of token 0
  int32_t ctx;       // positions from here on are chunk rows
  int32_t lo_min;    // the first row's window begins here: [sinks, lo_min) is seen by no row
  int32_t pmax;      // last position that a row sees
  int tiles;         // key tiles of the unit
  int low, skip;     // tile j < low is tile j, else tile j + skip
  int nctx;          // context key tiles of the sequence
  bool poison;
  bool run;          // false: nothing to do (a segment list's end)
  int part;          // prefix: the partial's segment
};

struct Tile {
  int32_t pos0;      // position of its first key
  int nk;            // keys
  bool ctx;          // from the cache
  int32_t chunk;     // chunk row of its first key (dense tiles)
};

__device__ __forceinline__ Tile tile_of(const Unit& u, int j) {
  Tile t;
  const int x = j < u.low ? j : j + u.skip;
  t.ctx = x < u.nctx;
  if (t.ctx) {
    t.pos0 = x * kTile;
    t.nk = min(kTile, u.ctx - t.pos0);
    t.chunk = 0;
  } else {
    t.chunk = (x - u.nctx) * kTile;
    t.pos0 = u.ctx + t.chunk;
    t.nk = min(kTile, u.pmax + 1 - t.pos0);
  }
  return t;
}

// The units of one CTA, in order; every role walks the same sequence.
struct Walk {
  uint32_t k;        // next unit (windowed prefill) or next item (prefix)
  uint32_t x, end;   // prefix: rest of the item's key tiles on the line
  int rt;            // prefix: its row group
};

__device__ __forceinline__ Walk walk_begin() { return Walk{blockIdx.x, 0, 0, 0}; }

// Windowed prefill: row groups of sequence b are ceil(n_b / a.group_tokens).
__device__ __forceinline__ bool chunk_ok(const RowsArgs& a, int b, int32_t& s0, int32_t& n) {
  s0 = __ldg(a.query_start + b);
  const int32_t s1 = __ldg(a.query_start + b + 1);
  n = s1 - s0;
  return s0 >= 0 && s1 >= s0 && n <= a.max_query_len && s1 <= a.num_tokens;
}

// Row groups of sequences up to and including b (a lane each, from a multiple
// of 32), and of b alone.
__device__ __forceinline__ int groups_scan(const RowsArgs& a, int b, int& mine) {
  int32_t s0, n;
  mine = b < a.num_seqs && chunk_ok(a, b, s0, n) ? (n + a.group_tokens - 1) / a.group_tokens : 0;
  int x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (static_cast<int>(threadIdx.x & 31) >= o) x += y;
  }
  return x;
}

template <bool kPrefix>
__device__ __forceinline__ bool walk_next(const RowsArgs& a, const int* before, Walk& w, Unit& u) {
  if constexpr (kPrefix) {
    const int32_t len = __ldg(a.lens);
    if (len < 1 || len > a.max_ctx_len) return false;  // the join reports it
    // counts of units, tiles and blocks fit 31 bits (checked on the host)
    const PrefixSplit sp = prefix_split(len, a.num_kv_heads, a.key_blocks);
    const uint32_t tiles = sp.tiles, block = sp.block, all = tiles * a.num_kv_heads;
    if (w.x >= w.end) {
      const uint32_t kb = w.k / static_cast<uint32_t>(a.row_groups);
      if (kb * block >= all) return false;
      w.rt = static_cast<int>(w.k - kb * a.row_groups);
      w.x = kb * block;
      w.end = min(all, w.x + block);
      w.k += gridDim.x;
    }
    u.kvh = static_cast<int>(w.x / tiles);
    const int j0 = static_cast<int>(w.x - u.kvh * tiles);
    const int n = static_cast<int>(min(w.end, (u.kvh + 1) * tiles) - w.x);
    u.part = static_cast<int>(w.x / block - u.kvh * tiles / block);
    w.x += n;
    u.seq = 0;
    u.i0 = w.rt * a.group_tokens;
    u.n = a.num_tokens;
    u.row0 = 0;
    u.ctx = len;
    u.lo_min = 0;
    u.pmax = len - 1;
    u.tiles = n;
    u.low = 0;
    u.skip = j0;
    u.nctx = static_cast<int>(tiles);
    u.poison = false;
    return true;
  } else {
    int32_t s0, n;
    while (true) {
      int b, g;
      if (before) {
        const int blocks = (a.num_seqs + 31) / 32;
        const uint32_t heads = a.num_kv_heads;
        if (w.k >= before[blocks] * heads) return false;
        const int x = static_cast<int>(w.k / heads);
        u.kvh = static_cast<int>(w.k - x * heads);
        w.k += gridDim.x;
        int lo = 0, hi = blocks;  // the 32 sequences: largest lo with before[lo] <= x
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (before[mid] <= x) lo = mid;
          else hi = mid;
        }
        // the sequence among them: a lane each (the whole warp walks together)
        const int lane = threadIdx.x & 31;
        int mine;
        const int upto = groups_scan(a, lo * 32 + lane, mine) + before[lo];
        const int at = __ffs(__ballot_sync(0xffffffffu, upto > x)) - 1;
        b = lo * 32 + at;
        g = x - __shfl_sync(0xffffffffu, upto - mine, at);
        chunk_ok(a, b, s0, n);
      } else {
        const uint32_t heads = a.num_kv_heads, per = a.num_seqs * heads;
        if (w.k >= per * a.row_groups) return false;
        g = static_cast<int>(w.k / per);
        const uint32_t rem = w.k - g * per;
        w.k += gridDim.x;
        b = static_cast<int>(rem / heads);
        u.kvh = static_cast<int>(rem - b * heads);
        if (!chunk_ok(a, b, s0, n) || g * a.group_tokens >= n) continue;
      }
      const int32_t C = __ldg(a.lens + b);
      u.poison = !(C >= 0 && C <= a.max_ctx_len &&
                   C <= static_cast<int64_t>(a.max_blocks_per_seq) * a.block_size);
      u.ctx = u.poison ? 0 : C;
      u.seq = b;
      // later tokens first: their lists are the longest
      const int groups = (n + a.group_tokens - 1) / a.group_tokens;
      u.i0 = (groups - 1 - g) * a.group_tokens;
      u.n = n;
      u.row0 = s0;
      const int32_t last = min(n, u.i0 + a.group_tokens) - 1;
      u.pmax = u.ctx + last;
      u.lo_min = max(0, u.ctx + u.i0 - a.window + 1);
      u.nctx = (u.ctx + kTile - 1) / kTile;
      const int total = u.nctx + last / kTile + 1;
      const int sinks = a.num_sinks <= u.ctx
                            ? (a.num_sinks + kTile - 1) / kTile
                            : u.nctx + (a.num_sinks - u.ctx + kTile - 1) / kTile;
      const int first = u.lo_min < u.ctx ? u.lo_min / kTile
                                         : u.nctx + (u.lo_min - u.ctx) / kTile;
      u.low = min(sinks, first);
      u.skip = first - u.low;
      u.tiles = total - u.skip;
      return true;
    }
  }
}

// 2^x by the hardware's approximate exponential: relative error well below the
// 16-bit rounding that p goes through; inputs are at most 15 here.
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack16(float a, float b, __nv_bfloat16*) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack16(float a, float b, __half*) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The largest of three in one instruction.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Two floats in one 64-bit register, for the packed float32 instructions.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Bring a tile's bytes into L2.
__device__ __forceinline__ void tma_prefetch_4d(const void* tmap, int32_t x, int32_t y, int32_t z,
                                                int32_t w) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// Eight 32-bit words to p (32-byte aligned) in one store: a whole sector.  A
// thread stores its own row, so a warp's store touches 32 rows, and 16-byte
// stores would write every sector twice.
__device__ __forceinline__ void st_sector(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
// 16 elements of a row, from element i (a multiple of 16) of `out`, which is
// 16-byte aligned: by sectors where it is 32-byte aligned.
__device__ __forceinline__ void store_16(void* out, int64_t i, int32_t dtype, bool sectors,
                                         const float (&v)[16]) {
  if (!sectors) {
    store_row16(out, i, dtype, v);
    return;
  }
  uint32_t w[8];
  if (dtype == PA_F32) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(v[8 * h + k]);
      st_sector(static_cast<float*>(out) + i + 8 * h, w);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k)
    w[k] = dtype == PA_BF16 ? pack16(v[2 * k], v[2 * k + 1], static_cast<__nv_bfloat16*>(nullptr))
                            : pack16(v[2 * k], v[2 * k + 1], static_cast<__half*>(nullptr));
  st_sector(static_cast<uint16_t*>(out) + i, w);
}

// Bits e of [lo, hi) within a 32-key word that starts at key c0.
__device__ __forceinline__ uint32_t range_bits(int lo, int hi, int c0) {
  const int a = max(lo - c0, 0), b = min(hi - c0, 32);
  if (a >= b) return 0u;
  const uint32_t up = b >= 32 ? 0xffffffffu : ((1u << b) - 1u);
  return up & (0xffffffffu << a);
}

// Each thread reads 32 consecutive columns of its tensor-memory lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// Four MMAs of one 64-element slice (descriptors 32 bytes apart), or of 64 keys
// (P 8 columns apart), issued by one elected lane: one election for the four.
__device__ __forceinline__ void mma4_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        bool accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p, e, t;\n"
      "elect.sync _|e, 0xffffffff;\n"
      "setp.ne.b32 p, %10, 0;\n"
      "setp.eq.b32 t, 0, 0;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %5, %9, p;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %2, %6, %9, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %3, %7, %9, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %4, %8, %9, t;\n"
      "}\n" ::"r"(d),
      "l"(a), "l"(a + 2), "l"(a + 4), "l"(a + 6), "l"(b), "l"(b + 2), "l"(b + 4), "l"(b + 6),
      "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint64_t b0, uint64_t b1,
                                        uint64_t b2, uint64_t b3, uint32_t idesc,
                                        bool accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p, e, t;\n"
      "elect.sync _|e, 0xffffffff;\n"
      "setp.ne.b32 p, %10, 0;\n"
      "setp.eq.b32 t, 0, 0;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %5, %9, p;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%2], %6, %9, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%3], %7, %9, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%4], %8, %9, t;\n"
      "}\n" ::"r"(d),
      "r"(a), "r"(a + 8), "r"(a + 16), "r"(a + 24), "l"(b0), "l"(b1), "l"(b2), "l"(b3),
      "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}

// x of lane 0, for values that all lanes hold alike.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

__device__ __forceinline__ void sync256() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

}  // namespace rw

// qmap: q as (64, Hq, rows, D / 64), box (64, G, nq, 1); knmap / vnmap: the
// chunk's keys and values as (64, Hkv, T, D / 64), boxes (64, 1, 128, 1) and
// (64, 1, BS, D / 64) (windowed prefill only); kcmap / vcmap: the caches as
// rows of head_dim (box 64 x BS, and a whole block slice-major).
template <typename T, int D, int BS, bool kPrefix, bool kDual>
__global__ void __launch_bounds__(rw::kThreads, 1)
    pa_rows_kernel(const RowsArgs a, const __grid_constant__ CUtensorMap qmap,
                   const __grid_constant__ CUtensorMap knmap,
                   const __grid_constant__ CUtensorMap vnmap,
                   const __grid_constant__ CUtensorMap kcmap,
                   const __grid_constant__ CUtensorMap vcmap, long long budget) {
  using namespace rw;
  using Lay = Layout<D>;
  constexpr int NST = Lay::kStages;
  constexpr int kSl = Lay::kSlices;
  constexpr int kVT = Lay::kVTokens;
  constexpr bool kChain = D == 256;   // one accumulator, the maximum handed on
  static_assert(D == 128 || D == 256, "head_dim");
  static_assert(BS % 16 == 0 && kTile % BS == 0 && kVT % BS == 0, "block size");
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr unsigned kAll = 0xffffffffu;

  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (sm100::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* qs = smem;
  uint8_t* ring = smem + Lay::kRingOff;
  Ctrl& c = *reinterpret_cast<Ctrl*>(smem + Lay::kCtrlOff);

  // The warp index and what the MMA warp branches on or addresses with go
  // through uniform(): known to be the same in all lanes, they stay in uniform
  // registers, where the MMA instruction takes its operands from.
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  static_assert(!kDual || D == 128, "two row tiles");
  constexpr bool dual = kDual;

  if constexpr (kPrefix) asm volatile("griddepcontrol.launch_dependents;");

  if (tid == 0) {
    for (int s = 0; s < NST; ++s) {
      sm100::mbar_init(&c.full[s], 1);
      sm100::mbar_init(&c.empty[s], 1);
    }
    sm100::mbar_init(&c.qfull, 1);
    sm100::mbar_init(&c.qempty, 1);
    for (int s = 0; s < 2; ++s) {
      sm100::mbar_init(&c.s_full[s], 1);
      sm100::mbar_init(&c.p_ready[s][0], 128);
      sm100::mbar_init(&c.p_ready[s][1], 128);
      sm100::mbar_init(&c.o_done[s], 1);
      sm100::mbar_init(&c.m_next[s], 128);
    }
    sm100::mbar_init(&c.o_free, 256);
    for (int p = 0; p < kProducers; ++p) sm100::mbar_init(&c.tail[p], 1);
    sm100::mbar_init(&c.drain, 1);
    sm100::mbar_init(&c.never, 1);
    c.abort = 0;
    if (kPrefix && blockIdx.x == 0) {
      const int32_t len = __ldg(a.lens);
      if (len < 0 || len > a.max_ctx_len) set_status(a.status, PA_ERR_BAD_SEQ_LEN);
    }
  }
  if (warp == kMmaWarp) {
    sm100::tmem_alloc(&c.tmem, kTmemCols);
    sm100::tmem_relinquish();
  }
  if (warp == kMmaWarp + 1 && lane == 0) {
    sm100::tma_prefetch_desc(&qmap);
    sm100::tma_prefetch_desc(&kcmap);
    sm100::tma_prefetch_desc(&vcmap);
    if (!kPrefix) {
      sm100::tma_prefetch_desc(&knmap);
      sm100::tma_prefetch_desc(&vnmap);
    }
  }
  // windowed prefill of up to kRowsMaxCompact sequences: only row groups that
  // exist are walked
  const bool compact = !kPrefix && a.num_seqs <= kRowsMaxCompact;
  if (compact && warp == 0) {
    int carry = 0, mine;
    for (int b0 = 0; b0 < a.num_seqs; b0 += 32) {
      if (lane == 0) c.before[b0 / 32] = carry;
      carry += __shfl_sync(kAll, groups_scan(a, b0 + lane, mine), 31);
    }
    if (lane == 0) c.before[(a.num_seqs + 31) / 32] = carry;
  }
  sm100::fence_proxy_async_smem();
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = uniform(c.tmem);
  const int* before = compact ? c.before : nullptr;
  volatile int* abort_flag = &c.abort;

  if (warp >= kMmaWarp) {
    // one instruction for the whole warpgroup, before its roles part
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    uint64_t keep;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(keep));
    if (warp == kRowWarp) {
      // ========================= row loader =========================================
      // The unit's row tiles, as soon as the last unit's QK^T are done with theirs.
      // The rows come from HBM in 128-byte pieces, several microseconds for a
      // tile: so the next unit's are fetched into L2 while this one runs.
      uint32_t un = 0;
      bool ok = true;
      Walk wk = walk_begin();
      Unit u;
      const int copies = dual ? 2 * kSl : kSl;
      bool more = true;
      for (int i = 0;; ++i) {
        // i = 0: find the first unit; then load one and find the next
        if (i > 0) {
          ok = __all_sync(kAll, sm100::mbar_wait(&c.qempty, (un & 1) ^ 1, budget, abort_flag));
          if (!ok) break;
          // rows past the sequence belong to others or are filled with zeros;
          // their results are never stored
          if (lane == 0)
            sm100::mbar_arrive_expect_tx(&c.qfull, copies * a.row_tokens * a.group * 128);
          __syncwarp();
          if (lane < copies)
            sm100::tma_load_4d(qs + lane * kSliceBytes, &qmap, &c.qfull, 0, u.kvh * a.group,
                               static_cast<int32_t>(u.row0) + u.i0 + lane / kSl * a.row_tokens,
                               lane % kSl, keep);
          ++un;
        }
        more = walk_next<kPrefix>(a, before, wk, u);
        if (!more) break;
        if (i > 0 && lane < copies)
          tma_prefetch_4d(&qmap, 0, u.kvh * a.group,
                          static_cast<int32_t>(u.row0) + u.i0 + lane / kSl * a.row_tokens,
                          lane % kSl);
      }
      if (!ok) {
        if (lane == 0) c.abort = 1;
        if (un > 0) sm100::mbar_wait(&c.qfull, (un - 1) & 1, budget, nullptr);
      }
    } else if (warp > kMmaWarp) {
      // ========================= producers ==========================================
      // Both walk the stages in the order the MMA warp takes them -- dual: keys,
      // values of each tile; else keys 0, then (keys j, values j - 1), then the
      // last values -- and each fills every other one.
      const uint32_t pid = static_cast<uint32_t>(warp - kMmaWarp - 1);
      uint64_t* my_tail = &c.tail[pid];
      uint32_t g = 0, tn = 0;
      int tail_pending = -1;
      bool ok = true;

      // Block id of each lane's block of a context tile; loaded a tile ahead.
      auto ctx_id = [&](const Unit& u, int j) -> int32_t {
        if (j >= u.tiles) return -1;
        const Tile t = tile_of(u, j);
        if (!t.ctx || lane >= (t.nk + BS - 1) / BS) return -1;
        return __ldg(a.block_tables + static_cast<int64_t>(u.seq) * a.max_blocks_per_seq +
                     t.pos0 / BS + lane);
      };
      // Its TMA row; a block outside the pool, or one that no row sees, becomes
      // a negative row, which TMA fills with zeros instead of reading memory.
      auto ctx_row = [&](const Unit& u, const Tile& t, int32_t id) -> int32_t {
        const int32_t p = t.pos0 + lane * BS;
        const bool seen = kPrefix || p < a.num_sinks || p + BS > u.lo_min;
        return (!seen || id < 0 || id >= a.num_blocks) ? -BS : (id * a.num_kv_heads + u.kvh) * BS;
      };
      auto wait_empty = [&](int slot) {
        return __all_sync(kAll, sm100::mbar_wait(&c.empty[slot], ((g / NST) & 1) ^ 1, budget,
                                                 abort_flag)) != 0;
      };

      auto issue_k = [&](const Unit& u, const Tile& t, int32_t y) -> bool {
        constexpr int kMaxBlk = kTile / BS;
        const int nblk = (t.nk + BS - 1) / BS;
        for (int sl = 0; sl < kSl; sl += 2, ++g) {
          if (g % kProducers != pid) continue;
          const int slot = g % NST;
          if (!wait_empty(slot)) return false;
          uint8_t* st = ring + slot * kStage;
          if (t.ctx) {
            // one lane per block and slice
            const int blk = lane % kMaxBlk, half = lane / kMaxBlk;
            const int32_t yj = __shfl_sync(kAll, y, blk);
            if (lane == 0) sm100::mbar_arrive_expect_tx(&c.full[slot], 2 * nblk * BS * 128);
            __syncwarp();
            if (half < 2 && blk < nblk)
              sm100::tma_load_2d(st + half * kSliceBytes + blk * BS * 128, &kcmap, &c.full[slot],
                                 (sl + half) * 64, yj, keep);
          } else {
            if (lane == 0) sm100::mbar_arrive_expect_tx(&c.full[slot], kStage);
            __syncwarp();
            if (lane < 2)
              sm100::tma_load_4d(st + lane * kSliceBytes, &knmap, &c.full[slot], 0, u.kvh,
                                 static_cast<int32_t>(u.row0) + t.chunk, sl + lane, keep);
          }
          __syncwarp();
        }
        return true;
      };

      // Values of a tile.  Keys that no row sees -- past the tile's last key up
      // to the end of its 16-key MMA step, and the run between the sinks and
      // the first row's window -- are cleared before the stage is handed on:
      // their p is zero, but 0 * NaN would be NaN.  Such a stage lands on the
      // producer's own barrier first.
      auto issue_v = [&](const Unit& u, const Tile& t, int32_t y) -> bool {
        const int nv = (t.nk + kVT - 1) / kVT;
        // the unseen run [h0, h1) of the tile; of a context tile, blocks inside it
        // have come as zeros, so only the ends in blocks that are seen remain:
        // [h0, e0) and [e1, h1)
        const int h0 = kPrefix ? 0 : max(0, a.num_sinks - t.pos0);
        const int h1 = kPrefix ? 0 : max(h0, min(t.nk, u.lo_min - t.pos0));
        const int e0 = t.ctx ? min(h1, (h0 + BS - 1) / BS * BS) : h1;
        const int e1 = t.ctx && h0 < h1 ? max(e0, h1 / BS * BS) : h1;
        for (int v = 0; v < nv; ++v, ++g) {
          if (g % kProducers != pid) continue;
          const int slot = g % NST;
          if (!wait_empty(slot)) return false;
          const int toks = min(kVT, t.nk - v * kVT);
          const int ncp = (toks + BS - 1) / BS;  // copies, of BS rows each
          // rows of this stage to clear: [a0, a1), [b0, b1) and [toks, z1)
          const int a0 = max(h0 - v * kVT, 0), a1 = max(a0, min(e0 - v * kVT, toks));
          const int b0 = max(e1 - v * kVT, 0), b1 = max(b0, min(h1 - v * kVT, toks));
          const int z1 = (toks + 15) / 16 * 16;
          const bool clear = a0 < a1 || b0 < b1 || toks < z1;
          uint64_t* land = clear ? my_tail : &c.full[slot];
          uint8_t* st = ring + slot * kStage;
          if (lane == 0) sm100::mbar_arrive_expect_tx(land, ncp * BS * D * 2);
          __syncwarp();
          if (t.ctx) {
            const int32_t yj = __shfl_sync(kAll, y, (v * kVT / BS + lane) & 31);
            if (lane < ncp)
              sm100::tma_load_3d(st + lane * BS * D * 2, &vcmap, land, 0, yj, 0, keep);
          } else if (lane < ncp) {
            sm100::tma_load_4d(st + lane * BS * D * 2, &vnmap, land, 0, u.kvh,
                               static_cast<int32_t>(u.row0) + t.chunk + v * kVT + lane * BS, 0,
                               keep);
          }
          __syncwarp();
          if (clear) {
            tail_pending = slot;
            if (!__all_sync(kAll, sm100::mbar_wait(my_tail, tn & 1, budget, abort_flag)))
              return false;
            ++tn;
            tail_pending = -1;
            auto zero = [&](int r0, int r1) {
              for (int i = lane; i < (r1 - r0) * kSl * 8; i += 32) {
                const int line = i / 8, r = r0 + line / kSl, sl = line % kSl;
                *reinterpret_cast<uint4*>(st + ((r / BS * kSl + sl) * BS + r % BS) * 128 +
                                          i % 8 * 16) = make_uint4(0u, 0u, 0u, 0u);
              }
            };
#pragma unroll 1
            for (int x = 0; x < 3; ++x)
              zero(x == 0 ? a0 : x == 1 ? b0 : toks, x == 0 ? a1 : x == 1 ? b1 : z1);
            sm100::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(&c.full[slot]);
          }
        }
        return true;
      };

      Walk wk = walk_begin();
      Unit u;
      while (ok && walk_next<kPrefix>(a, before, wk, u)) {
        // j = -1 only looks up tile 0's blocks; the last round has values alone
        int32_t y = 0, yprev = 0, id = 0;
        Tile t{}, tprev{};
#pragma unroll 1
        for (int j = -1; j <= u.tiles && ok; ++j) {
          if (j >= 0) {
            yprev = y;
            tprev = t;
            t = tile_of(u, j);
            y = t.ctx ? ctx_row(u, t, id) : 0;
          }
          id = ctx_id(u, j + 1);
          if (j >= 0 && j < u.tiles) ok = issue_k(u, t, y);
          if (dual ? j >= 0 && j < u.tiles : j > 0)
            if (ok) ok = issue_v(u, dual ? t : tprev, dual ? y : yprev);
        }
      }
      if (!ok) {
        if (lane == 0) c.abort = 1;
        // copies already issued must land before the CTA may exit
        for (uint32_t gg = g > NST ? g - NST : 0; gg < g; ++gg)
          if (gg % kProducers == pid && static_cast<int>(gg % NST) != tail_pending)
            sm100::mbar_wait(&c.full[gg % NST], (gg / NST) & 1, budget, nullptr);
        if (tail_pending >= 0) sm100::mbar_wait(my_tail, tn & 1, budget, nullptr);
      }
    } else {
      // ========================= MMA issuer =========================================
      // One MMA occupies the tensor core for 64 (N = 128) or 128 cycles and this
      // warp issues in order, one instruction every few cycles, so every
      // instruction between MMAs counts: slots are compile-time, ring positions
      // are counted, descriptors are a base plus constants, four MMAs share an
      // election, and nothing is waited for that an earlier wait implies.
      constexpr uint32_t id_qk = sm100::idesc_f16(kBf16, false, false, 128, kTile);
      constexpr uint32_t id_pv = sm100::idesc_f16(kBf16, false, true, 128, D);
      const uint64_t q_desc = sm100::smem_desc(sm100::smem_u32(qs), 16, 1024, sm100::kSw128);
      const uint64_t k_desc = sm100::smem_desc(sm100::smem_u32(ring), 16, 1024, sm100::kSw128);
      const uint64_t v_desc =
          sm100::smem_desc(sm100::smem_u32(ring), BS * 128, 1024, sm100::kSw128);
      struct Ring {
        uint32_t slot, phase;
        __device__ __forceinline__ void next() {
          if (++slot == NST) {
            slot = 0;
            phase ^= 1;
          }
        }
      };
      Ring rg{0, 0};              // next stage of the ring
      Ring rk{0, 0}, rv{0, 0};    // dual: stages of the current key and value tiles
      uint32_t un = 0;            // units
      uint32_t parity[2] = {0, 0};  // of the P.V in each slot
      bool ok = true;
      using S0 = std::integral_constant<int, 0>;
      using S1 = std::integral_constant<int, 1>;
      if (a.selftest_stall)
        ok = __all_sync(kAll, sm100::mbar_wait(&c.never, 0, budget, abort_flag));
      auto wait_for = [&](uint64_t* bar, uint32_t phase) {
        const bool r = __all_sync(kAll, sm100::mbar_wait(bar, phase, budget, abort_flag)) != 0;
        sm100::tc_fence_after();
        return r;
      };
      // logits into slot S: keys from the ring, or (dual, slot 1) those in hand
      auto qk = [&](auto slot) -> bool {
        const int S = slot;
        const bool kFresh = !kDual || S == 0, kDone = !kDual || S == 1;
        if (kFresh) rk = rg;
        Ring r = rk;
        const uint32_t d = tmem + S * kTile;
        const uint64_t qd = q_desc + (kDual && S ? kSl * kSliceBytes / 16 : 0);
#pragma unroll
        for (int st = 0; st < Lay::kKStages; ++st) {
          if (kFresh && !wait_for(&c.full[r.slot], r.phase)) return false;
          const uint64_t kd = k_desc + r.slot * (kStage / 16);
          mma4_ss(d, qd + 2 * st * (kSliceBytes / 16), kd, id_qk, st != 0);
          mma4_ss(d, qd + (2 * st + 1) * (kSliceBytes / 16), kd + kSliceBytes / 16, id_qk, true);
          if (kDone) sm100::mma_commit_elect(&c.empty[r.slot]);
          r.next();
        }
        if (kFresh) rg = r;
        return true;
      };
      // the MMAs of keys r0 .. r0 + 63 of one value stage (rows of BS per slice),
      // as many as the stage's `toks` keys reach
      auto pv_keys = [&](auto from, uint32_t stage, uint32_t at, uint32_t o, int toks, bool first) {
        constexpr int r0 = decltype(from)::value;
        const uint64_t vd = v_desc + stage * (kStage / 16);
        auto off = [](int r) {
          return static_cast<uint64_t>(((r / BS) * BS * D * 2 + (r % BS) * 128) / 16);
        };
        if (toks >= r0 + 64) {
          mma4_ts(o, at + r0 / 2, vd + off(r0), vd + off(r0 + 16), vd + off(r0 + 32),
                  vd + off(r0 + 48), id_pv, !first || r0 != 0);
          return;
        }
#pragma unroll 1
        for (int r = r0; r < toks; r += 16)
          sm100::mma_f16_ts_elect(o, at + r / 2, vd + off(r), id_pv, !first || r != 0);
      };
      // P.V of slot S over a tile of nk keys; `first`: the accumulator starts anew
      auto pv = [&](auto slot, int nk, bool first) -> bool {
        const int S = slot;
        const bool kFresh = !kDual || S == 0, kDone = !kDual || S == 1;
        if (kFresh) rv = rg;
        Ring r = rv;
        if (kFresh && !wait_for(&c.full[r.slot], r.phase)) return false;
        if (!wait_for(&c.p_ready[S][0], parity[S])) return false;
        const uint32_t o = tmem + kOCol + (kChain ? 0 : S * 128);
        const uint32_t at = tmem + S * kTile;
        // keys 0-63, then, when their P is there too, keys 64-127
        pv_keys(S0{}, r.slot, at, o, nk, first);
        if constexpr (kVT == 64) {
          if (kDone) sm100::mma_commit_elect(&c.empty[r.slot]);
          r.next();
        }
        if (!wait_for(&c.p_ready[S][1], parity[S])) return false;
        parity[S] ^= 1;
        if constexpr (kVT == 64) {
          if (nk > 64) {
            if (kFresh && !wait_for(&c.full[r.slot], r.phase)) return false;
            pv_keys(S0{}, r.slot, at + 32, o, nk - 64, false);
            if (kDone) sm100::mma_commit_elect(&c.empty[r.slot]);
            r.next();
          }
        } else {
          if (nk > 64) pv_keys(std::integral_constant<int, 64>{}, r.slot, at, o, nk, false);
          if (kDone) sm100::mma_commit_elect(&c.empty[r.slot]);
          r.next();
        }
        if (kFresh) rg = r;
        // a step's softmax may have to rescale the accumulator: with one
        // accumulator per slot, the logits it has waited for imply that the
        // slot's last P.V is done; with one for both slots they do not
        if constexpr (kChain) sm100::mma_commit_elect(&c.o_done[S]);
        return true;
      };

      Walk wk = walk_begin();
      Unit u;
      while (ok) {
        const bool more = walk_next<kPrefix>(a, before, wk, u);
        if (!__all_sync(kAll, more)) break;
        ok = wait_for(&c.qfull, un & 1);
        if (!ok) break;
        ++un;
        const int tiles = uniform(u.tiles);
        int nk = 0, nk_prev = 0;
        // QK^T of tile j, P.V of the step before; one more round for the last P.V
#pragma unroll 1
        for (int j = 0; j <= tiles; ++j) {
          const bool more_keys = j < tiles;
          if (more_keys) {
            nk = uniform(tile_of(u, j).nk);
          }
          if constexpr (kDual) {
            if (more_keys) {
              if (!(ok = qk(S0{}))) break;
              sm100::mma_commit_elect(&c.s_full[0]);
            } else {
              sm100::mma_commit_elect(&c.o_done[0]);
            }
            if (j > 0 && !(ok = pv(S1{}, nk_prev, j == 1))) break;
            if (!more_keys) {
              sm100::mma_commit_elect(&c.o_done[1]);
              break;
            }
            if (!(ok = qk(S1{}))) break;
            if (j == tiles - 1) sm100::mma_commit_elect(&c.qempty);
            sm100::mma_commit_elect(&c.s_full[1]);
            if (!(ok = pv(S0{}, nk, j == 0))) break;
          } else {
            if (more_keys) {
              if (!(ok = qk(j & 1))) break;
              if (j == tiles - 1) sm100::mma_commit_elect(&c.qempty);
              sm100::mma_commit_elect(&c.s_full[j & 1]);
            } else if (!kChain && tiles > 1) {
              // the slot before the last is done with its accumulator
              sm100::mma_commit_elect(&c.o_done[j & 1]);
            }
            if (j > 0) {
              // one accumulator: not before the last unit's has been read
              if (kChain && j == 1 && un > 1 && !(ok = wait_for(&c.o_free, un & 1))) break;
              if (!(ok = pv((j - 1) & 1, nk_prev, kChain ? j == 1 : j <= 2))) break;
              if (!kChain && !more_keys) sm100::mma_commit_elect(&c.o_done[(j - 1) & 1]);
            }
          }
          nk_prev = nk;
        }
      }
      if (!ok) {
        if (lane == 0) c.abort = 1;
        // no MMA may still be running when tensor memory is released
        sm100::mma_commit_elect(&c.drain);
        sm100::mbar_wait(&c.drain, 0, budget, nullptr);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ========================= softmax + epilogue =================================
    // Slot = warpgroup; thread r of it owns row r of the slot's row tile
    // (tensor-memory lane r).  Every thread runs the same iterations and
    // barriers whatever happens; a failed wait only marks the abort, which
    // ends later waits.
    const int slot = warp >> 2;
    const int r = tid & 127;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t sbuf = tmem + lane_base + slot * kTile;
    const uint32_t obuf = tmem + lane_base + kOCol + (kChain ? 0 : slot * 128);
    const float sl2 = a.scale_log2;
    uint32_t done[2] = {0, 0};  // steps of each slot in the units before
    uint32_t units = 0;         // units in which this slot had a step
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!sm100::mbar_wait(bar, parity & 1, budget, abort_flag)) c.abort = 1;
    };
    // token and head of this row within the unit
    const int tile = dual ? slot : 0;
    const int tok = r / a.group, head = r - tok * a.group;
    const bool row_in = tok < a.row_tokens;
    Walk wk = walk_begin();
    Unit u;
    while (walk_next<kPrefix>(a, before, wk, u)) {
      const int K = dual ? 2 * u.tiles : u.tiles;
      const int32_t i = u.i0 + tile * a.row_tokens + tok;
      const bool row_ok = row_in && i < u.n;
      // window of the row (rows that are not stored take the first one's)
      const int32_t p = u.ctx + (row_ok ? i : u.i0);
      const int32_t lo = p - a.window + 1;
      float m_ref = -INFINITY, lsum = 0.f;
      bool bad = u.poison;
      for (int k = slot; k < K; k += 2) {
        const Tile t = tile_of(u, dual ? k >> 1 : k);
        // a context block outside the pool poisons the unit (blocks that no
        // row sees are not looked at); tested after P is written
        int32_t blk_id = 0;
        if (t.ctx && lane < (t.nk + BS - 1) / BS) {
          const int32_t bp = t.pos0 + lane * BS;
          if (kPrefix || bp < a.num_sinks || bp + BS > u.lo_min)
            blk_id = __ldg(a.block_tables + static_cast<int64_t>(u.seq) * a.max_blocks_per_seq +
                           t.pos0 / BS + lane);
        }
        wait(&c.s_full[slot], done[slot] + (k >> 1));
        sm100::tc_fence_after();
        __syncwarp();
        float s[kTile];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(sbuf + 32 * q, s + 32 * q);
        sm100::tmem_wait_ld();
        // rows see all of the tile, or the keys of a mask
        const bool whole =
            kPrefix ? t.nk == kTile
                    : t.nk == kTile && t.pos0 + kTile - 1 <= u.ctx + u.i0 &&
                          (t.pos0 >= u.pmax - a.window + 1 || t.pos0 + kTile <= a.num_sinks);
        if (!whole) {
          const int hi = kPrefix ? t.nk : min(t.nk, p - t.pos0 + 1);
          const int from = kPrefix ? 0 : lo - t.pos0;
          const int sk = kPrefix ? 0 : a.num_sinks - t.pos0;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t bits = range_bits(0, hi, 32 * q) &
                                  (range_bits(from, kTile, 32 * q) | range_bits(0, sk, 32 * q));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(bits >> e & 1u)) s[32 * q + e] = -INFINITY;
          }
        }
        // The row's reference maximum before this step: the slot's own, or the
        // other slot's after the step before.  P is computed against it at once,
        // while the tile's maximum is still being found; only when that exceeds the
        // one the reference was taken from by more than 2^8 (the first tile, rarely
        // later) the reference moves, what the sum and the accumulator hold is
        // rescaled, and the first keys are taken again.
        const float m_old = m_ref;
        if constexpr (kChain) {
          if (k > 0) {
            const int o = slot ^ 1;
            wait(&c.m_next[o], done[o] + ((k - 1) >> 1));
            m_ref = c.mref[r];
          }
        }
        const float m_in = m_ref;
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < kTile; e += 8)
#pragma unroll
          for (int x = 0; x < 4; ++x) mx[x] = max3(mx[x], s[e + 2 * x], s[e + 2 * x + 1]);
        const float mt = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * sl2;
        const bool move = mt > m_in + (kRescaleLog2 + kBelowLog2<T>);  // also from -inf
        if (move) m_ref = mt - kBelowLog2<T>;
        if constexpr (kChain) {
          c.mref[r] = m_ref;
          sm100::mbar_arrive(&c.m_next[slot]);
        }
        // p = 2^(s * scale * log2(e) - m), two keys per 32-bit column over the
        // logits this thread has read
        float neg_m = m_in == -INFINITY ? 0.f : -m_in;
        const uint64_t sc2 = pair(sl2, sl2);
        uint64_t neg2, add[2];
        auto exps = [&](int e0, float (&w)[16]) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float p0, p1;
            unpair(fma2(pair(s[e0 + e], s[e0 + e + 1]), sc2, neg2), p0, p1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            add[(e >> 1) & 1] = add2(add[(e >> 1) & 1], pair(p0, p1));
            w[e / 2] = __uint_as_float(pack16(p0, p1, static_cast<T*>(nullptr)));
          }
        };
        // what the accumulator holds of the steps before, at the new reference
        auto rescale = [&]() {
          const float corr = move ? (m_in == -INFINITY ? 0.f : exp2f(m_in - m_ref)) : 1.f;
          if constexpr (kChain) {
            wait(&c.o_done[slot ^ 1], done[slot ^ 1] + ((k - 1) >> 1));
            sm100::tc_fence_after();
            __syncwarp();
          }  // one accumulator per slot is complete: see the MMA warp
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 16) {
            float ov[16];
            sm100::tmem_ld16(obuf + c0, ov);
            sm100::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) ov[e] *= corr;
            sm100::tmem_st16(obuf + c0, ov);
          }
          sm100::tmem_wait_st();
        };
        // head_dim 256 leaves the softmax twice the time (its products take
        // twice as long): there the reference is moved first
        float w0[16], w1[16];
        for (bool again = kChain;;) {
          if (again && __any_sync(kAll, move)) {
            neg_m = m_ref == -INFINITY ? 0.f : -m_ref;
            if (kChain ? k > 0 : k >= 2) rescale();
          }
          neg2 = pair(neg_m, neg_m);
          add[0] = add[1] = 0;
          exps(0, w0);
          exps(32, w1);
          if (again || !__any_sync(kAll, move)) break;
          again = true;
        }
        if (m_ref != m_old) lsum *= m_old == -INFINITY ? 0.f : exp2f(m_old - m_ref);
        sm100::tmem_st16(sbuf, w0);
        sm100::tmem_st16(sbuf + 16, w1);
        sm100::tmem_wait_st();
        sm100::tc_fence_before();
        sm100::mbar_arrive(&c.p_ready[slot][0]);
        exps(64, w0);
        sm100::tmem_st16(sbuf + 32, w0);
        exps(96, w1);
        sm100::tmem_st16(sbuf + 48, w1);
        sm100::tmem_wait_st();
        sm100::tc_fence_before();
        sm100::mbar_arrive(&c.p_ready[slot][1]);
        float sum0, sum1;
        unpair(add2(add[0], add[1]), sum0, sum1);
        lsum += sum0 + sum1;
        bad |= __any_sync(kAll, blk_id < 0 || blk_id >= a.num_blocks) != 0;
      }
      // ---- epilogue: the row's accumulator over its sum ----------------------------
      const int mine = slot == 0 ? (K + 1) >> 1 : K >> 1;  // this slot's steps
      float total = lsum, m_end = m_ref;
      int c_lo = 0, c_hi = D;
      if constexpr (kChain) {
        // both slots' sums at the last reference; each slot stores half the columns
        sync256();
        m_end = c.mref[r];
        if (m_end != m_ref) lsum *= m_ref == -INFINITY ? 0.f : exp2f(m_ref - m_end);
        c.lsum[slot][r] = bad ? -1.f : lsum;  // a sum is never negative: -1 is a bad block
        sync256();
        total = c.lsum[0][r] + c.lsum[1][r];
        bad |= c.lsum[0][r] == -1.f || c.lsum[1][r] == -1.f;
        c_lo = slot * (D / 2);
        c_hi = c_lo + D / 2;
        const int o = (K - 1) & 1;
        wait(&c.o_done[o], done[o] + ((K - 1) >> 1));
      } else if (mine > 0) {
        wait(&c.o_done[slot], units);
        ++units;
      }
      sm100::tc_fence_after();
      __syncwarp();
      const bool poison = bad || *abort_flag != 0;
      const float inv = poison ? qnan() : total > 0.f ? 1.f / total : 0.f;
      const int64_t orow = (u.row0 + i) * a.num_heads + u.kvh * a.group + head;
      const bool empty = !kChain && mine == 0;
      int64_t at = orow;
      if constexpr (kPrefix)
        at = orow * a.num_parts + (D == 128 && !dual ? 2 * u.part + slot : u.part);
      const bool sectors = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
#pragma unroll 1
      for (int c0 = c_lo; c0 < c_hi; c0 += 32) {
        float ov[32];
        tmem_ld32(obuf + c0, ov);
        sm100::tmem_wait_ld();
        if (row_ok) {
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = empty ? 0.f : ov[e] * inv;
#pragma unroll
          for (int e = 0; e < 32; e += 16) {
            float(&part)[16] = *reinterpret_cast<float(*)[16]>(&ov[e]);
            if constexpr (kPrefix)
              store_16(a.part_out, at * D + c0 + e, PA_F32, true, part);
            else
              store_16(a.out, at * D + c0 + e, a.out_dtype, sectors, part);
          }
        }
      }
      if constexpr (kPrefix) {
        if (row_ok && c_lo == 0) {
          a.part_max[at] = poison ? qnan() : m_end * kLn2;
          a.part_sum[at] = total;
          if (poison)
            set_status(a.status, *abort_flag ? PA_ERR_DEVICE_TIMEOUT : PA_ERR_BAD_BLOCK_ID);
        }
      }
      sm100::tc_fence_before();
      if constexpr (kChain) sm100::mbar_arrive(&c.o_free);
      done[0] += (K + 1) >> 1;
      done[1] += K >> 1;
    }
  }

  // ---- teardown -------------------------------------------------------------------
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  if (warp == kMmaWarp) sm100::tmem_dealloc(tmem, kTmemCols);
  // the join, a dependent of this grid, reads what the pass before it wrote
  if constexpr (kPrefix) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Persistent launch: one CTA per SM (it takes nearly all shared memory and all
// tensor-memory columns).
template <typename T, int D, int BS, bool kPrefix, bool kDual>
cudaError_t launch_rows_v(const RowsArgs& a, const CUtensorMap (&m)[5], int grid, bool pdl,
                          cudaStream_t s) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
  auto kern = pa_rows_kernel<T, D, BS, kPrefix, kDual>;
  // set once per device; concurrent first calls set the same attribute
  static std::atomic<bool> configured[128];
  if (!configured[dev].load(std::memory_order_acquire)) {
    if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             rw::Layout<D>::kSmem))
      return e;
    configured[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(rw::kThreads, 1, 1);
  cfg.dynamicSmemBytes = rw::Layout<D>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  const long long budget = a.selftest_stall ? rw::kSelftestBudget : rw::kWaitBudget;
  return cudaLaunchKernelEx(&cfg, kern, a, m[0], m[1], m[2], m[3], m[4], budget);
}

template <typename T, int BS, bool kPrefix>
cudaError_t launch_rows_128(const RowsArgs& a, const CUtensorMap (&m)[5], int grid, bool pdl,
                            cudaStream_t s) {
  // a windowed prefill always takes two row tiles
  if constexpr (kPrefix)
    if (!a.dual) return launch_rows_v<T, 128, BS, kPrefix, false>(a, m, grid, pdl, s);
  return launch_rows_v<T, 128, BS, kPrefix, true>(a, m, grid, pdl, s);
}

template <typename T, bool kPrefix>
cudaError_t launch_rows_t(const RowsArgs& a, const CUtensorMap (&m)[5], int grid, bool pdl,
                          cudaStream_t s) {
  if (a.head_dim == 256 && a.block_size == 16)
    return launch_rows_v<T, 256, 16, kPrefix, false>(a, m, grid, pdl, s);
  if (a.head_dim == 256 && a.block_size == 32)
    return launch_rows_v<T, 256, 32, kPrefix, false>(a, m, grid, pdl, s);
  if (a.head_dim != 128) return cudaErrorInvalidValue;
  if (a.block_size == 16) return launch_rows_128<T, 16, kPrefix>(a, m, grid, pdl, s);
  if (a.block_size == 32) return launch_rows_128<T, 32, kPrefix>(a, m, grid, pdl, s);
  if (a.block_size == 64) return launch_rows_128<T, 64, kPrefix>(a, m, grid, pdl, s);
  return cudaErrorInvalidValue;
}

}  // namespace pa
