// pa_span.cuh -- which tokens a windowed query sees, and where they lie.
//
// A query at position p sees t <= p with t < S (sinks) or t >= ws, ws =
// max(0, p + 1 - W).  Two lists of the same tokens are used:
//   * the plain list (CUDA-core kernel): the sinks below ws, then ws .. p;
//   * the block list (tensor-core decode kernel, which copies whole blocks):
//     the sinks' ceil(S / BS) blocks, then the blocks from ws / BS on.  With
//     `shift` blocks left out between the two, list token v of the sequence
//     is token v (sink blocks) or v + shift * BS.  The tokens of these blocks
//     that the query does not see are one run of list tokens,
//     [S, ws - shift * BS): the rest of the last sink block and the start of
//     the window's first block.  Every block of the list holds a visible
//     token, so no aligned part of the list is empty.
#pragma once

#include <cstdint>

namespace pa {

struct WindowSpan {
  int32_t len;     // tokens of the block list
  int32_t h0, h1;  // its invisible run (empty when h0 >= h1)
  int32_t sinks;   // sink blocks: entries below this are not shifted
  int32_t shift;   // blocks left out after them
};

// L tokens, the query at L - 1 (L >= 0); window >= 1, num_sinks >= 0.
__host__ __device__ inline WindowSpan window_span(int32_t L, int32_t window, int32_t num_sinks,
                                                  int32_t block_size) {
  WindowSpan w;
  const int32_t ws = L > window ? L - window : 0;
  w.sinks = num_sinks / block_size + (num_sinks % block_size != 0);
  const int32_t skip = ws / block_size - w.sinks;
  w.shift = skip > 0 ? skip : 0;
  w.len = L - w.shift * block_size;
  w.h0 = num_sinks;
  w.h1 = ws - w.shift * block_size;
  return w;
}

// The longest block list of sequences of at most max_len tokens.
inline int64_t window_max_len(int64_t max_len, int64_t window, int64_t num_sinks,
                              int64_t block_size) {
  const int64_t most = window + block_size - 1 + (num_sinks + block_size - 1) / block_size *
                                                     block_size;
  return max_len < most ? max_len : most;
}

// How the tensor-core prefix pass splits a prefix of `len` tokens: the key
// tiles (128 tokens) of all KV heads, head after head, are cut into key blocks
// of `block` tiles, at most `key_blocks` of them.  The part of a head in one
// key block is a segment: one partial result of the head's rows.
struct PrefixSplit {
  uint32_t tiles;  // key tiles of a head
  uint32_t block;  // key tiles of a key block (>= 1)
  // segments of head kvh: the key blocks with a tile of it
  __host__ __device__ int segments(uint32_t kvh) const {
    return tiles ? static_cast<int>(((kvh + 1) * tiles - 1) / block - kvh * tiles / block) + 1 : 0;
  }
};

// The tiles of all heads must number less than 2^31.
__host__ __device__ inline PrefixSplit prefix_split(int32_t len, uint32_t num_kv_heads,
                                                    uint32_t key_blocks) {
  PrefixSplit s;
  s.tiles = (static_cast<uint32_t>(len) + 127) / 128;
  const uint32_t all = s.tiles * num_kv_heads;
  s.block = all > key_blocks ? (all + key_blocks - 1) / key_blocks : 1;
  return s;
}

}  // namespace pa
