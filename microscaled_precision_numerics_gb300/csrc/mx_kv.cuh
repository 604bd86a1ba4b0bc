// mx_kv.cuh -- byte layout of the NVFP4 key/value cache, shared by the kernels that write and read it.
//
// The cache is [pages, kv heads, page_size / 16] records of 18 * D bytes, D the head dimension: 16 tokens of one
// head, K codes (16 rows of D / 2 bytes), K block scales (16 rows of D / 16 bytes), V codes (16 rows of D / 2),
// V block scales ([D / 16][16], the tokens of a block side by side).  A record is contiguous whatever the page
// size, so the attention kernel fetches 16 tokens of both K and V as one run of bytes (2304 for D = 128).
//
// K is contracted along D, so a thread wants whole rows of it and the scales of neighbouring blocks; V is
// contracted along the tokens, so a thread wants the scales of neighbouring tokens as a pair: hence the two
// orders of the scales.  Token i's V scales sit at position i ^ ((i >> 1) & 1): the attention kernel gives the rows of
// an 8-row matrix fragment to tokens 0 1 3 2 4 5 7 6, so that the four rows a thread quad loads together lie in
// both halves of the 128-byte bank line instead of one.
#pragma once

#include <cstdint>

namespace mxk {

constexpr int KV_GROUP = 16;                                   // tokens of a record

__host__ __device__ constexpr int kv_record_bytes(int D) { return 18 * D; }
__host__ __device__ constexpr int kv_k_scales(int D) { return 8 * D; }        // offset of the K block scales
__host__ __device__ constexpr int kv_v_codes(int D) { return 9 * D; }         // offset of the V codes
__host__ __device__ constexpr int kv_v_scales(int D) { return 17 * D; }       // offset of the V block scales

// Fragment row <-> token inside 8 tokens, and position <-> token of a V scale (its own inverse).
__host__ __device__ constexpr int kv_token_of_row(int r) { return r ^ ((r >> 1) & 1); }

}  // namespace mxk
