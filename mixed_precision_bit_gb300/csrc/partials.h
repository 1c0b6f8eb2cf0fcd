// The decode kernels' split partials without their merge, for calls that merge them with
// partials of their own.  Row = (sequence, query head); a row's `splits` partials of
// kPartialFloats floats are consecutive: the running maximum m of the scores in log2 units
// (-inf: nothing attended, the rest is not written), the sum l of 2^(score - m), two
// unused, o[128] = sum of 2^(score - m) * v.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "kitty.h"

namespace kitty {

constexpr int kPartialFloats = 132;

// Workspace of the partials (at least two a row).  The configuration and sizes are checked
// by the caller.
size_t decode_partial_bytes(const kitty_cfg* cfg, int B, int max_pages);
size_t f16kv_partial_bytes(const kitty_cfg* cfg, int B, int max_pages);

// A grid that the caller launches between the checks and the partials' launch, which is then
// its dependent: it neither reads nor waits for it, but one block ends after it, so what
// waits for the partials has waited for both.
struct GridAhead {
  int (*launch)(void* arg);  // KITTY_OK or an error code
  void* arg;
};

// The arguments and checks of kitty_decode_attention / kitty_f16kv_decode up to the merge;
// out is checked, not written.  *splits: the partials of each row, set before the launches.
// ahead may be NULL.
int decode_partials(const kitty_cfg* cfg, const void* q, const void* pool, int32_t pool_pages,
                    const int32_t* block_table, int32_t max_pages, const int32_t* num_pages,
                    const void* tail_k, const void* tail_v, const int32_t* tail_len, float sm_scale,
                    void* out, int32_t out_dtype, float* ws, size_t ws_bytes, int32_t B,
                    int32_t* d_status, void* stream, int* splits, const GridAhead* ahead);
int f16kv_partials(const kitty_cfg* cfg, const void* q, const void* pool, int32_t pool_pages,
                   const int32_t* block_table, int32_t max_pages, const int32_t* ctx_len,
                   float sm_scale, void* out, int32_t out_dtype, float* ws, size_t ws_bytes,
                   int32_t B, int32_t* d_status, void* stream, int* splits, const GridAhead* ahead);

}  // namespace kitty
