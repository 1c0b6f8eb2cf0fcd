// The prefix kernel of the shared-prefix decode: its arguments, plan and launch.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kitty.h"

namespace kitty {

struct PrefixArgs {
  const uint16_t* q;            // [B][Hq][128]
  const uint8_t* pool;
  const int32_t* table;         // [n_prefix] page ids
  const int32_t* prefix_pages;  // [B] or null: all share the whole prefix
  float* ws;                    // partials [B * Hq][slots]
  int32_t* d_status;
  float sm_log2;                // sm_scale * log2(e)
  uint32_t wait_polls;
  int pool_pages, n_prefix, B, Hq, Hkv, g, n_hi, blob, in_dtype;
  int splits, slots;            // of the prefix's tiles; partials a row
};

struct PrefixPlan {
  int units;   // (kv head, 256 rows) blocks of a split
  int splits;  // splits of the prefix
  int slots;   // partials a row
};

PrefixPlan prefix_plan(const kitty_cfg* cfg, bool packed, int B, int n_prefix, int max_pages);

// KITTY_OK or an error code.  A dependent launch behind it may start once all of its blocks
// have started.
int prefix_launch(const kitty_cfg* cfg, bool packed, const PrefixArgs& args, const PrefixPlan& plan,
                  cudaStream_t stream);

}  // namespace kitty
