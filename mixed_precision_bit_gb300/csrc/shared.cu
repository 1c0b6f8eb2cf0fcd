// Decode attention of a batch whose sequences share a prefix (sm_103a).
//
//   out[b][hq] = softmax(sm_scale * q . [K_prefix; K_b]) . [V_prefix; V_b]
//
// with the prefix's pages attended once for the whole batch and each sequence's own
// cache by the split-K decode.  Three launches: the prefix kernel's partials; behind it, as a
// dependent that fills the SMs that the prefix leaves, the decode kernel's partials over the
// own pages and tails; and one merge of both.  (The prefix kernel behind the decode kernel
// waited for whole SMs: 16 x 4096 tokens 20.7 against 17.2 us.)
#include "grid_dep.cuh"
#include "host_common.h"
#include "kitty_common.cuh"
#include "partials.h"
#include "prefix.h"

#include <algorithm>
#include <cmath>

namespace kitty {
namespace {

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct MergeParams {
  const float *a, *b;  // partials of the prefix and of the own pages, row-major
  void* out;
  int32_t* d_status;
  int na, nb, rows, out_dtype, wide;  // wide: out is 16-byte aligned
};

// WARPS warps a row (4 / WARPS rows a block).  Every warp reads the row's maxima, one slot a
// lane, and weighs them; warp w sums slots w, w + WARPS, ... of the unscaled outputs, four
// channels a lane, requested together with the maxima; the warps' sums meet in shared memory.
// A slot that attended nothing (m = -inf) has weight 0 and its outputs are not used.
constexpr int kAhead = 8;

template <int WARPS>
__global__ void __launch_bounds__(128) merge_kernel(const MergeParams p) {
  constexpr int kRound = WARPS * kAhead;  // slots of a row taken at once
  static_assert(kRound <= 32, "a lane a slot");
  __shared__ float4 part[4][32];
  grid_wait();
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31, w = wid % WARPS;
  const int row = blockIdx.x * (4 / WARPS) + wid / WARPS;
  const bool in = row < p.rows;
  const int n = in ? p.na + p.nb : 0;
  const float* a = p.a + (size_t)(in ? row : 0) * p.na * kPartialFloats;
  const float* b = p.b + (size_t)(in ? row : 0) * p.nb * kPartialFloats;
  auto slot = [&](int s) { return s < p.na ? a + (size_t)s * kPartialFloats : b + (size_t)(s - p.na) * kPartialFloats; };
  float ms = -INFINITY, L = 0.f;
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < n; s0 += kRound) {
    const int end = min(n, s0 + kRound);
    const float2 ml = s0 + lane < end ? *reinterpret_cast<const float2*>(slot(s0 + lane)) : make_float2(-INFINITY, 0.f);
    float4 o[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int s = s0 + w + k * WARPS;
      o[k] = s < end ? reinterpret_cast<const float4*>(slot(s) + 4)[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float mr = fmaxf(ml.x, ms);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mr = fmaxf(mr, __shfl_xor_sync(0xFFFFFFFFu, mr, d));
    if (mr == -INFINITY) continue;
    const float f = ms == -INFINITY ? 0.f : exp2_fast(ms - mr);
    const float e = ml.x == -INFINITY ? 0.f : exp2_fast(ml.x - mr);
    float l = e == 0.f ? 0.f : ml.y * e;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
    L = L * f + l;
    O = make_float4(O.x * f, O.y * f, O.z * f, O.w * f);
    ms = mr;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const float es = __shfl_sync(0xFFFFFFFFu, e, w + k * WARPS);
      if (es != 0.f) {
        O.x = fmaf(o[k].x, es, O.x);
        O.y = fmaf(o[k].y, es, O.y);
        O.z = fmaf(o[k].z, es, O.z);
        O.w = fmaf(o[k].w, es, O.w);
      }
    }
  }
  if (WARPS > 1) {
    part[wid][lane] = O;
    __syncthreads();
    if (w != 0) return;
#pragma unroll
    for (int k = 1; k < WARPS; ++k) {
      const float4 x = part[wid + k][lane];
      O = make_float4(O.x + x.x, O.y + x.y, O.z + x.z, O.w + x.w);
    }
  }
  if (!in) return;
  const bool ok = L != 0.f;
  if (!ok && lane == 0) set_status(p.d_status, KITTY_ST_EMPTY);
  const float r[4] = {ok ? O.x / L : 0.f, ok ? O.y / L : 0.f, ok ? O.z / L : 0.f, ok ? O.w / L : 0.f};
  const size_t i = (size_t)row * kD + 4 * lane;
  if (p.wide) {  // the outputs are 16-byte aligned
    if (p.out_dtype == KITTY_F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + i) = make_float4(r[0], r[1], r[2], r[3]);
    } else {
      uint2 h;
      if (p.out_dtype == KITTY_BF16) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(r[0], r[1]), y = __floats2bfloat162_rn(r[2], r[3]);
        h = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
      } else {
        h = make_uint2(h2_bits(__floats2half2_rn(r[0], r[1])), h2_bits(__floats2half2_rn(r[2], r[3])));
      }
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + i) = h;
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (p.out_dtype == KITTY_F32) static_cast<float*>(p.out)[i + k] = r[k];
    else if (p.out_dtype == KITTY_BF16) static_cast<__nv_bfloat16*>(p.out)[i + k] = __float2bfloat16_rn(r[k]);
    else static_cast<__half*>(p.out)[i + k] = __float2half_rn(r[k]);
  }
}

size_t prefix_bytes(const kitty_cfg* cfg, const PrefixPlan& plan, int B) {
  return (size_t)B * cfg->num_q_heads * plan.slots * kPartialFloats * sizeof(float);
}

int check_shared(const kitty_cfg* cfg, bool packed, int B, int n_prefix, int max_pages) {
  const int rc = check_cfg(cfg, packed ? 32 : 4);
  if (rc != KITTY_OK) return rc;
  if (B < 0 || n_prefix < 0 || max_pages < 0) return KITTY_ERR_INVALID_ARG;
  return KITTY_OK;
}

int workspace(const kitty_cfg* cfg, bool packed, int B, int n_prefix, int max_pages, size_t* bytes) {
  const int rc = check_shared(cfg, packed, B, n_prefix, max_pages);
  if (rc != KITTY_OK) return rc;
  if (!bytes) return KITTY_ERR_INVALID_ARG;
  *bytes = 0;
  if (B == 0) return KITTY_OK;
  *bytes = prefix_bytes(cfg, prefix_plan(cfg, packed, B, n_prefix, max_pages), B) +
           (packed ? decode_partial_bytes(cfg, B, max_pages) : f16kv_partial_bytes(cfg, B, max_pages));
  return KITTY_OK;
}

// Launches the prefix kernel, for GridAhead.
struct PrefixCall {
  const kitty_cfg* cfg;
  bool packed;
  PrefixArgs args;
  PrefixPlan plan;
  cudaStream_t stream;
  static int launch(void* arg) {
    const PrefixCall* c = static_cast<const PrefixCall*>(arg);
    return prefix_launch(c->cfg, c->packed, c->args, c->plan, c->stream);
  }
};

// Checks; then the prefix kernel, the own pages' partials (`own` checks the rest and launches
// both) behind the prefix's in the workspace, and the merge.
template <class Own>
int shared_attention(const kitty_cfg* cfg, bool packed, const void* q, const void* pool,
                     int32_t pool_pages, const int32_t* prefix_table, int32_t n_prefix,
                     const int32_t* prefix_pages, int32_t max_pages, float sm_scale, void* out,
                     int32_t out_dtype, void* ws, size_t ws_bytes, int32_t B, int32_t* d_status,
                     void* stream, Own own) {
  int rc = check_shared(cfg, packed, B, n_prefix, max_pages);
  if (rc != KITTY_OK) return rc;
  if (n_prefix > 0 && (!prefix_table || !pool || !aligned16(pool))) return KITTY_ERR_INVALID_ARG;
  if (B == 0) return KITTY_OK;
  if (q && !aligned16(q)) return KITTY_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  PrefixCall call = {cfg, packed, {}, prefix_plan(cfg, packed, B, n_prefix, max_pages), s};
  const size_t mine = prefix_bytes(cfg, call.plan, B);
  if (ws_bytes < mine || !ws || !aligned16(ws)) return KITTY_ERR_WORKSPACE;
  float* own_ws = static_cast<float*>(ws) + mine / sizeof(float);
  PrefixArgs& p = call.args;
  p.q = static_cast<const uint16_t*>(q);
  p.pool = static_cast<const uint8_t*>(pool);
  p.table = prefix_table;
  p.prefix_pages = prefix_pages;
  p.ws = static_cast<float*>(ws);
  p.d_status = d_status;
  p.sm_log2 = sm_scale * 1.4426950408889634f;
  p.wait_polls = cfg->decode_wait_polls > 0 ? (uint32_t)cfg->decode_wait_polls : 1u << 22;
  p.pool_pages = pool_pages;
  p.n_prefix = n_prefix;
  p.B = B;
  p.Hq = cfg->num_q_heads;
  p.Hkv = cfg->num_kv_heads;
  p.g = p.Hq / p.Hkv;
  p.n_hi = cfg->n_hi;
  p.blob = (int)blob_bytes(cfg->n_hi, cfg->lo_bit, v_bits(cfg));
  p.in_dtype = cfg->in_dtype;
  p.splits = call.plan.splits;
  p.slots = call.plan.slots;
  MergeParams m = {static_cast<float*>(ws), own_ws, out, d_status, call.plan.slots, 0, B * cfg->num_q_heads, out_dtype, aligned16(out)};
  const GridAhead ahead = {PrefixCall::launch, &call};
  rc = own(own_ws, ws_bytes - mine, &m.nb, call.plan.splits > 0 ? &ahead : nullptr);
  if (rc != KITTY_OK) return rc;
  const int n = m.na + m.nb;
  const cudaError_t e = n <= kAhead
      ? launch_dependent(merge_kernel<1>, dim3((unsigned)((m.rows + 3) / 4)), 128, 0, s, m)
      : n <= 2 * kAhead
      ? launch_dependent(merge_kernel<2>, dim3((unsigned)((m.rows + 1) / 2)), 128, 0, s, m)
      : launch_dependent(merge_kernel<4>, dim3((unsigned)m.rows), 128, 0, s, m);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? KITTY_OK : KITTY_ERR_CUDA;
}

}  // namespace
}  // namespace kitty

using namespace kitty;

extern "C" int kitty_shared_workspace_bytes(const kitty_cfg* cfg, int32_t B, int32_t n_prefix,
                                            int32_t max_pages, size_t* bytes) {
  return workspace(cfg, true, B, n_prefix, max_pages, bytes);
}

extern "C" int kitty_f16kv_shared_workspace_bytes(const kitty_cfg* cfg, int32_t B, int32_t n_prefix,
                                                  int32_t max_pages, size_t* bytes) {
  return workspace(cfg, false, B, n_prefix, max_pages, bytes);
}

extern "C" int kitty_decode_attention_shared(
    const kitty_cfg* cfg, const void* q, const void* pool, int32_t pool_pages,
    const int32_t* prefix_table, int32_t n_prefix, const int32_t* prefix_pages,
    const int32_t* block_table, int32_t max_pages, const int32_t* num_pages, const void* tail_k,
    const void* tail_v, const int32_t* tail_len, float sm_scale, void* out, int32_t out_dtype,
    void* workspace, size_t workspace_bytes, int32_t B, int32_t* d_status, void* stream) {
  return shared_attention(
      cfg, true, q, pool, pool_pages, prefix_table, n_prefix, prefix_pages, max_pages, sm_scale, out,
      out_dtype, workspace, workspace_bytes, B, d_status, stream,
      [&](float* ws, size_t bytes, int* splits, const GridAhead* ahead) {
        return decode_partials(cfg, q, pool, pool_pages, block_table, max_pages, num_pages, tail_k,
                               tail_v, tail_len, sm_scale, out, out_dtype, ws, bytes, B, d_status,
                               stream, splits, ahead);
      });
}

extern "C" int kitty_f16kv_decode_shared(const kitty_cfg* cfg, const void* q, const void* pool,
                                         int32_t pool_pages, const int32_t* prefix_table,
                                         int32_t n_prefix, const int32_t* prefix_pages,
                                         const int32_t* block_table, int32_t max_pages,
                                         const int32_t* ctx_len, float sm_scale, void* out,
                                         int32_t out_dtype, void* workspace, size_t workspace_bytes,
                                         int32_t B, int32_t* d_status, void* stream) {
  return shared_attention(
      cfg, false, q, pool, pool_pages, prefix_table, n_prefix, prefix_pages, max_pages, sm_scale, out,
      out_dtype, workspace, workspace_bytes, B, d_status, stream,
      [&](float* ws, size_t bytes, int* splits, const GridAhead* ahead) {
        return f16kv_partials(cfg, q, pool, pool_pages, block_table, max_pages, ctx_len, sm_scale, out,
                              out_dtype, ws, bytes, B, d_status, stream, splits, ahead);
      });
}
