// Decode attention of a batch whose sequences share a prefix (sm_103a).
//
//   out[b][hq] = softmax(sm_scale * q . [K_prefix; K_b]) . [V_prefix; V_b]
//
// with the prefix's pages attended once for the whole batch and each sequence's own
// cache by the split-K decode.  Three launches: the decode kernel's partials over the
// own pages and tails, the prefix kernel's partials, and one merge of both.
#include "grid_dep.cuh"
#include "host_common.h"
#include "kitty_common.cuh"
#include "partials.h"

#include <algorithm>
#include <cmath>

namespace kitty {
namespace {

struct SharedParams {
  const uint16_t* q;
  const uint8_t* pool;
  const int32_t* table;         // [n_prefix] page ids
  const int32_t* prefix_pages;  // [B] or null: all share the whole prefix
  float* ws;                    // prefix partials [B * Hq][splits]
  int32_t* d_status;
  float sm_log2;
  int pool_pages, n_prefix, B, Hq, Hkv, g, splits, n_hi, blob, w, v, in_dtype, packed;
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Key and Value of token t, channel c of a packed page (kitty_page_bytes has the layout).
__device__ float packed_key(const uint8_t* blob, const BlobLayout& l, int w, int t, int c,
                            const int* row_of) {
  auto code = [&](const uint8_t* plane, int col, int cols) -> uint32_t {
    const int ks = col >> 4, half = (col >> 3) & 1, qq = (col >> 1) & 3, e = col & 1;
    const int lane = 4 * (t & 7) + qq, tau = t >> 3;
    const uint32_t* p = reinterpret_cast<const uint32_t*>(plane);
    const uint32_t x = w == 2 ? p[lane * (cols / 16) + ks] : p[lane * (cols / 8) + 2 * ks + (tau >> 1)];
    const int bit = 16 * e + 8 * half + (w == 2 ? 2 * tau : 4 * (tau & 1)) + 2;
    return __funnelshift_r(x, x, bit) & ((1u << w) - 1u);
  };
  const int j = c >> 4, h = (c >> 3) & 1, qq = (c >> 1) & 3, e = c & 1;
  const float S = __half2float(reinterpret_cast<const __half*>(blob + l.ks)[c]);
  const float M = __half2float(reinterpret_cast<const __half*>(blob + l.km)[((qq * 8 + j) * 2 + h) * 2 + e]);
  float k = M + S * (float)code(blob + l.kbase, c, kD);
  if (row_of[c] >= 0) k += S / (float)(1 << w) * (float)code(blob + l.kextra, row_of[c], l.n_hi);
  return k;
}

__device__ float packed_value(const uint8_t* blob, const BlobLayout& l, int v, int t, int c) {
  const int mc = c >> 4, rh = (c >> 3) & 1, r = c & 7;
  const int kt = t >> 4, half = (t >> 3) & 1, qq = (t >> 1) & 3, e = t & 1;
  const int lane = 4 * r + qq;
  const uint32_t* p = reinterpret_cast<const uint32_t*>(blob + l.vbase);
  const uint32_t x = v == 2 ? p[lane * 8 + (mc >> 1) * 2 + kt] : p[lane * 16 + (mc >> 1) * 4 + kt * 2 + (mc & 1)];
  const int bit = 16 * e + 8 * half + (v == 2 ? 2 * (2 * (mc & 1) + rh) : 4 * rh) + 2;
  const uint32_t code = __funnelshift_r(x, x, bit) & ((1u << v) - 1u);
  const int at = (c >> 5) * 32 + qq * 8 + kt * 4 + half * 2 + e;
  const float S = __half2float(reinterpret_cast<const __half*>(blob + l.vs)[at]);
  const float M = __half2float(reinterpret_cast<const __half*>(blob + l.vm)[at]);
  return M + S * (float)code;
}

// One block per (sequence and kv head, split): its pages one after the other into shared
// memory in fp32, then for each query head the page's 32 scores (four warps, eight
// tokens each), the running softmax and the product with the Values (a thread a channel).
__global__ void __launch_bounds__(128) prefix_kernel(const SharedParams p) {
  __shared__ float ks[kPage][kD], vs[kPage][kD];
  __shared__ float sc[kPage];
  __shared__ int row_of[kD];
  extern __shared__ float state[];  // per head: q[128], o[128], then m and l
  grid_trigger();
  const int b = blockIdx.x / p.Hkv, kvh = blockIdx.x % p.Hkv, s = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  float* qs = state;
  float* os = state + p.g * kD;
  float* ml = os + p.g * kD;
  int n = p.prefix_pages != nullptr ? p.prefix_pages[b] : p.n_prefix;
  if (n < 0 || n > p.n_prefix) {
    if (tid == 0 && s == 0 && kvh == 0) set_status(p.d_status, KITTY_ST_BAD_LEN);
    n = 0;
  }
  for (int h = 0; h < p.g; ++h) {
    qs[h * kD + tid] = bits16_to_f32(p.q[((size_t)b * p.Hq + kvh * p.g + h) * kD + tid], p.in_dtype);
    os[h * kD + tid] = 0.f;
    if (tid == 0) {
      ml[2 * h] = -INFINITY;
      ml[2 * h + 1] = 0.f;
    }
  }
  const int p0 = (int)((long)p.n_prefix * s / p.splits);
  const int p1 = min(n, (int)((long)p.n_prefix * (s + 1) / p.splits));
  const BlobLayout lay(p.n_hi, p.w, p.v);
  for (int i = p0; i < p1; ++i) {
    const int id = p.table[i];
    if (id < 0 || id >= p.pool_pages) {
      if (tid == 0) set_status(p.d_status, KITTY_ST_BAD_PAGE);
      continue;
    }
    __syncthreads();
    const uint8_t* blob = p.pool + ((size_t)id * p.Hkv + kvh) * p.blob;
    if (p.packed) {
      row_of[tid] = -1;
      __syncthreads();
      if (tid < p.n_hi) {
        const int js = tid >> 4, h = (tid >> 3) & 1, qq = (tid >> 1) & 3, e = tid & 1;
        row_of[blob[lay.kch + js * 16 + qq * 4 + h * 2 + e] & 127] = tid;
      }
      __syncthreads();
      const float S = __half2float(reinterpret_cast<const __half*>(blob + lay.ks)[tid]);
      const float Sv = __half2float(reinterpret_cast<const __half*>(blob + lay.vs)[tid]);
      if (S * (float)(1 << p.w) > 65504.f || Sv * (float)(1 << p.v) > 65504.f) set_status(p.d_status, KITTY_ST_RANGE);
      for (int t = 0; t < kPage; ++t) {
        ks[t][tid] = packed_key(blob, lay, p.w, t, tid, row_of);
        vs[t][tid] = packed_value(blob, lay, p.v, t, tid);
      }
    } else {
      const uint16_t* x = reinterpret_cast<const uint16_t*>(blob);
      for (int t = 0; t < kPage; ++t) {
        ks[t][tid] = bits16_to_f32(x[t * kD + tid], p.in_dtype);
        vs[t][tid] = bits16_to_f32(x[(kPage + t) * kD + tid], p.in_dtype);
      }
    }
    __syncthreads();
    for (int h = 0; h < p.g; ++h) {
      for (int t = 8 * wid; t < 8 * wid + 8; ++t) {
        float d = 0.f;
        for (int c = lane; c < kD; c += 32) d = fmaf(qs[h * kD + c], ks[t][c], d);
        for (int x = 16; x > 0; x >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, x);
        if (lane == 0) sc[t] = d * p.sm_log2;
      }
      __syncthreads();
      float m = ml[2 * h], l = ml[2 * h + 1], mx = m;
      for (int t = 0; t < kPage; ++t) mx = fmaxf(mx, sc[t]);
      const float a = exp2_fast(m - mx);
      float o = os[h * kD + tid] * a;
      l *= a;
      for (int t = 0; t < kPage; ++t) {
        const float e = exp2_fast(sc[t] - mx);
        l += e;
        o = fmaf(e, vs[t][tid], o);
      }
      os[h * kD + tid] = o;
      __syncthreads();
      if (tid == 0) {
        ml[2 * h] = mx;
        ml[2 * h + 1] = l;
      }
    }
  }
  __syncthreads();
  for (int h = 0; h < p.g; ++h) {
    float* part = p.ws + (((size_t)b * p.Hq + kvh * p.g + h) * p.splits + s) * kPartialFloats;
    part[4 + tid] = os[h * kD + tid];
    if (tid == 0) {
      part[0] = ml[2 * h];
      part[1] = ml[2 * h + 1];
    }
  }
  grid_wait();  // the merge waits for this grid: so that it has waited for the one before, too
}

struct MergeParams {
  const float *a, *b;  // partials of the prefix and of the own pages, row-major
  void* out;
  int32_t* d_status;
  int na, nb, rows, out_dtype;
};

// One warp a row: the partials of both lists in order, four channels a lane.
__global__ void __launch_bounds__(128) merge_kernel(const MergeParams p) {
  grid_wait();
  const int row = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= p.rows) return;
  const float* a = p.a + (size_t)row * p.na * kPartialFloats;
  const float* b = p.b + (size_t)row * p.nb * kPartialFloats;
  float ms = -INFINITY;
  for (int s = 0; s < p.na; ++s) ms = fmaxf(ms, a[s * kPartialFloats]);
  for (int s = 0; s < p.nb; ++s) ms = fmaxf(ms, b[s * kPartialFloats]);
  float L = 0.f;
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
  if (ms != -INFINITY) {
    for (int s = 0; s < p.na + p.nb; ++s) {
      const float* x = s < p.na ? a + s * kPartialFloats : b + (s - p.na) * kPartialFloats;
      if (x[0] == -INFINITY) continue;
      const float e = exp2_fast(x[0] - ms);
      const float4 o = reinterpret_cast<const float4*>(x + 4)[lane];
      L += x[1] * e;
      O.x += o.x * e;
      O.y += o.y * e;
      O.z += o.z * e;
      O.w += o.w * e;
    }
  }
  const bool ok = L > 0.f;
  if (!ok && lane == 0) set_status(p.d_status, KITTY_ST_EMPTY);
  const float r[4] = {ok ? O.x / L : 0.f, ok ? O.y / L : 0.f, ok ? O.z / L : 0.f, ok ? O.w / L : 0.f};
  const size_t i = (size_t)row * kD + 4 * lane;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (p.out_dtype == KITTY_F32) static_cast<float*>(p.out)[i + k] = r[k];
    else if (p.out_dtype == KITTY_BF16) static_cast<__nv_bfloat16*>(p.out)[i + k] = __float2bfloat16_rn(r[k]);
    else static_cast<__half*>(p.out)[i + k] = __float2half_rn(r[k]);
  }
}

int plan_splits(const kitty_cfg* cfg, int B, int n_prefix) {
  if (n_prefix == 0) return 0;
  const int units = B * cfg->num_kv_heads;
  return std::max(1, std::min({n_prefix, 16, (8 * sm_count() + units - 1) / units}));
}

size_t prefix_bytes(const kitty_cfg* cfg, int B, int n_prefix) {
  return (size_t)B * cfg->num_q_heads * plan_splits(cfg, B, n_prefix) * kPartialFloats * sizeof(float);
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
  *bytes = B == 0 ? 0
                  : prefix_bytes(cfg, B, n_prefix) + (packed ? decode_partial_bytes(cfg, B, max_pages)
                                                             : f16kv_partial_bytes(cfg, B, max_pages));
  return KITTY_OK;
}

// Checks, the own pages' partials (`own` launches them behind the prefix's in the
// workspace), the prefix kernel and the merge.
template <class Own>
int shared_attention(const kitty_cfg* cfg, bool packed, const void* q, const void* pool,
                     int32_t pool_pages, const int32_t* prefix_table, int32_t n_prefix,
                     const int32_t* prefix_pages, int32_t max_pages, float sm_scale, void* out,
                     int32_t out_dtype, void* ws, size_t ws_bytes, int32_t B, int32_t* d_status,
                     void* stream, Own own) {
  size_t need = 0;
  int rc = workspace(cfg, packed, B, n_prefix, max_pages, &need);
  if (rc != KITTY_OK) return rc;
  if (n_prefix > 0 && (!prefix_table || !pool || !aligned16(pool))) return KITTY_ERR_INVALID_ARG;
  if (B == 0) return KITTY_OK;
  if (q && !aligned16(q)) return KITTY_ERR_INVALID_ARG;
  if (ws_bytes < need || !ws || !aligned16(ws)) return KITTY_ERR_WORKSPACE;
  SharedParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.pool = static_cast<const uint8_t*>(pool);
  p.table = prefix_table;
  p.prefix_pages = prefix_pages;
  p.ws = static_cast<float*>(ws);
  p.d_status = d_status;
  p.sm_log2 = sm_scale * 1.4426950408889634f;
  p.pool_pages = pool_pages;
  p.n_prefix = n_prefix;
  p.B = B;
  p.Hq = cfg->num_q_heads;
  p.Hkv = cfg->num_kv_heads;
  p.g = p.Hq / p.Hkv;
  p.splits = plan_splits(cfg, B, n_prefix);
  p.n_hi = cfg->n_hi;
  p.w = cfg->lo_bit;
  p.v = v_bits(cfg);
  p.packed = packed;
  p.blob = packed ? (int)blob_bytes(cfg->n_hi, p.w, p.v) : 2 * kPage * kD * 2;
  p.in_dtype = cfg->in_dtype;
  const size_t mine = prefix_bytes(cfg, B, n_prefix);
  float* own_ws = p.ws + mine / sizeof(float);
  MergeParams m = {p.ws, own_ws, out, d_status, p.splits, 0, B * p.Hq, out_dtype};
  rc = own(own_ws, ws_bytes - mine, &m.nb);
  if (rc != KITTY_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  e = cudaFuncSetAttribute(prefix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 40 << 10);
  if (e == cudaSuccess && p.splits > 0)
    e = launch_dependent(prefix_kernel, dim3((unsigned)B * p.Hkv, p.splits), 128,
                         (size_t)p.g * (2 * kD + 2) * sizeof(float), s, p);
  if (e == cudaSuccess)
    e = launch_dependent(merge_kernel, dim3((unsigned)((m.rows + 3) / 4)), 128, 0, s, m);
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
      [&](float* ws, size_t bytes, int* splits) {
        return decode_partials(cfg, q, pool, pool_pages, block_table, max_pages, num_pages, tail_k,
                               tail_v, tail_len, sm_scale, out, out_dtype, ws, bytes, B, d_status,
                               stream, splits);
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
      [&](float* ws, size_t bytes, int* splits) {
        return f16kv_partials(cfg, q, pool, pool_pages, block_table, max_pages, ctx_len, sm_scale, out,
                              out_dtype, ws, bytes, B, d_status, stream, splits);
      });
}
