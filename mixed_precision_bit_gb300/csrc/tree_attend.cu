// Attention of drafted tokens over a sequence's cache and over each other (sm_103a).
//
//   out[t][hq] = softmax(sm_scale * q . [K_prefix; K_b; K_tree]) . [V_prefix; V_b; V_tree]
//
// One block per (drafted token, kv head): every page is dequantized to fp32 in shared memory, a
// warp takes a head's 32 scores, a thread a channel of the outputs.
#include "grid_dep.cuh"
#include "host_common.h"
#include "kitty_common.cuh"

#include <cmath>

namespace kitty {
namespace {

constexpr int kMaxNodes = KITTY_TREE_MAX_NODES;

struct TreeParams {
  const uint16_t *q, *k, *v;
  size_t q_stride, k_stride, v_stride;
  const int32_t* seq_start;
  const unsigned long long* visible;
  const uint8_t* pool;
  const int32_t *prefix_table, *prefix_pages, *block_table;
  const int32_t *num_pages, *tail_len;  // packed cache
  const uint16_t *tail_k, *tail_v;
  const int32_t* ctx_len;  // 16-bit cache
  void* out;
  int32_t* d_status;
  float sm_log2;
  int n_tokens, max_nodes, pool_pages, n_prefix, max_pages, B, Hq, Hkv, g, n_hi, blob, in_dtype, out_dtype;
};

__device__ __forceinline__ void store_o(void* out, int dt, size_t i, float v) {
  if (dt == KITTY_F32) static_cast<float*>(out)[i] = v;
  else if (dt == KITTY_BF16) static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(out)[i] = __float2half_rn(v);
}

__device__ __forceinline__ uint32_t code_at(const uint8_t* plane, int word, int bit, uint32_t mask) {
  const uint32_t w = reinterpret_cast<const uint32_t*>(plane)[word];
  return __funnelshift_r(w, w, bit & 31) & mask;
}

// A page of a kv head in fp32: thread = channel.
template <int W, int V>
__device__ void unpack_page(const uint8_t* blob, int n_hi, float (*K)[kD + 1], float (*Vs)[kD + 1], int8_t* rank) {
  const BlobLayout lay(n_hi, W, V);
  const int c = threadIdx.x, j = c >> 4, h = (c >> 3) & 1, qq = (c & 7) >> 1, e = c & 1;
  rank[c] = -1;
  __syncthreads();
  if (c < n_hi) rank[blob[lay.kch + (c >> 4) * 16 + ((c & 7) >> 1) * 4 + ((c >> 3) & 1) * 2 + (c & 1)] & 127] = (int8_t)c;
  __syncthreads();
  const int x = rank[c];
  auto half_at = [&](int at, int i) { return __half2float(reinterpret_cast<const __half*>(blob + at)[i]); };
  const float S = half_at(lay.ks, c), M = half_at(lay.km, ((qq * 8 + j) * 2 + h) * 2 + e);
  auto key_code = [&](const uint8_t* plane, int col, int cols, int t) {
    const int lane = 4 * (t & 7) + ((col & 7) >> 1), bit = 16 * (col & 1) + 8 * ((col >> 3) & 1);
    return W == 2 ? code_at(plane, lane * (cols / 16) + (col >> 4), bit + 2 * (t >> 3) + 2, 3u)
                  : code_at(plane, lane * 2 * (cols / 16) + 2 * (col >> 4) + (t >> 4), bit + 4 * ((t >> 3) & 1) + 2, 15u);
  };
  for (int t = 0; t < kPage; ++t) {
    float code = (float)key_code(blob + lay.kbase, c, kD, t);
    if (x >= 0) code += (float)key_code(blob + lay.kextra, x, n_hi, t) * (1.0f / (1 << W));
    K[t][c] = fmaf(S, code, M);
    const int G = c >> 5, at = G * 32 + ((t >> 1) & 3) * 8 + (t >> 4) * 4 + ((t >> 3) & 1) * 2 + (t & 1);
    const int lane = 4 * (c & 7) + ((t & 7) >> 1), bit = 16 * (t & 1) + 8 * ((t >> 3) & 1);
    const uint32_t vc = V == 2 ? code_at(blob + lay.vbase, lane * 8 + G * 2 + (t >> 4), bit + 2 * (2 * ((c >> 4) & 1) + ((c >> 3) & 1)) + 2, 3u)
                               : code_at(blob + lay.vbase, lane * 16 + G * 4 + (t >> 4) * 2 + ((c >> 4) & 1), bit + 4 * ((c >> 3) & 1) + 2, 15u);
    Vs[t][c] = fmaf(half_at(lay.vs, at), (float)vc, half_at(lay.vm, at));
  }
}

// What this row's sequence holds: its prefix pages, own pages, and tokens in the last of them (packed:
// in the tail).
struct Held {
  int prefix, pages, last;
};

template <bool PACKED, int W, int V>
__global__ void __launch_bounds__(128) tree_simple_kernel(const TreeParams p) {
  __shared__ float K[kPage][kD + 1], Vs[kPage][kD + 1];
  __shared__ uint16_t q[32][kD];
  __shared__ float prob[32][kPage];
  __shared__ float ms[32], ls[32], fs[32];
  __shared__ int8_t rank[kD];
  const int t = blockIdx.x, kvh = blockIdx.y, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  int lo = 0, hi = p.B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (p.seq_start[mid + 1] <= t) lo = mid + 1;
    else hi = mid;
  }
  const int b = lo;
  if (b >= p.B) return;
  const int first = p.seq_start[b], end = p.seq_start[b + 1], n = end - first, node = t - first;
  if (first < 0 || node < 0 || end > p.n_tokens) {
    if (tid == 0) set_status(p.d_status, KITTY_ST_BAD_SEQ);
    return;
  }
  Held held = {p.n_prefix, 0, 0};
  if (p.n_prefix > 0 && p.prefix_pages != nullptr) held.prefix = p.prefix_pages[b];
  bool bad = n > p.max_nodes;
  if (held.prefix < 0 || held.prefix > p.n_prefix) {
    if (tid == 0) set_status(p.d_status, KITTY_ST_BAD_LEN);
    held.prefix = 0;
  }
  if (PACKED) {
    held.pages = p.num_pages[b];
    held.last = p.tail_len[b];
    if (held.pages < 0 || held.pages > p.max_pages || held.last < 0 || held.last > kPage) bad = true;
  } else {
    const int len = p.ctx_len[b];
    if (len < 0 || len > p.max_pages * kPage) bad = true;
    held.pages = (len + kPage - 1) / kPage;
    held.last = len - (held.pages - 1) * kPage;
  }
  if (bad) {
    if (tid == 0) set_status(p.d_status, KITTY_ST_BAD_LEN);
    return;
  }
  const unsigned long long all = n == 64 ? ~0ull : (1ull << n) - 1;
  const unsigned long long sees = (p.visible != nullptr ? p.visible[t] : (node == 63 ? ~0ull : (2ull << node) - 1)) & all;
  bool range = false, finite = true;
  auto take = [&](uint16_t bits) {
    const float x = bits16_to_f32(bits, p.in_dtype);
    finite = finite && fabsf(x) <= 3.4028235e38f;
    range = range || (PACKED && fabsf(x) > 65504.f);
    return x;
  };
  for (int h = 0; h < p.g; ++h) take(q[h][tid] = p.q[(size_t)t * p.q_stride + ((size_t)kvh * p.g + h) * kD + tid]);
  if (tid < 32) {
    ms[tid] = -INFINITY;
    ls[tid] = 0.f;
  }
  float O[32];
#pragma unroll
  for (int h = 0; h < 32; ++h) O[h] = 0.f;
  // one tile of up to 32 tokens, in K and Vs; bit i of `mask`: token i is seen
  auto attend = [&](uint32_t mask) {
    __syncthreads();
    for (int h = w; h < p.g; h += 4) {
      float s = 0.f;
      for (int c = 0; c < kD; ++c) s = fmaf(bits16_to_f32(q[h][c], p.in_dtype), K[lane][c], s);
      s = (mask >> lane) & 1u ? s * p.sm_log2 : -INFINITY;
      float m = s;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
      m = fmaxf(m, ms[h]);
      const float e = m == -INFINITY || s == -INFINITY ? 0.f : exp2f(s - m);
      const float f = ms[h] == -INFINITY ? 0.f : exp2f(ms[h] - m);
      float l = e;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
      prob[h][lane] = e;
      __syncwarp();
      if (lane == 0) {
        ls[h] = ls[h] * f + l;
        ms[h] = m;
        fs[h] = f;
      }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 32; ++h) {
      if (h >= p.g) break;
      float o = O[h] * fs[h];
      for (int i = 0; i < kPage; ++i)
        if ((mask >> i) & 1u) o = fmaf(prob[h][i], Vs[i][tid], o);
      O[h] = o;
    }
    __syncthreads();
  };
  const size_t blob16 = (size_t)2 * kPage * kD;
  for (int x = 0; x < held.prefix + held.pages; ++x) {
    const bool own = x >= held.prefix;
    const int id = own ? p.block_table[(size_t)b * p.max_pages + x - held.prefix] : p.prefix_table[x];
    if (id < 0 || id >= p.pool_pages) {
      if (tid == 0) set_status(p.d_status, KITTY_ST_BAD_PAGE);
      continue;
    }
    uint32_t mask = 0xFFFFFFFFu;
    if (PACKED) {
      unpack_page<W, V>(p.pool + ((size_t)id * p.Hkv + kvh) * p.blob, p.n_hi, K, Vs, rank);
    } else {
      const int rows = own && x == held.prefix + held.pages - 1 ? held.last : kPage;
      if (rows < kPage) mask = (1u << rows) - 1;
      const uint16_t* blob = reinterpret_cast<const uint16_t*>(p.pool) + ((size_t)id * p.Hkv + kvh) * blob16;
      for (int i = 0; i < rows; ++i) {
        K[i][tid] = bits16_to_f32(blob[i * kD + tid], p.in_dtype);
        Vs[i][tid] = bits16_to_f32(blob[(kPage + i) * kD + tid], p.in_dtype);
      }
    }
    attend(mask);
  }
  if (PACKED && held.last > 0) {
    const size_t at = ((size_t)b * p.Hkv + kvh) * kPage * kD + tid;
    for (int i = 0; i < held.last; ++i) {
      K[i][tid] = take(p.tail_k[at + i * kD]);
      Vs[i][tid] = take(p.tail_v[at + i * kD]);
    }
    attend(held.last == kPage ? 0xFFFFFFFFu : (1u << held.last) - 1);
  }
  for (int j0 = 0; j0 < n; j0 += kPage) {
    const uint32_t mask = (uint32_t)(sees >> j0);
    for (int i = 0; i < kPage; ++i) {
      if (!((mask >> i) & 1u)) continue;
      const size_t row = (size_t)first + j0 + i;
      K[i][tid] = take(p.k[row * p.k_stride + (size_t)kvh * kD + tid]);
      Vs[i][tid] = take(p.v[row * p.v_stride + (size_t)kvh * kD + tid]);
    }
    if (mask != 0) attend(mask);
  }
  if (!finite) set_status(p.d_status, KITTY_ST_NONFINITE);
  else if (range) set_status(p.d_status, KITTY_ST_RANGE);
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 32; ++h) {
    if (h >= p.g) break;
    const float L = ls[h];
    store_o(p.out, p.out_dtype, ((size_t)t * p.Hq + (size_t)kvh * p.g + h) * kD + tid, L != 0.f ? O[h] / L : 0.f);
    if (L == 0.f && tid == 0) set_status(p.d_status, KITTY_ST_EMPTY);
  }
}

bool rows_ok(const void* p, int64_t stride, int heads) {
  return p != nullptr && aligned16(p) && stride >= (int64_t)heads * kD && stride % 8 == 0;
}

int check_tree(const kitty_cfg* cfg, int B, int n_tokens, int max_nodes, int n_prefix, int max_pages) {
  const int rc = check_cfg(cfg, 32);
  if (rc != KITTY_OK) return rc;
  if (B < 0 || n_tokens < 0 || n_prefix < 0 || max_pages < 0 || max_nodes < 1) return KITTY_ERR_INVALID_ARG;
  return max_nodes > kMaxNodes ? KITTY_ERR_UNSUPPORTED : KITTY_OK;
}

int workspace(const kitty_cfg* cfg, int B, int n_tokens, int max_nodes, int n_prefix, int max_pages, size_t* bytes) {
  const int rc = check_tree(cfg, B, n_tokens, max_nodes, n_prefix, max_pages);
  if (rc != KITTY_OK) return rc;
  if (!bytes) return KITTY_ERR_INVALID_ARG;
  *bytes = 0;
  return KITTY_OK;
}

// Checks of what both caches' calls share, and their part of p; 1: nothing to do.
int tree_params(const kitty_cfg* cfg, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                const void* v, int64_t v_stride, int32_t n_tokens, const int32_t* seq_start,
                const uint64_t* visible, int32_t max_nodes, const void* pool, int32_t pool_pages,
                const int32_t* prefix_table, int32_t n_prefix, const int32_t* prefix_pages,
                const int32_t* block_table, int32_t max_pages, float sm_scale, void* out, int32_t out_dtype,
                int32_t B, int32_t* d_status, TreeParams* p) {
  const int rc = check_tree(cfg, B, n_tokens, max_nodes, n_prefix, max_pages);
  if (rc != KITTY_OK) return rc;
  if (pool_pages < 0 || (out_dtype != KITTY_F32 && out_dtype != KITTY_BF16 && out_dtype != KITTY_F16))
    return KITTY_ERR_INVALID_ARG;
  if (B == 0 || n_tokens == 0) return 1;
  const int Hq = cfg->num_q_heads, Hkv = cfg->num_kv_heads;
  if (Hkv > 65535) return KITTY_ERR_UNSUPPORTED;
  if (!rows_ok(q, q_stride, Hq) || !rows_ok(k, k_stride, Hkv) || !rows_ok(v, v_stride, Hkv) || !seq_start ||
      (reinterpret_cast<uintptr_t>(visible) & 7u) != 0 || !out || !aligned16(out) || !std::isfinite(sm_scale) ||
      (max_pages > 0 && (!block_table || !pool)) || (n_prefix > 0 && (!prefix_table || !pool)) ||
      (pool && !aligned16(pool)))
    return KITTY_ERR_INVALID_ARG;
  p->q = static_cast<const uint16_t*>(q);
  p->k = static_cast<const uint16_t*>(k);
  p->v = static_cast<const uint16_t*>(v);
  p->q_stride = (size_t)q_stride;
  p->k_stride = (size_t)k_stride;
  p->v_stride = (size_t)v_stride;
  p->seq_start = seq_start;
  p->visible = reinterpret_cast<const unsigned long long*>(visible);
  p->pool = static_cast<const uint8_t*>(pool);
  p->prefix_table = prefix_table;
  p->prefix_pages = prefix_pages;
  p->block_table = block_table;
  p->out = out;
  p->d_status = d_status;
  p->sm_log2 = sm_scale * 1.4426950408889634f;
  p->n_tokens = n_tokens;
  p->max_nodes = max_nodes;
  p->pool_pages = pool_pages;
  p->n_prefix = n_prefix;
  p->max_pages = max_pages;
  p->B = B;
  p->Hq = Hq;
  p->Hkv = Hkv;
  p->g = Hq / Hkv;
  p->n_hi = cfg->n_hi;
  p->blob = (int)blob_bytes(cfg->n_hi, cfg->lo_bit, v_bits(cfg));
  p->in_dtype = cfg->in_dtype;
  p->out_dtype = out_dtype;
  return KITTY_OK;
}

template <class Kernel>
int launch(Kernel kernel, const TreeParams& p, cudaStream_t s) {
  kernel<<<dim3((unsigned)p.n_tokens, (unsigned)p.Hkv), 128, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? KITTY_OK : KITTY_ERR_CUDA;
}

}  // namespace
}  // namespace kitty

using namespace kitty;

extern "C" int kitty_tree_workspace_bytes(const kitty_cfg* cfg, int32_t B, int32_t n_tokens, int32_t max_nodes,
                                          int32_t n_prefix, int32_t max_pages, size_t* bytes) {
  return workspace(cfg, B, n_tokens, max_nodes, n_prefix, max_pages, bytes);
}

extern "C" int kitty_f16kv_tree_workspace_bytes(const kitty_cfg* cfg, int32_t B, int32_t n_tokens,
                                                int32_t max_nodes, int32_t n_prefix, int32_t max_pages,
                                                size_t* bytes) {
  return workspace(cfg, B, n_tokens, max_nodes, n_prefix, max_pages, bytes);
}

extern "C" int kitty_tree_attention(const kitty_cfg* cfg, const void* q, int64_t q_stride, const void* k,
                                    int64_t k_stride, const void* v, int64_t v_stride, int32_t n_tokens,
                                    const int32_t* seq_start, const uint64_t* visible, int32_t max_nodes,
                                    const void* pool, int32_t pool_pages, const int32_t* prefix_table,
                                    int32_t n_prefix, const int32_t* prefix_pages, const int32_t* block_table,
                                    int32_t max_pages, const int32_t* num_pages, const void* tail_k,
                                    const void* tail_v, const int32_t* tail_len, float sm_scale, void* out,
                                    int32_t out_dtype, void* workspace, size_t workspace_bytes, int32_t B,
                                    int32_t* d_status, void* stream) {
  TreeParams p = {};
  const int rc = tree_params(cfg, q, q_stride, k, k_stride, v, v_stride, n_tokens, seq_start, visible, max_nodes,
                             pool, pool_pages, prefix_table, n_prefix, prefix_pages, block_table, max_pages,
                             sm_scale, out, out_dtype, B, d_status, &p);
  if (rc != KITTY_OK) return rc == 1 ? KITTY_OK : rc;
  if (!num_pages || !tail_len || !tail_k || !tail_v || !aligned16(tail_k) || !aligned16(tail_v))
    return KITTY_ERR_INVALID_ARG;
  p.num_pages = num_pages;
  p.tail_len = tail_len;
  p.tail_k = static_cast<const uint16_t*>(tail_k);
  p.tail_v = static_cast<const uint16_t*>(tail_v);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cfg->lo_bit == 2) return launch(tree_simple_kernel<true, 2, 2>, p, s);
  return v_bits(cfg) == 2 ? launch(tree_simple_kernel<true, 4, 2>, p, s) : launch(tree_simple_kernel<true, 4, 4>, p, s);
}

extern "C" int kitty_f16kv_tree_attention(const kitty_cfg* cfg, const void* q, int64_t q_stride, const void* k,
                                          int64_t k_stride, const void* v, int64_t v_stride, int32_t n_tokens,
                                          const int32_t* seq_start, const uint64_t* visible, int32_t max_nodes,
                                          const void* pool, int32_t pool_pages, const int32_t* prefix_table,
                                          int32_t n_prefix, const int32_t* prefix_pages,
                                          const int32_t* block_table, int32_t max_pages, const int32_t* ctx_len,
                                          float sm_scale, void* out, int32_t out_dtype, void* workspace,
                                          size_t workspace_bytes, int32_t B, int32_t* d_status, void* stream) {
  TreeParams p = {};
  const int rc = tree_params(cfg, q, q_stride, k, k_stride, v, v_stride, n_tokens, seq_start, visible, max_nodes,
                             pool, pool_pages, prefix_table, n_prefix, prefix_pages, block_table, max_pages,
                             sm_scale, out, out_dtype, B, d_status, &p);
  if (rc != KITTY_OK) return rc == 1 ? KITTY_OK : rc;
  if (!ctx_len) return KITTY_ERR_INVALID_ARG;
  p.ctx_len = ctx_len;
  return launch(tree_simple_kernel<false, 2, 2>, p, static_cast<cudaStream_t>(stream));
}
