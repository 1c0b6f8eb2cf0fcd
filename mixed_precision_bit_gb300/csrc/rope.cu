// Positions for the caches: per-head RMS norm and rotation of queries and keys as a
// pass of its own (before quantize_pages, a prefill or a fused step), and on the way
// into the packed cache's tails or the 16-bit cache's pages.
//
// What bounds them.  Every row is read once and written once: bytes, with many heads a token
// (4095 tokens of 72 half-rotated rows without a norm 25.0 us, 89% of the copy rate).  With fewer heads the
// issue of instructions comes near it (8192 tokens of 40 rows 32.6 us, 76%; 73 to 76% of issue
// slots): a token's sines, computed once, by one thread a pair, and shared by its heads
// through shared memory, and per row the norm's sum (four shuffles over 16 lanes), the
// rotation (both channels of a pair in one lane, two pairs an instruction) and the
// conversions.  A few tokens take one launch's latency, 2.5 to 5 us.  One block takes a token,
// so that nothing but its own position stands between its loads and its sines.
#include "rope.cuh"
#include "grid_dep.cuh"
#include "host_common.h"
#include "quant_tile.cuh"

#include <cmath>

namespace kitty {
namespace {

// A token's block: many tokens take 64 threads with five rows a 16-lane group in flight (40
// query and key rows in two rounds, 16 blocks an SM), few tokens 256 threads with three (48
// rows in one round: the shortest block).  Measured, us: 8192 tokens of 40 rows 32.9 against 48.6
// (128 threads: 35.0 to 39.1), 64 tokens 4.9 against 3.2; 8180 appended tokens of 48 rows 43.8
// against 58.8, 64 tokens 7.7 against 4.5 (before the arithmetic took two pairs at a time:
// now 32.6, 2.6, 42.0 and 4.0 as chosen).
struct ManyTokens {
  static constexpr int kThreads = 64, kAhead = 5, kBlocks = 16;
};
struct FewTokens {
  static constexpr int kThreads = 256, kAhead = 3, kBlocks = 3;
};
// Many: more tokens than two large blocks an SM.
inline bool many_tokens(int n) { return n > 2 * sm_count(); }

// Queries and keys of token blockIdx.x, out of place or in place (a lane writes only
// the channels that it read).
template <int DT, class B>
__global__ void __launch_bounds__(B::kThreads, B::kBlocks) norm_rope_kernel(
    const RopeParams p, const uint16_t* q, size_t q_stride, const uint16_t* k, size_t k_stride,
    const int32_t* positions, uint16_t* qo, size_t qo_stride, uint16_t* ko, size_t ko_stride,
    int H1, int H2) {
  __shared__ float2 cs[kD / 2];
  const size_t t = blockIdx.x;
  TokenRows rows = {q + t * q_stride, k + t * k_stride, nullptr, qo + t * qo_stride,
                    ko + t * ko_stride, nullptr, kD, H1, H2};
  RopeLane L = rope_lane(p);
  uint4 x[B::kAhead];
  rope_load<B::kThreads>(rows, L, 0, x);
  rope_angles(p, positions[t], cs);
  __syncthreads();
  rope_token<DT, B::kThreads>(p, L, cs, rows, x);
}

// The 16-bit page blob of one (page, kv head): K [32][128] then V [32][128].
constexpr size_t kBlob16 = (size_t)2 * kPage * kD;  // in 16-bit elements

struct Append16 {
  RopeParams rope;
  const uint16_t *q, *k, *v;
  size_t q_stride, k_stride, v_stride, qo_stride;
  uint16_t* qo;  // null: no queries
  uint16_t* pool;
  int32_t* block_table;
  int32_t* ctx_len;
  const int32_t* new_page_ids;
  const int32_t* seq_start;  // null: one token a sequence
  const int32_t* pos_base;
  int32_t* d_status;
  int pool_pages, max_pages, B, Hq, Hkv, counted;
};

// A sequence's length before its n new tokens, or -1 (reported) when it cannot take them.
__device__ __forceinline__ int length_before(const Append16& p, int b, int n, bool report) {
  const int have = p.ctx_len[b];
  const long before = p.counted ? (long)have - n : have;
  const long room = (long)p.max_pages * kPage;
  if (before < 0 || before + n > room) {
    if (report) set_status(p.d_status, before < 0 || before > room ? KITTY_ST_BAD_LEN : KITTY_ST_TABLE_FULL);
    return -1;
  }
  return (int)before;
}

// Token blockIdx.x.  The new tokens' own page ids come from new_page_ids (entry of the
// token that begins the page), so no block depends on another's block-table write.
template <int DT, class B>
__global__ void __launch_bounds__(B::kThreads, B::kBlocks) f16kv_append_rope_kernel(const Append16 p) {
  __shared__ float2 cs[kD / 2];
  grid_trigger();
  const int t = blockIdx.x;
  TokenRows rows = {p.q + (size_t)t * p.q_stride, p.k + (size_t)t * p.k_stride,
                    p.v + (size_t)t * p.v_stride, p.qo + (size_t)t * p.qo_stride, nullptr, nullptr,
                    kBlob16, p.qo != nullptr ? p.Hq : 0, p.Hkv};
  RopeLane L = rope_lane(p.rope);
  uint4 x[B::kAhead];
  rope_load<B::kThreads>(rows, L, 0, x);
  int b = t, first = t, n = 1;
  if (p.seq_start != nullptr) {
    // b = sequences that end at or before token t: one load a thread a round
    b = 0;
    for (int s0 = 0; s0 < p.B; s0 += B::kThreads) {
      const int s = s0 + threadIdx.x;
      b += __syncthreads_count(s < p.B && p.seq_start[s + 1] <= t);
    }
    if (b >= p.B) return;  // a row behind the last sequence
    first = p.seq_start[b];
    n = p.seq_start[b + 1] - first;
    if (first < 0 || t < first || t - first >= n || p.seq_start[b + 1] > (int)gridDim.x) {  // out of order
      if (threadIdx.x == 0) set_status(p.d_status, KITTY_ST_BAD_SEQ);
      return;
    }
  }
  const int i = t - first;
  const int before = length_before(p, b, n, threadIdx.x == 0);
  if (before < 0) return;
  const int pos = before + i, slot = pos % kPage, page = pos / kPage;
  const int id = !p.counted && slot <= i ? p.new_page_ids[t - slot]
                                         : p.block_table[(size_t)b * p.max_pages + page];
  if (id < 0 || id >= p.pool_pages) {
    if (threadIdx.x == 0) set_status(p.d_status, KITTY_ST_BAD_PAGE);
    return;
  }
  rope_angles(p.rope, (int64_t)pos + (p.pos_base != nullptr ? p.pos_base[b] : 0), cs);
  __syncthreads();  // the angles; and every thread has read the length
  rows.ko = p.pool + (size_t)id * p.Hkv * kBlob16 + (size_t)slot * kD;
  rows.vo = rows.ko + (size_t)kPage * kD;
  rope_token<DT, B::kThreads>(p.rope, L, cs, rows, x);
  if (p.seq_start == nullptr && !p.counted && threadIdx.x == 0) {
    // this block is all of the sequence's append
    if (slot == 0) p.block_table[(size_t)b * p.max_pages + page] = id;
    p.ctx_len[b] = pos + 1;
  }
}

// After a ragged append: one warp a sequence enters its new pages in the block table
// and, if every one of its tokens was its own and has a page, advances its length.
// A token goes to the sequence whose index is the number of ends at or before it; that
// number rises with the token, so a sequence's tokens are all its own if the first and
// the last are.  With starts out of order some are not: reported, not advanced.
__global__ void __launch_bounds__(128) f16kv_append_rope_finish(const Append16 p, int n_tokens) {
  grid_wait();
  const int b = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (b >= p.B) return;
  // all loads at once: what depends on the starts is arithmetic
  const int first = p.seq_start[b], end = p.seq_start[b + 1], n = end - first;
  const int e0 = lane < p.B ? p.seq_start[lane + 1] : 0;
  const int before = length_before(p, b, n, false);
  if (first == end) return;
  bool mine = first >= 0 && first < end && end <= n_tokens;
  if (mine) {
    int c0 = 0, c1 = 0;  // ends at or before the first and the last token
    for (int s = lane; s < p.B; s += 32) {
      const int e = s == lane ? e0 : p.seq_start[s + 1];
      c0 += e <= first;
      c1 += e < end;
    }
    mine = __reduce_add_sync(0xFFFFFFFFu, c0) == b && __reduce_add_sync(0xFFFFFFFFu, c1) == b;
  }
  if (!mine) {
    if (lane == 0) set_status(p.d_status, KITTY_ST_BAD_SEQ);
    return;
  }
  if (before < 0) return;
  bool ok = true;
  if (before % kPage != 0) {
    const int id = p.block_table[(size_t)b * p.max_pages + before / kPage];
    ok = id >= 0 && id < p.pool_pages;
  }
  for (int i = (kPage - before % kPage) % kPage + kPage * lane; i < n; i += kPage * 32) {
    const int id = p.new_page_ids[first + i];
    if (id >= 0 && id < p.pool_pages) p.block_table[(size_t)b * p.max_pages + (before + i) / kPage] = id;
    else ok = false;
  }
  if (__all_sync(0xFFFFFFFFu, ok) && lane == 0) p.ctx_len[b] = before + n;
}

struct AppendTail {
  RopeParams rope;
  const uint16_t *q, *k, *v;
  size_t q_stride, k_stride, v_stride, qo_stride;
  uint16_t* qo;
  uint16_t *tail_k, *tail_v;
  int32_t* tail_len;
  float *run_sum, *run_sumsq;
  int32_t* run_count;
  const int32_t* flush_page_ids;
  int32_t* block_table;
  int32_t* num_pages;
  const int32_t* pos_base;
  uint8_t* pool;
  int32_t* d_status;
  int pool_pages, max_pages, n_hi, Hq, Hkv, running, counted;
};

// One block per (sequence, kv head): its query rows, its key row and its value row,
// then, when the tail is full and a page id is given, the tail's quantization.  The
// rules are those of the append without rotation.
template <int DT, int W, int V>
__global__ void __launch_bounds__(kQThreads) append_rope_kernel(const AppendTail p) {
  __shared__ QuantSmem sm;
  __shared__ float2 cs[kD / 2];
  grid_trigger();
  const int b = blockIdx.x, h = blockIdx.y, c = threadIdx.x;
  const int g = p.Hq / p.Hkv;
  TokenRows rows = {p.q + (size_t)b * p.q_stride + (size_t)h * g * kD,
                    p.k + (size_t)b * p.k_stride + (size_t)h * kD,
                    p.v + (size_t)b * p.v_stride + (size_t)h * kD,
                    p.qo + (size_t)b * p.qo_stride + (size_t)h * g * kD, nullptr, nullptr, 0,
                    p.qo != nullptr ? g : 0, 1};
  RopeLane L = rope_lane(p.rope);
  uint4 x[2];  // 16 rows a round: a group of up to 14 query heads
  rope_load<kQThreads>(rows, L, 0, x);
  const int fid = p.flush_page_ids[b];
  int len = p.tail_len[b], np = p.num_pages[b];
  if (p.counted) {  // the lengths count the new token: undo that
    if (len == 0 && fid >= 0) {
      len = kPage;
      np -= 1;
    }
    len -= 1;
  }
  if (len < 0 || len > kPage || np < 0 || np > p.max_pages) {
    if (c == 0) set_status(p.d_status, KITTY_ST_BAD_LEN);
    return;
  }
  if (len == kPage) {
    if (c == 0) set_status(p.d_status, KITTY_ST_TAIL_FULL);
    return;
  }
  rope_angles(p.rope, (int64_t)np * kPage + len + (p.pos_base != nullptr ? p.pos_base[b] : 0), cs);
  __syncthreads();
  const size_t sh = (size_t)b * p.Hkv + h;
  rows.ko = p.tail_k + (sh * kPage + len) * kD;
  rows.vo = p.tail_v + (sh * kPage + len) * kD;
  rope_token<DT, kQThreads>(p.rope, L, cs, rows, x);
  const int n = len + 1;
  if (fid >= 0 && n < kPage) {
    if (c == 0) set_status(p.d_status, KITTY_ST_BAD_FLUSH);
    return;
  }
  if (n < kPage || fid < 0) return;
  if (np >= p.max_pages) {
    if (c == 0) set_status(p.d_status, KITTY_ST_TABLE_FULL);
    return;
  }
  if (fid >= p.pool_pages) {
    if (c == 0) set_status(p.d_status, KITTY_ST_BAD_PAGE);
    return;
  }
  __syncthreads();  // the new rows are visible to the whole block
  const BlobLayout lay(p.n_hi, W, V);
  float rs = 0.f, rq = 0.f;
  int rc = 0;
  if (p.running) {
    rs = p.run_sum[sh * kD + c];
    rq = p.run_sumsq[sh * kD + c];
    rc = p.run_count[sh];
  }
  quantize_tile<DT, W, V>(sm, p.tail_k + sh * kPage * kD, p.tail_v + sh * kPage * kD, kD, p.n_hi,
                          p.running != 0, rs, rq, rc,
                          p.pool + ((size_t)fid * p.Hkv + h) * lay.bytes, p.d_status);
  if (p.running) {
    p.run_sum[sh * kD + c] = rs;
    p.run_sumsq[sh * kD + c] = rq;
    if (c == 0) p.run_count[sh] = rc;
  }
}

// Lengths and block table, once every head of a sequence has used the old ones.
__global__ void __launch_bounds__(128) append_rope_finish(const AppendTail p, int B) {
  grid_wait();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= B) return;
  const int np = p.num_pages[b];
  if (np < 0 || np > p.max_pages) return;  // nothing was appended
  append_finalize_one(b, p.tail_len, p.flush_page_ids, p.block_table, p.max_pages, p.num_pages,
                      p.pool_pages);
}

int rope_params(const kitty_rope* r, RopeParams* p) {
  if (r == nullptr || r->rot_dim < 0 || r->rot_dim > kD ||
      (r->layout != KITTY_ROPE_HALF && r->layout != KITTY_ROPE_INTERLEAVED) ||
      !std::isfinite(r->amplitude) || !(r->eps >= 0.f) || !std::isfinite(r->eps) ||
      (r->rot_dim > 0 && (r->turns == nullptr || (reinterpret_cast<uintptr_t>(r->turns) & 7u) != 0)))
    return KITTY_ERR_INVALID_ARG;
  if (r->rot_dim % 16 != 0) return KITTY_ERR_UNSUPPORTED;
  p->turns = r->turns;
  p->q_weight = static_cast<const uint16_t*>(r->q_weight);
  p->k_weight = static_cast<const uint16_t*>(r->k_weight);
  p->amplitude = r->amplitude;
  p->eps = r->eps;
  p->rot = r->rot_dim;
  p->interleaved = r->layout == KITTY_ROPE_INTERLEAVED;
  return KITTY_OK;
}

// Rows [n][heads][128], `stride` elements from token to token, 16-byte accesses.
bool rows_ok(const void* p, int64_t stride, int heads) {
  return p != nullptr && aligned16(p) && stride >= (int64_t)heads * kD && stride % 8 == 0;
}

}  // namespace
}  // namespace kitty

using namespace kitty;

extern "C" int kitty_norm_rope(const kitty_cfg* cfg, const kitty_rope* rope, const void* q,
                               int64_t q_stride, const void* k, int64_t k_stride,
                               const int32_t* positions, int32_t n_tokens, void* q_out,
                               int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                               void* stream) {
  int rc = check_cfg(cfg);
  if (rc != KITTY_OK) return rc;
  RopeParams p = {};
  rc = rope_params(rope, &p);
  if (rc != KITTY_OK) return rc;
  const int Hq = cfg->num_q_heads, Hkv = cfg->num_kv_heads;
  if (n_tokens < 0) return KITTY_ERR_INVALID_ARG;
  if (n_tokens == 0) return KITTY_OK;
  if (!positions || (!q && !k) || (q && (!rows_ok(q, q_stride, Hq) || !rows_ok(q_out, q_out_stride, Hq))) ||
      (k && (!rows_ok(k, k_stride, Hkv) || !rows_ok(k_out, k_out_stride, Hkv))))
    return KITTY_ERR_INVALID_ARG;
  const bool many = many_tokens(n_tokens), bf = cfg->in_dtype == KITTY_BF16;
  auto launch = [&](auto kernel) {
    kernel<<<(unsigned)n_tokens, many ? ManyTokens::kThreads : FewTokens::kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        p, static_cast<const uint16_t*>(q), (size_t)q_stride, static_cast<const uint16_t*>(k),
        (size_t)k_stride, positions, static_cast<uint16_t*>(q_out), (size_t)q_out_stride,
        static_cast<uint16_t*>(k_out), (size_t)k_out_stride, q ? Hq : 0, k ? Hkv : 0);
  };
  if (many) bf ? launch(norm_rope_kernel<KITTY_BF16, ManyTokens>) : launch(norm_rope_kernel<KITTY_F16, ManyTokens>);
  else bf ? launch(norm_rope_kernel<KITTY_BF16, FewTokens>) : launch(norm_rope_kernel<KITTY_F16, FewTokens>);
  return cudaGetLastError() == cudaSuccess ? KITTY_OK : KITTY_ERR_CUDA;
}

extern "C" int kitty_f16kv_append_rope(const kitty_cfg* cfg, const kitty_rope* rope, const void* q,
                                       int64_t q_stride, const void* k_new, int64_t k_stride,
                                       const void* v_new, int64_t v_stride, int32_t n_tokens,
                                       void* q_out, int64_t q_out_stride, void* pool,
                                       int32_t pool_pages, int32_t* block_table, int32_t max_pages,
                                       int32_t* ctx_len, const int32_t* new_page_ids,
                                       const int32_t* seq_start, const int32_t* pos_base,
                                       int32_t counted, int32_t B, int32_t* d_status, void* stream) {
  int rc = check_cfg(cfg);
  if (rc != KITTY_OK) return rc;
  Append16 p = {};
  rc = rope_params(rope, &p.rope);
  if (rc != KITTY_OK) return rc;
  const int Hq = cfg->num_q_heads, Hkv = cfg->num_kv_heads;
  if (B < 0 || n_tokens < 0 || max_pages < 0 || pool_pages < 0 || (!seq_start && n_tokens != B))
    return KITTY_ERR_INVALID_ARG;
  if (B == 0 || n_tokens == 0) return KITTY_OK;
  if (!rows_ok(k_new, k_stride, Hkv) || !rows_ok(v_new, v_stride, Hkv) ||
      (q && (!rows_ok(q, q_stride, Hq) || !rows_ok(q_out, q_out_stride, Hq))) || !pool ||
      !aligned16(pool) || !block_table || !ctx_len || (!counted && !new_page_ids))
    return KITTY_ERR_INVALID_ARG;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k_new);
  p.v = static_cast<const uint16_t*>(v_new);
  p.q_stride = q ? (size_t)q_stride : 0;
  p.k_stride = (size_t)k_stride;
  p.v_stride = (size_t)v_stride;
  p.qo_stride = q ? (size_t)q_out_stride : 0;
  p.qo = q ? static_cast<uint16_t*>(q_out) : nullptr;
  p.pool = static_cast<uint16_t*>(pool);
  p.block_table = block_table;
  p.ctx_len = ctx_len;
  p.new_page_ids = new_page_ids;
  p.seq_start = seq_start;
  p.pos_base = pos_base;
  p.d_status = d_status;
  p.pool_pages = pool_pages;
  p.max_pages = max_pages;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.counted = counted != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool many = many_tokens(n_tokens), bf = cfg->in_dtype == KITTY_BF16;
  auto launch = [&](auto kernel) {
    kernel<<<(unsigned)n_tokens, many ? ManyTokens::kThreads : FewTokens::kThreads, 0, s>>>(p);
  };
  if (many) bf ? launch(f16kv_append_rope_kernel<KITTY_BF16, ManyTokens>) : launch(f16kv_append_rope_kernel<KITTY_F16, ManyTokens>);
  else bf ? launch(f16kv_append_rope_kernel<KITTY_BF16, FewTokens>) : launch(f16kv_append_rope_kernel<KITTY_F16, FewTokens>);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && seq_start && !counted)
    e = launch_dependent(f16kv_append_rope_finish, dim3((unsigned)((B + 3) / 4)), 128, 0, s, p, (int)n_tokens);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? KITTY_OK : KITTY_ERR_CUDA;
}

extern "C" int kitty_append_rope(const kitty_cfg* cfg, const kitty_rope* rope, const void* q,
                                 int64_t q_stride, const void* k_new, int64_t k_stride,
                                 const void* v_new, int64_t v_stride, void* q_out,
                                 int64_t q_out_stride, void* tail_k, void* tail_v,
                                 int32_t* tail_len, float* run_sum, float* run_sumsq,
                                 int32_t* run_count, const int32_t* flush_page_ids,
                                 int32_t* block_table, int32_t max_pages, int32_t* num_pages,
                                 void* pool, int32_t pool_pages, const int32_t* pos_base,
                                 int32_t counted, int32_t B, int32_t* d_status, void* stream) {
  int rc = check_cfg(cfg);
  if (rc != KITTY_OK) return rc;
  AppendTail p = {};
  rc = rope_params(rope, &p.rope);
  if (rc != KITTY_OK) return rc;
  const int Hq = cfg->num_q_heads, Hkv = cfg->num_kv_heads;
  if (B < 0 || max_pages < 0 || pool_pages < 0) return KITTY_ERR_INVALID_ARG;
  if (B == 0) return KITTY_OK;
  if (!rows_ok(k_new, k_stride, Hkv) || !rows_ok(v_new, v_stride, Hkv) ||
      (q && (!rows_ok(q, q_stride, Hq) || !rows_ok(q_out, q_out_stride, Hq))) || !tail_k ||
      !tail_v || !tail_len || !flush_page_ids || !block_table || !num_pages || !pool ||
      !aligned16(tail_k) || !aligned16(tail_v) || !aligned16(pool))
    return KITTY_ERR_INVALID_ARG;
  const bool running = cfg->rank_mode != KITTY_RANK_PAGE;  // sequence mode appends as running
  if (running && (!run_sum || !run_sumsq || !run_count)) return KITTY_ERR_INVALID_ARG;
  if (Hkv > 65535) return KITTY_ERR_UNSUPPORTED;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k_new);
  p.v = static_cast<const uint16_t*>(v_new);
  p.q_stride = q ? (size_t)q_stride : 0;
  p.k_stride = (size_t)k_stride;
  p.v_stride = (size_t)v_stride;
  p.qo_stride = q ? (size_t)q_out_stride : 0;
  p.qo = q ? static_cast<uint16_t*>(q_out) : nullptr;
  p.tail_k = static_cast<uint16_t*>(tail_k);
  p.tail_v = static_cast<uint16_t*>(tail_v);
  p.tail_len = tail_len;
  p.run_sum = run_sum;
  p.run_sumsq = run_sumsq;
  p.run_count = run_count;
  p.flush_page_ids = flush_page_ids;
  p.block_table = block_table;
  p.num_pages = num_pages;
  p.pos_base = pos_base;
  p.pool = static_cast<uint8_t*>(pool);
  p.d_status = d_status;
  p.pool_pages = pool_pages;
  p.max_pages = max_pages;
  p.n_hi = cfg->n_hi;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.running = running;
  p.counted = counted != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)B, (unsigned)Hkv);
  auto launch = [&](auto kernel) { kernel<<<grid, kQThreads, 0, s>>>(p); };
  const bool bf = cfg->in_dtype == KITTY_BF16;
  if (cfg->lo_bit == 2) bf ? launch(append_rope_kernel<KITTY_BF16, 2, 2>) : launch(append_rope_kernel<KITTY_F16, 2, 2>);
  else if (v_bits(cfg) == 2) bf ? launch(append_rope_kernel<KITTY_BF16, 4, 2>) : launch(append_rope_kernel<KITTY_F16, 4, 2>);
  else bf ? launch(append_rope_kernel<KITTY_BF16, 4, 4>) : launch(append_rope_kernel<KITTY_F16, 4, 4>);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && !counted)
    e = launch_dependent(append_rope_finish, dim3((unsigned)((B + 127) / 128)), 128, 0, s, p, (int)B);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? KITTY_OK : KITTY_ERR_CUDA;
}
