// A step of drafted tokens around the attention: ancestor masks and positions of trees, block
// tables and slot maps from lengths with the free pages on the device, and the accepted path
// into either cache (sm_103a).
//
// What bounds them.  A few kilobytes each, but for the commits' rows: the latency of a launch and of
// the loads that depend on one another.  So each takes one launch where it can, and loads what
// does not depend on other loads together.
// Measured, calls one after another in a CUDA graph: masks and positions of 512 x 64 nodes 1.9 us; page
// tables of a step of 64 sequences, taken and given back, 9.7 us, of 256 prompts with slot maps 20.7 (a
// block, because a sequence's pages depend on what those before it take); paths of 64 sequences into
// packed tails 6.7 us, with the lengths 7.7, of 128 into 16-bit pages 3.4 and 4.1.
#include "grid_dep.cuh"
#include "host_common.h"
#include "quant_tile.cuh"

#include <algorithm>

namespace kitty {
namespace {

constexpr int kMaxNodes = KITTY_TREE_MAX_NODES;

// Sequence b's rows [first, first + count), or false (reported if asked to) where its starts are
// out of order or beyond the rows.
__device__ __forceinline__ bool rows_of(const int32_t* seq_start, int b, int n_tokens, int& first, int& count,
                                        int32_t* d_status, bool report) {
  first = seq_start[b];
  const int end = seq_start[b + 1];
  count = end - first;
  if (first >= 0 && first <= end && end <= n_tokens) return true;
  if (report) set_status(d_status, KITTY_ST_BAD_SEQ);
  return false;
}

// ------------------------------------------------------------- masks and positions
struct PlanParams {
  const int32_t *parents, *seq_start, *num_pages, *lens, *pos_base;
  unsigned long long* visible;
  int32_t* positions;
  int32_t* d_status;
  int n_tokens, B;
};

// Four warps a block, a tree a warp, two nodes a lane.  mask(i) = {i} + mask(parent(i)), by doubling:
// after round r a node's mask holds its 2^r nearest ancestors and `up` is the 2^r-th, so six
// rounds cover 64 nodes however deep the tree.
__global__ void __launch_bounds__(128) tree_plan_kernel(const PlanParams p) {
  __shared__ unsigned long long mask[4][kMaxNodes];
  __shared__ int8_t up[4][kMaxNodes];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.x * 4 + w;
  if (b >= p.B) return;
  int first, n;
  const int held = p.lens[b] + (p.num_pages != nullptr ? kPage * p.num_pages[b] : 0) +
                   (p.pos_base != nullptr ? p.pos_base[b] : 0);
  if (!rows_of(p.seq_start, b, p.n_tokens, first, n, p.d_status, lane == 0)) return;
  if (n > kMaxNodes) {
    if (lane == 0) set_status(p.d_status, KITTY_ST_BAD_LEN);
    return;
  }
  unsigned long long m[2];
  int u[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = lane + 32 * k;
    u[k] = i < n ? p.parents[first + i] : -1;
    if (u[k] < -1 || u[k] >= i) {
      set_status(p.d_status, KITTY_ST_BAD_TREE);
      u[k] = -1;
    }
    m[k] = 1ull << i;
  }
  for (int r = 0; r < 6; ++r) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      mask[w][lane + 32 * k] = m[k];
      up[w][lane + 32 * k] = (int8_t)u[k];
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (u[k] >= 0) {
        m[k] |= mask[w][u[k]];
        u[k] = up[w][u[k]];
      }
    }
    __syncwarp();
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = lane + 32 * k;
    if (i >= n) continue;
    if (p.visible != nullptr) p.visible[first + i] = m[k];
    if (p.positions != nullptr) p.positions[first + i] = held + __popcll(m[k]) - 1;
  }
}

// ------------------------------------------------------------- block tables
constexpr int kPThreads = 1024;  // sequences of a round

struct PageParams {
  const int32_t *num_pages, *lens, *seq_start;
  int32_t *held, *block_table, *free_ids, *free_count;
  long long* slots;
  int32_t* new_page_ids;
  int32_t* d_status;
  int n_tokens, extra, partial, shrink, max_pages, pool_pages, B;
};

// Pages that sequence b is to have, or -1 (reported) when it keeps what it has; `have`: what it has.
__device__ __forceinline__ int pages_wanted(const PageParams& p, int b, int& have) {
  have = p.held[b];
  long n = (long)p.lens[b] + min(p.extra, 0) + (p.num_pages != nullptr ? (long)kPage * p.num_pages[b] : 0);
  bool bad = p.lens[b] < 0 || (p.num_pages != nullptr && p.num_pages[b] < 0) || have < 0 || have > p.max_pages;
  if (p.seq_start != nullptr) {
    int first, count;
    if (!rows_of(p.seq_start, b, p.n_tokens, first, count, p.d_status, true)) return -1;
    n += count;
  }
  bad = bad || n < 0;
  if (bad) {
    set_status(p.d_status, KITTY_ST_BAD_LEN);
    return -1;
  }
  const int begun = p.partial ? kPage - 1 : 0;
  if ((n + begun) / kPage > p.max_pages) {
    set_status(p.d_status, KITTY_ST_TABLE_FULL);
    return -1;
  }
  // tokens that may come: as many as the row has room for
  return (int)min((n + max(p.extra, 0) + begun) / kPage, (long)p.max_pages);
}

// Inclusive sum over the block's threads.  `sums`: 32 entries.
__device__ __forceinline__ int block_scan(int x, int* sums) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();  // the last scan's sums have been read
  if (lane == 31) sums[w] = x;
  __syncthreads();
  if (w == 0) {
    int s = sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, s, d);
      if (lane >= d) s += y;
    }
    sums[lane] = s;
  }
  __syncthreads();
  return x + (w > 0 ? sums[w - 1] : 0);
}

// Places of `at` (rising) that are <= j: the thread whose pages item j belongs to.
__device__ __forceinline__ int owner(const int* at, int n, int j) {
  int lo = 0, hi = n;  // at[lo - 1] <= j < at[hi]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= j) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// One block: the stack's top moves from sequence to sequence.  1024 sequences a round: counts by a
// scan, then the pages themselves, one a thread, whose sequence is found in the counts'
// ends, so that one long row costs no more than many short ones.  First what is given back, from the
// last sequences to the first; then what is taken.
__global__ void __launch_bounds__(kPThreads) page_tables_kernel(const PageParams p) {
  __shared__ int ends[kPThreads], base[kPThreads], sums[32], any;
  __shared__ uint8_t corrupt[kPThreads];  // sequences that hold an id out of range
  const int tid = threadIdx.x;
  grid_trigger();
  int top = *p.free_count;
  if (top < 0 || top > p.pool_pages) {
    if (tid == 0) set_status(p.d_status, KITTY_ST_BAD_LEN);
    return;
  }
  const int rounds = (p.B + kPThreads - 1) / kPThreads;
  if (p.shrink) {
    for (int r = rounds - 1; r >= 0; --r) {
      const int b = r * kPThreads + tid;
      int have = 0, want = b < p.B ? pages_wanted(p, b, have) : -1;
      bool drop = want >= 0 && want < have;
      for (;;) {  // a second time if a sequence's ids are out of range: without it
        const int mine = drop ? have - want : 0;
        const int end = block_scan(mine, sums);
        ends[tid] = end;
        base[tid] = want;
        corrupt[tid] = 0;
        __syncthreads();
        const int total = sums[31];
        if (total == 0) break;
        bool bad = false;
        for (int j = tid; j < total; j += kPThreads) {
          const int s = owner(ends, kPThreads, j);
          const int col = base[s] + j - (s > 0 ? ends[s - 1] : 0);
          const int id = p.block_table[(size_t)(r * kPThreads + s) * p.max_pages + col];
          if (id < 0 || id >= p.pool_pages) {
            corrupt[s] = 1;
            bad = true;
          }
        }
        bad = __syncthreads_or(bad) != 0;
        if (!bad && total <= p.pool_pages - top) {  // (their sum may pass 32 bits)
          for (int j = tid; j < total; j += kPThreads) {
            const int s = owner(ends, kPThreads, j);
            const int col = base[s] + j - (s > 0 ? ends[s - 1] : 0);
            int32_t* entry = p.block_table + (size_t)(r * kPThreads + s) * p.max_pages + col;
            p.free_ids[top + total - 1 - j] = *entry;
            *entry = -1;
          }
          if (drop) p.held[b] = want;
          top += total;
          break;
        }
        if (tid == 0) set_status(p.d_status, KITTY_ST_BAD_PAGE);
        if (!bad) break;  // more pages than the pool has: some are there twice
        drop = drop && corrupt[tid] == 0;
        __syncthreads();
      }
      __syncthreads();
    }
  }
  bool room = true;  // no sequence so far went without
  for (int r = 0; r < rounds && room; ++r) {
    const int b = r * kPThreads + tid;
    int have = 0;
    const int want = b < p.B ? pages_wanted(p, b, have) : -1;
    const int more = max(0, want - have);
    const int end = block_scan(more, sums);
    const bool served = end <= top;
    if (!served && more > 0) set_status(p.d_status, KITTY_ST_NO_PAGES);
    ends[tid] = end;
    base[tid] = have;
    if (tid == 0) any = 0;
    __syncthreads();
    if (served) atomicMax(&any, end);
    room = __syncthreads_and(served) != 0;
    const int total = any;  // of the sequences that are served: the first ones
    for (int j = tid; j < total; j += kPThreads) {
      const int s = owner(ends, kPThreads, j);
      const int col = base[s] + j - (s > 0 ? ends[s - 1] : 0);
      int id = p.free_ids[top - 1 - j];
      if (id < 0 || id >= p.pool_pages) {
        set_status(p.d_status, KITTY_ST_BAD_PAGE);
        id = -1;
      }
      p.block_table[(size_t)(r * kPThreads + s) * p.max_pages + col] = id;
    }
    if (served && more > 0) p.held[b] = want;
    top -= total;
    __syncthreads();
  }
  if (!room) {  // later rounds: those that need pages are told
    for (int b = tid; b < p.B; b += kPThreads) {
      int have = 0;
      if (pages_wanted(p, b, have) > have) set_status(p.d_status, KITTY_ST_NO_PAGES);
    }
  }
  if (tid == 0) *p.free_count = top;
}

// New token t of its sequence, behind the tokens that it holds: its place in the pool.
__global__ void __launch_bounds__(256) slots_kernel(const PageParams p) {
  grid_wait();
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t >= p.n_tokens || t >= p.seq_start[p.B]) return;
  int lo = 0, hi = p.B;  // sequences that end at or before t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (p.seq_start[mid + 1] <= t) lo = mid + 1;
    else hi = mid;
  }
  const int b = lo;
  if (b >= p.B || p.seq_start[b] < 0 || p.seq_start[b] > t) return;
  const long pos = (long)p.lens[b] + (p.num_pages != nullptr ? (long)kPage * p.num_pages[b] : 0) + (t - p.seq_start[b]);
  const int have = p.held[b];
  int id = -1;
  if (pos >= 0 && pos / kPage < have && have <= p.max_pages) id = p.block_table[(size_t)b * p.max_pages + pos / kPage];
  if (p.slots != nullptr) p.slots[t] = id < 0 ? -1 : (long long)id * kPage + pos % kPage;
  if (p.new_page_ids != nullptr) p.new_page_ids[t] = pos % kPage == 0 ? id : -1;
}

// ------------------------------------------------------------- the accepted path
struct CommitParams {
  const uint16_t *k, *v;
  size_t k_stride, v_stride;
  const int32_t *seq_start, *path, *block_table;
  int32_t* path_len;  // of a refused sequence, set to 0 where the lengths advance
  uint16_t *tail_k, *tail_v;  // packed cache
  int32_t *tail_len, *num_pages;
  float *run_sum, *run_sumsq;
  int32_t* run_count;
  int32_t* ctx_len;  // 16-bit cache
  uint8_t* pool;
  int32_t* d_status;
  int n_tokens, path_width, max_pages, pool_pages, counted, B, Hkv, n_hi, running;
};

// What sequence b's n accepted tokens do: tokens held before, and whether they are taken.  The whole
// block calls this; every block of a sequence comes to the same answer, and the first one's
// thread 0 reports.  rows[i]: the row of accepted token i.
struct Accepted {
  int n;
  long before;
  bool ok;
};
template <bool PACKED>
__device__ __forceinline__ Accepted accepted(const CommitParams& p, int b, bool report, int* rows) {
  Accepted a = {p.path_len[b], 0, false};
  const int tid = threadIdx.x;
  const int node = tid < p.path_width ? p.path[(size_t)b * p.path_width + tid] : 0;
  int first, count, code = KITTY_ST_OK;
  const int len = PACKED ? p.tail_len[b] : p.ctx_len[b], np = PACKED ? p.num_pages[b] : 0;
  const bool mine = rows_of(p.seq_start, b, p.n_tokens, first, count, nullptr, false);
  const long room = (long)p.max_pages * kPage;
  const long held = (long)kPage * np + len;
  a.before = p.counted ? held - a.n : held;
  if (!mine) code = KITTY_ST_BAD_SEQ;
  else if (count > kMaxNodes) code = KITTY_ST_BAD_LEN;
  else if (a.n < 0 || a.n > p.path_width) code = KITTY_ST_BAD_TREE;
  else if (len < 0 || a.before < 0 || (PACKED ? len >= kPage || np < 0 || np > p.max_pages : a.before > room)) code = KITTY_ST_BAD_LEN;
  else if (PACKED ? (a.before + a.n) / kPage > p.max_pages : a.before + a.n > room) code = KITTY_ST_TABLE_FULL;
  bool bad_node = false, bad_page = false;
  if (code == KITTY_ST_OK && tid < a.n) {
    bad_node = node < 0 || node >= count;
    rows[tid] = first + node;
    // the page of this token, if it must be there: where it lies, or that its tail fills
    const long pos = a.before + tid;
    if (!PACKED || pos % kPage == kPage - 1) {
      const int id = p.block_table[(size_t)b * p.max_pages + pos / kPage];
      bad_page = id < 0 || id >= p.pool_pages;
    }
  }
  if (__syncthreads_or(bad_node)) code = KITTY_ST_BAD_TREE;
  else if (__syncthreads_or(bad_page)) code = KITTY_ST_BAD_PAGE;
  if (code != KITTY_ST_OK && report && tid == 0) set_status(p.d_status, code);
  a.ok = code == KITTY_ST_OK;
  return a;
}

// Accepted rows [i0, i1) of kv head h to rows slot0 + i of a 128-channel array, 16 lanes a row, Keys
// and Values side by side.
__device__ __forceinline__ void copy_rows(const CommitParams& p, const int* rows, int h, int i0, int i1, uint16_t* kd,
                                          uint16_t* vd, int slot0) {
  const int c = 8 * (threadIdx.x & 15);
  for (int x = 2 * i0 + (threadIdx.x >> 4); x < 2 * i1; x += (int)blockDim.x / 16) {
    const int i = x >> 1;
    const size_t row = rows[i];
    const uint16_t* src = x & 1 ? p.v + row * p.v_stride : p.k + row * p.k_stride;
    uint16_t* dst = (x & 1 ? vd : kd) + (size_t)(slot0 + i) * kD;
    *reinterpret_cast<uint4*>(dst + c) = *reinterpret_cast<const uint4*>(src + (size_t)h * kD + c);
  }
}

// One block per (sequence, kv head): the tail filled up to its 32 tokens, quantized into the page that
// the table holds, and so on; what is left stays in the tail.
template <int DT, int W, int V>
__global__ void __launch_bounds__(kQThreads) tree_commit_kernel(const CommitParams p) {
  __shared__ QuantSmem sm;
  __shared__ int rows[kMaxNodes];
  grid_trigger();
  const int b = blockIdx.x, h = blockIdx.y, c = threadIdx.x;
  const Accepted a = accepted<true>(p, b, h == 0, rows);
  if (!a.ok || a.n == 0) return;
  const size_t sh = (size_t)b * p.Hkv + h;
  uint16_t *tk = p.tail_k + sh * kPage * kD, *tv = p.tail_v + sh * kPage * kD;
  const BlobLayout lay(p.n_hi, W, V);
  int slot = (int)(a.before % kPage);
  long page = a.before / kPage;
  float rs = 0.f, rq = 0.f;
  int rc = 0;
  const bool fills = slot + a.n >= kPage;
  if (p.running && fills) {
    rs = p.run_sum[sh * kD + c];
    rq = p.run_sumsq[sh * kD + c];
    rc = p.run_count[sh];
  }
  for (int i = 0; i < a.n;) {
    const int take = min(a.n - i, kPage - slot);
    copy_rows(p, rows, h, i, i + take, tk, tv, slot - i);
    i += take;
    slot += take;
    if (slot < kPage) break;
    __syncthreads();  // the tail's rows are visible to the whole block
    const int id = p.block_table[(size_t)b * p.max_pages + page];
    quantize_tile<DT, W, V>(sm, tk, tv, kD, p.n_hi, p.running != 0, rs, rq, rc,
                            p.pool + ((size_t)id * p.Hkv + h) * lay.bytes, p.d_status);
    ++page;
    slot = 0;
  }
  if (p.running && fills) {
    p.run_sum[sh * kD + c] = rs;
    p.run_sumsq[sh * kD + c] = rq;
    if (c == 0) p.run_count[sh] = rc;
  }
}

// One block per (sequence, kv head): each accepted row to its place in the pages.
__global__ void __launch_bounds__(128) f16kv_tree_commit_kernel(const CommitParams p) {
  __shared__ int rows[kMaxNodes];
  grid_trigger();
  const int b = blockIdx.x, h = blockIdx.y;
  const Accepted a = accepted<false>(p, b, h == 0, rows);
  if (!a.ok) return;
  for (int i = 0; i < a.n;) {
    const long pos = a.before + i;
    const int slot = (int)(pos % kPage), take = min(a.n - i, kPage - slot);
    const int id = p.block_table[(size_t)b * p.max_pages + pos / kPage];
    uint16_t* blob = reinterpret_cast<uint16_t*>(p.pool) + ((size_t)id * p.Hkv + h) * 2 * kPage * kD;
    copy_rows(p, rows, h, i, i + take, blob, blob + kPage * kD, slot - i);
    i += take;
  }
}

// Lengths, once every head of a sequence has used the old ones: a block a sequence.  One that is refused
// leaves a path of no tokens: layers that find the lengths counted already would take its last cached
// tokens for the path's otherwise, and write over them.
template <bool PACKED>
__global__ void __launch_bounds__(kMaxNodes) tree_commit_finish(const CommitParams p) {
  __shared__ int rows[kMaxNodes];
  grid_wait();
  const int b = blockIdx.x;
  const Accepted a = accepted<PACKED>(p, b, false, rows);
  if (threadIdx.x != 0) return;
  if (!a.ok) {
    p.path_len[b] = 0;
    return;
  }
  const long after = a.before + a.n;
  if (PACKED) {
    p.num_pages[b] = (int)(after / kPage);
    p.tail_len[b] = (int)(after % kPage);
  } else {
    p.ctx_len[b] = (int)after;
  }
}

bool rows_ok(const void* p, int64_t stride, int heads) {
  return p != nullptr && aligned16(p) && stride >= (int64_t)heads * kD && stride % 8 == 0;
}

// Checks common to the commits; 1: nothing to do.
int commit_params(const kitty_cfg* cfg, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                  int32_t n_tokens, const int32_t* seq_start, const int32_t* path, int32_t path_width,
                  int32_t* path_len, const int32_t* block_table, int32_t max_pages, void* pool,
                  int32_t pool_pages, int32_t counted, int32_t B, int32_t* d_status, CommitParams* p) {
  const int rc = check_cfg(cfg);
  if (rc != KITTY_OK) return rc;
  if (B < 0 || n_tokens < 0 || path_width < 0 || max_pages < 0 || pool_pages < 0) return KITTY_ERR_INVALID_ARG;
  if (path_width > kMaxNodes) return KITTY_ERR_UNSUPPORTED;
  if (B == 0 || n_tokens == 0 || path_width == 0) return 1;
  const int Hkv = cfg->num_kv_heads;
  if (!rows_ok(k, k_stride, Hkv) || !rows_ok(v, v_stride, Hkv) || !seq_start || !path || !path_len ||
      !block_table || !pool || !aligned16(pool))
    return KITTY_ERR_INVALID_ARG;
  if (Hkv > 65535) return KITTY_ERR_UNSUPPORTED;
  p->k = static_cast<const uint16_t*>(k);
  p->v = static_cast<const uint16_t*>(v);
  p->k_stride = (size_t)k_stride;
  p->v_stride = (size_t)v_stride;
  p->seq_start = seq_start;
  p->path = path;
  p->path_len = path_len;
  p->block_table = block_table;
  p->pool = static_cast<uint8_t*>(pool);
  p->d_status = d_status;
  p->n_tokens = n_tokens;
  p->path_width = path_width;
  p->max_pages = max_pages;
  p->pool_pages = pool_pages;
  p->counted = counted != 0;
  p->B = B;
  p->Hkv = Hkv;
  p->n_hi = cfg->n_hi;
  return KITTY_OK;
}

template <bool PACKED>
int finish(const CommitParams& p, cudaStream_t s) {
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && !p.counted)
    e = launch_dependent(tree_commit_finish<PACKED>, dim3((unsigned)p.B), kMaxNodes, 0, s, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? KITTY_OK : KITTY_ERR_CUDA;
}

}  // namespace
}  // namespace kitty

using namespace kitty;

extern "C" int kitty_tree_plan(const int32_t* parents, const int32_t* seq_start, int32_t n_tokens,
                               const int32_t* num_pages, const int32_t* lens, const int32_t* pos_base,
                               uint64_t* visible, int32_t* positions, int32_t B, int32_t* d_status,
                               void* stream) {
  if (B < 0 || n_tokens < 0) return KITTY_ERR_INVALID_ARG;
  if (B == 0 || n_tokens == 0) return KITTY_OK;
  if (!parents || !seq_start || !lens || (!visible && !positions) || (reinterpret_cast<uintptr_t>(visible) & 7u) != 0)
    return KITTY_ERR_INVALID_ARG;
  const PlanParams p = {parents, seq_start, num_pages, lens, pos_base, reinterpret_cast<unsigned long long*>(visible),
                        positions, d_status, n_tokens, B};
  tree_plan_kernel<<<(unsigned)((B + 3) / 4), 128, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? KITTY_OK : KITTY_ERR_CUDA;
}

extern "C" int kitty_page_tables(const int32_t* num_pages, const int32_t* lens, const int32_t* seq_start,
                                 int32_t n_tokens, int32_t extra, int32_t partial, int32_t shrink,
                                 int32_t* held, int32_t* block_table, int32_t max_pages,
                                 int32_t* free_ids, int32_t* free_count, int32_t pool_pages,
                                 int64_t* slots, int32_t* new_page_ids, int32_t B, int32_t* d_status,
                                 void* stream) {
  if (B < 0 || n_tokens < 0 || max_pages < 0 || pool_pages < 0 || ((slots || new_page_ids) && !seq_start))
    return KITTY_ERR_INVALID_ARG;
  if (B == 0) return KITTY_OK;
  if (!lens || !held || !free_count || (max_pages > 0 && !block_table) || (pool_pages > 0 && !free_ids) ||
      (reinterpret_cast<uintptr_t>(slots) & 7u) != 0)
    return KITTY_ERR_INVALID_ARG;
  // a scan's sums are 32-bit
  if ((long)std::min(B, kPThreads) * max_pages > 0x7FFFFFFFl) return KITTY_ERR_UNSUPPORTED;
  const PageParams p = {num_pages, lens, seq_start, held, block_table, free_ids, free_count,
                        reinterpret_cast<long long*>(slots), new_page_ids, d_status, n_tokens, extra,
                        partial != 0, shrink != 0, max_pages, pool_pages, B};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  page_tables_kernel<<<1, kPThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && (slots || new_page_ids) && n_tokens > 0)
    e = launch_dependent(slots_kernel, dim3((unsigned)((n_tokens + 255) / 256)), 256, 0, s, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? KITTY_OK : KITTY_ERR_CUDA;
}

extern "C" int kitty_tree_commit(const kitty_cfg* cfg, const void* k, int64_t k_stride, const void* v,
                                 int64_t v_stride, int32_t n_tokens, const int32_t* seq_start,
                                 const int32_t* path, int32_t path_width, int32_t* path_len,
                                 void* tail_k, void* tail_v, int32_t* tail_len, float* run_sum,
                                 float* run_sumsq, int32_t* run_count, const int32_t* block_table,
                                 int32_t max_pages, int32_t* num_pages, void* pool, int32_t pool_pages,
                                 int32_t counted, int32_t B, int32_t* d_status, void* stream) {
  CommitParams p = {};
  const int rc = commit_params(cfg, k, k_stride, v, v_stride, n_tokens, seq_start, path, path_width, path_len,
                               block_table, max_pages, pool, pool_pages, counted, B, d_status, &p);
  if (rc != KITTY_OK) return rc == 1 ? KITTY_OK : rc;
  const bool running = cfg->rank_mode != KITTY_RANK_PAGE;  // sequence mode appends as running
  if (!tail_k || !tail_v || !tail_len || !num_pages || !aligned16(tail_k) || !aligned16(tail_v) ||
      (running && (!run_sum || !run_sumsq || !run_count)))
    return KITTY_ERR_INVALID_ARG;
  p.tail_k = static_cast<uint16_t*>(tail_k);
  p.tail_v = static_cast<uint16_t*>(tail_v);
  p.tail_len = tail_len;
  p.num_pages = num_pages;
  p.run_sum = run_sum;
  p.run_sumsq = run_sumsq;
  p.run_count = run_count;
  p.running = running;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)B, (unsigned)p.Hkv);
  auto launch = [&](auto kernel) { kernel<<<grid, kQThreads, 0, s>>>(p); };
  const bool bf = cfg->in_dtype == KITTY_BF16;
  if (cfg->lo_bit == 2) bf ? launch(tree_commit_kernel<KITTY_BF16, 2, 2>) : launch(tree_commit_kernel<KITTY_F16, 2, 2>);
  else if (v_bits(cfg) == 2) bf ? launch(tree_commit_kernel<KITTY_BF16, 4, 2>) : launch(tree_commit_kernel<KITTY_F16, 4, 2>);
  else bf ? launch(tree_commit_kernel<KITTY_BF16, 4, 4>) : launch(tree_commit_kernel<KITTY_F16, 4, 4>);
  return finish<true>(p, s);
}

extern "C" int kitty_f16kv_tree_commit(const kitty_cfg* cfg, const void* k, int64_t k_stride, const void* v,
                                       int64_t v_stride, int32_t n_tokens, const int32_t* seq_start,
                                       const int32_t* path, int32_t path_width, int32_t* path_len,
                                       void* pool, int32_t pool_pages, const int32_t* block_table,
                                       int32_t max_pages, int32_t* ctx_len, int32_t counted, int32_t B,
                                       int32_t* d_status, void* stream) {
  CommitParams p = {};
  const int rc = commit_params(cfg, k, k_stride, v, v_stride, n_tokens, seq_start, path, path_width, path_len,
                               block_table, max_pages, pool, pool_pages, counted, B, d_status, &p);
  if (rc != KITTY_OK) return rc == 1 ? KITTY_OK : rc;
  if (!ctx_len) return KITTY_ERR_INVALID_ARG;
  p.ctx_len = ctx_len;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  f16kv_tree_commit_kernel<<<dim3((unsigned)B, (unsigned)p.Hkv), 128, 0, s>>>(p);
  return finish<false>(p, s);
}
