// Attention of drafted tokens over a sequence's cache and over each other, on the fifth-generation
// tensor cores (sm_103a).
//
//   out[t][hq] = softmax(sm_scale * q . [K_prefix; K_b; K_tree]) . [V_prefix; V_b; V_tree]
//
// Rows.  The query heads of a kv head over the nodes of a sequence's tree, node by node: n * g
// rows that see the same cached tokens.  One block takes up to N of them (N = 16, 32, 64 by the
// largest tree) and a share of the sequence's tiles of 128 tokens.  Tokens are the
// products' 128 rows and query rows their N columns, so that a product costs what the rows
// need: 16 rows an eighth of 128.  Per tile
//   S^T = K Q^T         128 x N x 128, fp32 in tensor memory
//   p = 2^(s - m)       a thread a token: its scores from tensor memory, p to shared memory
//   O^T += V^T P^T      128 channels x N x 128 tokens, fp32 in tensor memory
// The reference m of a row is set 2^4 below its maximum over the first tile and moves only when a
// score passes it by more than 2^15: what p loses below 2^-25 is 2^-29 of the largest then.
// A row decides by its own scores, so its bytes do not depend on the others.
//
// Even and odd tiles are two pipelines with warps, references and outputs of their own, which share
// the products' warp and are joined at the end.  Every kind of work has its warps, and what bounds
// the block is the rate at which their instructions come: it was 3400 cycles a tile of 64 rows with
// the loops unrolled (120 KB of code) and is 2500 with loops of a few dozen instructions
// (94 KB, most of it run once; scores 16 columns at a time, a page's Keys in quarters).
// Measured, 8 kv heads, contexts spread below the given lengths; 2-bit pages: 64 sequences x 8192 tokens x
// 16 nodes x 4 heads 322 us (298 MB, 90 GFLOP: 280 TFLOP/s), 8 x 32768 x 64 nodes x 8 heads 909 us
// (361 GFLOP: 397 TFLOP/s), 4 x 1024 chains of 5 18 us; 16-bit pages: 32 x 8192 x 16 x 4 204 us (715 MB:
// 3.5 TB/s).
//
// Packed pages (four to a tile) are staged whole by bulk copies and dequantized straight into
// tensor memory: the planes' fragment order is that of 16-row stores of 128 bits, whose
// registers a lane has after one AND and one fused multiply-add for two codes.
//   Keys    (16 + code * 2^e) * S - 16 * S = S * code * 2^e, exact: e depends on the token's place
//           alone, and the thread of the token takes it off.  Boosted channels' low codes are
//           spread into base-plane order first and joined to 4-bit codes.  The channel
//           minima's q.M is a product of its own (mma.sync, 4 pages x N rows) into shared memory.
//   Values  (16 + code * 2^e - C) * S = S * (code - middle) * 2^e, exact; e depends on the channel
//           alone.  The groups' middles and a row of ones are multiplied with P by mma.sync: so
//           the sum of p is that of the rounded ones.
// 16-bit pages come by tiled TMA loads, swizzled, as operands in shared memory (Values as they
// lie, channels contiguous); p is a (high, rest) pair.
// The last tile is the sequence's loose tokens: its tail (16-bit: its last, partial page) and the
// drafted ones, 32 + 64 at most, copied row by row; masks apply there alone.
//
// Roundings: p to fp16 (2^-11), a group's middle to fp16, for 8-bit boosted Keys step * code to
// fp16; 16-bit pages: p to two halves.  "Exact" above holds while the results are no subnormal fp16:
// times 2^-4, Value steps below 2^-13 and loose Values below 2^-10 (bf16: 2^-13) lose up to 2^-21 each,
// Key steps below 2^-14 likewise.  (A scale of the page's own would take its largest step first, and an
// instruction a register in the loops that bound the block.)
#include "prefix.h"

#include <algorithm>
#include <atomic>
#include <cmath>

#include "grid_dep.cuh"
#include "host_common.h"
#include "kitty_common.cuh"
#include "partials.h"
#include "tcgen05.cuh"

namespace kitty {
namespace {

constexpr int kMaxNodes = KITTY_TREE_MAX_NODES;
constexpr int kTile = 128, kTilePages = 4;
// Warps: of each kind one half for the even tiles and one for the odd ones.  Softmax (a thread a
// token), the Keys' operand (a warp a page), the Values' (a warp a group of channels), q.M, the sums;
// then one that issues products and one that requests copies.  16-bit pages have no use for the
// operands' but for the loose tokens, and one of q.M's requests the Values.
constexpr int kSoftmaxWarps = 8, kKeyWarp = 8, kValueWarp = 16, kBiasWarp = 24, kSumWarp = 26, kMmaWarp = 30, kFetchWarp = 31;
constexpr int kTreeThreads = 1024;
constexpr int kMaxRaw = 4;        // staged tiles of packed pages: 2 or 4 (a warp sees every other one)
constexpr int kFlags = 16;        // tiles whose page flags are kept
constexpr int kLoose = 96;        // loose tokens: 32 of the tail, 64 nodes
constexpr int kLoosePitch = 272;
constexpr uint32_t kTreeWaitPolls = 1u << 20;
constexpr float kFloor = -1.0e30f;
constexpr float kSlack = 15.f;    // log2 units that a score may pass m by
constexpr float kMargin = -4.f;   // m against the maximum, when it is set
constexpr int kMaxSplits = 32;

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
  float* ws;
  int32_t* d_status;
  float sm_log2;
  uint32_t wait_polls;
  int n_tokens, max_nodes, pool_pages, n_prefix, max_pages, B, Hq, Hkv, g, n_hi, blob, in_dtype, out_dtype;
  const float* pre;  // the prefix kernel's partials, if it has attended the prefix
  int units, splits, slots, raw_stages;  // slots: of them, a row
  int direct;  // one partial a row: it is the output
};

// Packed pages: Key planes of W bits, Values of V bits; N rows.
template <int W_, int V_, int N_>
struct PackedTree {
  static constexpr bool kPacked = true, kBf16 = false, kPair = false;
  static constexpr int W = W_, V = V_, N = N_;
  static constexpr int kOpCols = 256;  // Keys' operands (two of 64 columns), then the Values'
};
// 16-bit pages.
template <bool BF, int N_>
struct PlainTree {
  static constexpr bool kPacked = false, kBf16 = BF, kPair = true;
  static constexpr int W = 0, V = 0, N = N_;
  static constexpr int kOpCols = 0;
};
template <class F>
struct Sizes {
  static constexpr int N = F::N;
  static constexpr int kQHalf = N * 128, kQ = 2 * kQHalf;
  static constexpr int kPHalf = kTile * 128, kP = kPHalf * (F::kPair ? 2 : 1);  // 128 tokens of 64 rows
  static constexpr int kSCol = F::kOpCols, kOCol = kSCol + 2 * N, kCols = kOCol + 2 * N;
  static constexpr int kHalf16 = kTile * 128, kTile16 = 2 * kHalf16;  // a 16-bit tile of Keys or Values
  static constexpr int kSpread = F::kPacked ? 512 * F::W : 0;         // a page's low codes in base-plane order
  static constexpr int kPs = F::kPacked ? 4 : 2;                      // tiles whose p are kept
  static constexpr int kFixed = kQ + kPs * kP + (F::kPacked ? 2 * kLoose * kLoosePitch + 8 * kSpread + 4 * 1024
                                                         : 4 * kTile16);
};

// Shared memory of a block of packed pages without its staged tiles, and with `stages` of them.
constexpr int kSharedMost = 227 * 1024;
template <class F>
constexpr int fixed_bytes() { return 1024 + Sizes<F>::kFixed; }

struct Held {  // of one sequence
  int first, n;              // its drafted rows
  int prefix, pages, loose;  // prefix pages, full pages of its own, tokens behind them
  bool ok;
  int code;
};

// What sequence b has and asks for; every block of it comes to the same answer.
template <bool PACKED>
__device__ __forceinline__ Held held_of(const TreeParams& p, int b) {
  Held h;
  h.first = p.seq_start[b];
  const int end = p.seq_start[b + 1];
  h.n = end - h.first;
  h.prefix = p.n_prefix > 0 && p.prefix_pages != nullptr ? p.prefix_pages[b] : p.n_prefix;
  bool bad;
  if (PACKED) {
    h.pages = p.num_pages[b];
    h.loose = p.tail_len[b];
    bad = h.pages < 0 || h.pages > p.max_pages || h.loose < 0 || h.loose > kPage;
  } else {
    const int len = p.ctx_len[b];
    bad = len < 0 || len > (long)p.max_pages * kPage;
    h.pages = len / kPage;
    h.loose = len % kPage;
  }
  h.code = KITTY_ST_OK;
  h.ok = true;
  if (h.prefix < 0 || h.prefix > p.n_prefix) {
    h.prefix = 0;
    h.code = KITTY_ST_BAD_LEN;
  }
  if (h.first < 0 || h.n < 0 || end > p.n_tokens) {
    h.ok = false;
    h.code = KITTY_ST_BAD_SEQ;
  } else if (h.n > p.max_nodes || (h.n > 0 && bad)) {
    h.ok = false;
    h.code = KITTY_ST_BAD_LEN;
  }
  return h;
}

// ------------------------------------------------------------- small pieces
// One poll of a barrier phase, in which the hardware may suspend the thread for a while.  (With a time
// given it becomes a loop of naps: 5000 of 11300 instructions a tile were polls and their votes.)
__device__ __forceinline__ bool try_phase(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Whole warp: waits for a phase, at most `polls` polls; false when it, or another warp of the block, has
// given up.
__device__ __forceinline__ bool wait_phase(uint64_t& bar, int parity, uint32_t polls, volatile int* abort) {
  const uint32_t a = smem_u32(&bar), ph = (uint32_t)parity;
#pragma unroll 1
  for (uint32_t i = 0; i < polls; ++i) {
    if (__all_sync(0xFFFFFFFFu, try_phase(a, ph))) return true;
    if (*abort != 0) return false;
  }
  *abort = 1;
  return false;
}

__device__ __forceinline__ float ex2a(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Maximum over the warp, through integers of the same order.  (An intrinsic, not an instruction in asm:
// that one was moved under a condition on the lane which alone used its result.)
__device__ __forceinline__ float warp_max(float x) {
  const int i = __float_as_int(x), k = __reduce_max_sync(0xFFFFFFFFu, i ^ ((i >> 31) & 0x7FFFFFFF));
  return __int_as_float(k ^ ((k >> 31) & 0x7FFFFFFF));
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts32(uint32_t a, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void sts8(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint32_t h2mul(uint32_t a, uint32_t b) { return h2_bits(__hmul2(bits_h2(a), bits_h2(b))); }
__device__ __forceinline__ uint32_t h2add(uint32_t a, uint32_t b) { return h2_bits(__hadd2(bits_h2(a), bits_h2(b))); }
__device__ __forceinline__ uint32_t h2fma(uint32_t a, uint32_t b, uint32_t c) {
  return h2_bits(__hfma2(bits_h2(a), bits_h2(b), bits_h2(c)));
}
__host__ __device__ constexpr uint32_t two(uint32_t half) { return half * 0x00010001u; }

// 16 lanes (rows) of tensor memory: the register pair (2i, 2i + 1) of lane (r, qq) goes to column
// 4i + qq of rows r and r + 8.
__device__ __forceinline__ void tmem_st_frag(uint32_t a, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t a, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(a));
}
__device__ __forceinline__ void tmem_st8(uint32_t a, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// C columns of this thread's lane.
template <int C>
__device__ __forceinline__ void tmem_load(uint32_t a, uint32_t (&x)[C]) {
  if constexpr (C >= 32) {
#pragma unroll
    for (int k = 0; k < C; k += 32) tmem_ld32(a + k, *reinterpret_cast<uint32_t(*)[32]>(x + k));
  } else {
#pragma unroll
    for (int k = 0; k < C; k += 8) tmem_ld8(a + k, x + k);
  }
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int k = 0; k < C; ++k) pin(x[k]);
}

// D(16x8 f32) = A(16x16 f16) * B(16x8 f16), warp-wide, where A's rows 8 .. 15 are zeros.
__device__ __forceinline__ void mma_rows8(float (&d)[4], uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%5}, {%7,%8}, "
      "{%9,%9,%9,%9};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(0u), "r"(a2), "r"(b0), "r"(b1), "f"(0.f));
}

// (a, b) = (a, b) * scale + (c, d)
__device__ __forceinline__ void fma2(uint32_t& a, uint32_t& b, uint64_t scale, uint32_t c, uint32_t d) {
  uint64_t e, s;
  asm("mov.b64 %0, {%1, %2};" : "=l"(e) : "r"(a), "r"(b));
  asm("mov.b64 %0, {%1, %2};" : "=l"(s) : "r"(c), "r"(d));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(e) : "l"(e), "l"(scale), "l"(s));
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(e));
}

// Or over the 128 threads of a softmax group, which all come here.
__device__ __forceinline__ bool group_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "barrier.cta.red.or.pred p, %2, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int id) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory"); }

// ------------------------------------------------------------- packed Keys
// A code at bits 2 + sh of a 16-bit half under the exponent of 16 reads 16 + code * 2^(sh - 4).
constexpr uint32_t k16 = two(0x4C00);
// (x & mask) | 16.0: one instruction, if both constants are in registers (the compiler made two of it).
struct Codes {
  uint32_t sixteen;
  __device__ __forceinline__ Codes() { asm volatile("mov.b32 %0, %1;" : "=r"(sixteen) : "n"(k16)); }
  __device__ __forceinline__ uint32_t operator()(uint32_t x, uint32_t mask) const {
    uint32_t y;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "r"(mask), "r"(sixteen));
    return y;
  }
};

// The low codes of a page's boosted channels, spread into base-plane order at `to` (512 W bytes,
// zeros where a channel has none).  Whole warp.
template <int W>
__device__ __forceinline__ void spread_low(uint32_t raw, uint32_t to, int n_hi) {
  const int lane = threadIdx.x & 31, r = lane >> 2, qq = lane & 3, nx = n_hi / 16;
  __syncwarp();  // the last page's have been read
#pragma unroll
  for (int i = 0; i < W; ++i) sts128(to + 16 * (lane + 32 * i), make_uint4(0, 0, 0, 0));
  __syncwarp();
  const uint32_t kch = raw + 512 * W + 4 * W * n_hi + 512, plane = raw + 512 * W + 2 * W * nx * lane;
  const uint32_t mine = to + 64 * W * r;  // the lanes of this lane's tokens
#pragma unroll 1
  for (int js = 0; js < nx; ++js) {
    const uint32_t ids = lds32(kch + 16 * js + 4 * qq);
#pragma unroll
    for (int mt = 0; mt < W / 2; ++mt) {
      // rotated back by two bits, byte 2e + h holds the column parity e, half h; ids: 2h + e
      uint32_t x = lds32(plane + 2 * W * js + 4 * mt);
      x = __funnelshift_r(x, x, 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t c = (ids >> (8 * i)) & 127u, byte = x >> (8 * (2 * (i & 1) + (i >> 1)));
        // word of channel c: lane (r, (c & 7) / 2), k-step c / 16 (W = 4: and mt); its byte there
        sts8(mine + 16 * W * ((c & 7) >> 1) + 2 * W * (c >> 4) + 4 * mt + 2 * (c & 1) + ((c >> 3) & 1), byte);
      }
    }
  }
  __syncwarp();
}

// A page's Keys, staged at raw, to the 32 lanes of tensor memory at `to`: 64 columns of channel pairs.
// (Spread words are not rotated as a plane's are: that is done here.)
template <int W>
__device__ __forceinline__ void put_keys(uint32_t raw, uint32_t to, uint32_t spread, int n_hi, int32_t* d_status) {
  const int lane = threadIdx.x & 31, qq = lane & 3;
  const uint32_t ks = raw + 512 * W + 4 * W * n_hi;
  const bool boosted = n_hi > 0;
  const Codes at16;
  if (boosted) spread_low<W>(raw, spread, n_hi);
#pragma unroll 1
  for (int part = 0; part < 4; ++part) {
  const uint32_t sq = ks + 64 * part + 4 * qq;
  uint32_t w[W], lo[W];  // of two k-steps
#pragma unroll
  for (int i = 0; i < W / 2; ++i) {
    const uint2 a = lds64(raw + 16 * W * lane + 4 * W * part + 8 * i);
    w[2 * i] = a.x;
    w[2 * i + 1] = a.y;
    if (boosted) {
      const uint2 c = lds64(spread + 16 * W * lane + 4 * W * part + 8 * i);
      lo[2 * i] = c.x;
      lo[2 * i + 1] = c.y;
    }
  }
  uint32_t a[2][8];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t S[2] = {lds32(sq + 32 * j), lds32(sq + 32 * j + 16)};
    const uint32_t T[2] = {h2mul(S[0], two(0xCC00)), h2mul(S[1], two(0xCC00))};  // -16 S
    if (W == 2) {
      if (!boosted) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t x = h ? __funnelshift_r(w[j], w[j], 8) : w[j];
          uint32_t* o0 = &a[0][2 * (2 * j + h)];
          uint32_t* o1 = &a[1][2 * (2 * j + h)];
          o0[0] = h2fma(at16(x, two(0x000C)), S[h], T[h]);
          o0[1] = h2fma(at16(x, two(0x0030)), S[h], T[h]);
          o1[0] = h2fma(at16(x, two(0x00C0)), S[h], T[h]);
          o1[1] = h2fma(at16(x, two(0x0300)), S[h], T[h]);
        }
      } else {
        // 4-bit codes at bits 2 and 6: of the tokens' blocks 0, 2 and of 1, 3.  lo: not rotated.
        const uint32_t y = __funnelshift_l(lo[j], lo[j], 2), up = __funnelshift_l(w[j], w[j], 2);
        const uint32_t A = (up & 0x33333333u) | (y & 0xCCCCCCCCu);
        const uint32_t B = (w[j] & 0x33333333u) | (lo[j] & 0xCCCCCCCCu);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t xa = h ? __funnelshift_r(A, A, 8) : A, xb = h ? __funnelshift_r(B, B, 8) : B;
          uint32_t* o0 = &a[0][2 * (2 * j + h)];
          uint32_t* o1 = &a[1][2 * (2 * j + h)];
          o0[0] = h2fma(at16(xa, two(0x003C)), S[h], T[h]);
          o0[1] = h2fma(at16(xb, two(0x003C)), S[h], T[h]);
          o1[0] = h2fma(at16(xa, two(0x03C0)), S[h], T[h]);
          o1[1] = h2fma(at16(xb, two(0x03C0)), S[h], T[h]);
        }
      }
    } else {
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const uint32_t x0 = w[(2 * j + mt) % W];
        const uint32_t l0 = boosted ? __funnelshift_l(lo[(2 * j + mt) % W], lo[(2 * j + mt) % W], 2) : 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t x = h ? __funnelshift_r(x0, x0, 8) : x0;
          uint32_t* o = &a[mt][2 * (2 * j + h)];
          o[0] = h2fma(at16(x, two(0x003C)), S[h], T[h]);
          o[1] = h2fma(at16(x, two(0x03C0)), S[h], T[h]);
          if (boosted) {  // + S / 16 * low code, rounded once
            const uint32_t l = h ? __funnelshift_r(l0, l0, 8) : l0, s = h2mul(S[h], two(0x2C00));
            o[0] = h2fma(h2add(at16(l, two(0x003C)), two(0xCC00)), s, o[0]);
            o[1] = h2fma(h2add(at16(l, two(0x03C0)), two(0xCC00)), s, o[1]);
          }
        }
      }
    }
  }
  tmem_st_frag(to + 16 * part, a[0]);
  tmem_st_frag(to + 16 * part + (16u << 16), a[1]);
  }
  const uint2 s4 = lds64(ks + 8 * lane);  // steps that times 16 leave fp16
  const uint32_t top = __vmaxu2(s4.x, s4.y);
  if (max(top & 0xFFFFu, top >> 16) >= 0x6C00u) set_status(d_status, KITTY_ST_RANGE);  // 4096 and more
}

// What a token's scores carry: its Keys are k * 2^key_exp.
template <class F>
__device__ __forceinline__ int key_exp(int lane, bool boosted) {
  const int tau = lane >> 3;
  if (F::W == 2) return boosted ? (tau < 2 ? -2 : 2) : 2 * tau - 4;
  return F::W == 4 ? 4 * (tau & 1) - 4 : 0;
}
// What a channel's outputs carry: its Values are v * 2^value_exp.
template <class F>
__device__ __forceinline__ int value_exp(int lane) {
  const int tau = lane >> 3;
  return F::V == 2 ? 2 * tau - 4 : F::V == 4 ? 4 * (tau & 1) - 4 : 0;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// A page's Values of channel group G, staged at raw: their centered codes times steps to 16 + 16
// lanes of tensor memory at `to` (16 columns), the groups' middles to `mids` ([group][64 bytes]).
template <int V>
__device__ __forceinline__ void put_values(uint32_t raw, uint32_t to, uint32_t mids, int G, int n_hi, int W, int32_t* d_status) {
  const int lane = threadIdx.x & 31, r = lane >> 2, qq = lane & 3;
  uint32_t a[2][8];
  uint32_t top = 0;
  const Codes at16;
  const uint32_t vb = raw + 512 * W + 4 * W * n_hi + 512 + n_hi, vs = vb + 512 * V, vm = vs + 256;
  uint32_t w[V];
  if (V == 2) {
    const uint2 x = lds64(vb + 32 * lane + 8 * G);
    w[0] = x.x;
    w[1] = x.y;
  } else {
    const uint4 x = lds128(vb + 64 * lane + 16 * G);
    w[0] = x.x;
    w[1] = x.y;
    w[2 % V] = x.z;
    w[3 % V] = x.w;
  }
  const uint4 s4 = lds128(vs + 64 * G + 16 * qq), m4 = lds128(vm + 64 * G + 16 * qq);
  const uint32_t S[4] = {s4.x, s4.y, s4.z, s4.w}, M[4] = {m4.x, m4.y, m4.z, m4.w};
  constexpr uint32_t mid = V == 2 ? two(0x3E00) : two(0x4780);  // 1.5, 7.5
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int kt = i >> 1, h = i & 1;
    top = __vmaxu2(top, S[i]);
    uint32_t* o0 = &a[0][2 * i];
    uint32_t* o1 = &a[1][2 * i];
    if (V == 2) {
      const uint32_t x = h ? __funnelshift_r(w[kt], w[kt], 8) : w[kt];
      // 16 + 1.5 * 2^e, e = -4, -2, 0, 2
      o0[0] = h2mul(h2add(at16(x, two(0x000C)), two(0xCC06)), S[i]);
      o0[1] = h2mul(h2add(at16(x, two(0x0030)), two(0xCC18)), S[i]);
      o1[0] = h2mul(h2add(at16(x, two(0x00C0)), two(0xCC60)), S[i]);
      o1[1] = h2mul(h2add(at16(x, two(0x0300)), two(0xCD80)), S[i]);
    } else {
#pragma unroll
      for (int mc = 0; mc < 2; ++mc) {
        const uint32_t y = w[(2 * kt + mc) % V], x = h ? __funnelshift_r(y, y, 8) : y;
        uint32_t* o = mc ? o1 : o0;
        // 16 + 7.5 * 2^e, e = -4, 0
        o[0] = h2mul(h2add(at16(x, two(0x003C)), two(0xCC1E)), S[i]);
        o[1] = h2mul(h2add(at16(x, two(0x03C0)), two(0xCDE0)), S[i]);
      }
    }
  }
  if (r == 0)
    sts128(mids + 64 * G + 16 * qq,
           make_uint4(h2fma(S[0], mid, M[0]), h2fma(S[1], mid, M[1]), h2fma(S[2], mid, M[2]), h2fma(S[3], mid, M[3])));
  tmem_st_frag(to, a[0]);
  tmem_st_frag(to + (16u << 16), a[1]);
  if (max(top & 0xFFFFu, top >> 16) > 0x6FFFu) set_status(d_status, KITTY_ST_RANGE);  // 8192 and more
}

// ------------------------------------------------------------- loose tokens and queries
__device__ __forceinline__ uint32_t to_half2(uint32_t x, int in_dtype) {
  if (in_dtype != KITTY_BF16) return x;
  return h2_bits(__floats2half2_rn(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u)));
}
// Largest magnitudes of two 16-bit values a word, as bits; what they say.
__device__ __forceinline__ uint32_t mag2(uint32_t m, uint32_t x) { return __vmaxu2(m, x & 0x7FFF7FFFu); }
__device__ __forceinline__ int mag_code(uint32_t m, bool packed, int in_dtype) {
  const uint32_t t = max(m & 0xFFFFu, m >> 16);
  if (t >= (in_dtype == KITTY_BF16 ? 0x7F80u : 0x7C00u)) return KITTY_ST_NONFINITE;
  if (packed && in_dtype == KITTY_BF16 && t > 0x477Fu) return KITTY_ST_RANGE;  // 65280: the largest below 65504
  return KITTY_ST_OK;
}

// Two 16-bit values a word, 0 for those that are not numbers.
__device__ __forceinline__ uint32_t numbers2(uint32_t x, int in_dtype) {
  return x & __vcmpltu2(x & 0x7FFF7FFFu, in_dtype == KITTY_BF16 ? two(0x7F80) : two(0x7C00));
}

struct Bars {  // by tile parity
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2];  // operands
  uint64_t sfull[2], sempty[2];
  // by tile: q.M may be two of a pipeline's tiles ahead, the sums one behind (16-bit pages: 0 and 1)
  uint64_t bias[4], bfree[4], pfull[4], pempty[4], mfull[4];
  uint64_t sums, drain;
  uint64_t raw[kMaxRaw], freed[kMaxRaw], loose[2];  // loose[1]: 16-bit pages, room for their Values
};

template <int N>
struct alignas(16) Shared {
  Bars bars;
  uint32_t tmem;
  int abort;
  uint32_t any[2];             // nodes that some node sees
  int loose;                   // parts of the loose tokens that are there
  uint8_t flags[kFlags];       // pages that are there, by tile
  int moved[4];                // by tile: whether its references moved
  float m[2][N], f[2][N];      // by pipeline: reference of each row; factor of its last move
  alignas(16) float bias[4][4][N];   // q.M of each page
  alignas(16) float shift[kSoftmaxWarps][N];
  float top[kSoftmaxWarps][N];       // maxima of a warp's tokens
  alignas(8) float sum[2][N], mid[2][4][N];
  float weight[2][N], total[N];      // of the two pipelines' outputs; a row's sum
  int row[N];                  // output row (token, query head); -1: none
  unsigned long long sees[N];
  uint32_t by[kMaxNodes][2];   // rows that see a node
};

template <class F>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_kernel(const TreeParams p, const __grid_constant__ CUtensorMap map) {
  using Z = Sizes<F>;
  constexpr int N = F::N;
  extern __shared__ uint8_t dyn[];
  __shared__ Shared<N> sh;
  grid_trigger();
  const int tid = threadIdx.x, lane = tid & 31;
  const int wid = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int unit = blockIdx.x % p.units, pair = blockIdx.x / p.units, kvh = pair % p.Hkv, b = pair / p.Hkv;
  const int split = blockIdx.y;
  const Held hd = held_of<F::kPacked>(p, b);
  const int R = min(N, hd.n * p.g - unit * N);  // rows of this block
  if (hd.code != KITTY_ST_OK && unit == 0 && split == 0 && kvh == 0 && tid == 0) set_status(p.d_status, hd.code);
  // behind a prefix kernel, which may still run: the last block ends after it, and so does this grid
  auto end_behind = [&] {
    if (p.slots > 0 && blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1) grid_wait();
  };
  if (!hd.ok || R <= 0) {
    end_behind();
    return;
  }
  const int pages = hd.prefix + hd.pages, tiles = (pages + kTilePages - 1) / kTilePages + 1;
  const int t0 = (int)((long)tiles * split / p.splits), n = (int)((long)tiles * (split + 1) / p.splits) - t0;
  // row x of the block: output row; node
  auto out_row = [&](int x) {
    const int i = unit * N + x, node = i / p.g;
    return (hd.first + node) * p.Hq + kvh * p.g + (i - node * p.g);
  };
  if (n == 0) {
    if (tid < R) p.ws[((size_t)out_row(tid) * p.splits + split) * kPartialFloats] = -INFINITY;
    end_behind();
    return;
  }
  const bool has_loose = t0 + n == tiles;
  volatile int* abort = &sh.abort;
  const uint32_t base = (smem_u32(dyn) + 1023u) & ~1023u;
  const uint32_t qs = base, ps = qs + Z::kQ, ops = ps + Z::kPs * Z::kP;  // ops: 16-bit tiles (Keys, then Values)
  const uint32_t loose = ops, spread = loose + 2 * kLoose * kLoosePitch, mids = spread + 8 * Z::kSpread;
  const uint32_t raws = mids + 4 * 1024;
  Bars& bar = sh.bars;
  auto a_of = [&](uint64_t& x) { return smem_u32(&x); };
  // place of tile i's p (and q.M, middles), and the parity of its use
  constexpr int kP2 = Z::kPs == 4 ? 2 : 1;
  auto at4 = [&](int i) { return i & (Z::kPs - 1); };
  auto turn4 = [&](int i) { return (i >> kP2) & 1; };
  auto wait = [&](uint64_t& x, int parity) { return wait_phase(x, parity, p.wait_polls, abort); };
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.kfull[i], F::kPacked ? 4 : 1);
      mbar_init(&bar.vfull[i], F::kPacked ? 4 : 1);
      mbar_init(&bar.kempty[i], 1);
      mbar_init(&bar.vempty[i], 1);
      mbar_init(&bar.sfull[i], 1);
      mbar_init(&bar.sempty[i], 4);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar.bias[i], 1);
      mbar_init(&bar.bfree[i], 4);
      mbar_init(&bar.pfull[i], 4);
      mbar_init(&bar.pempty[i], 3);  // the products, and the sums of each half of the rows
      mbar_init(&bar.mfull[i], 4);
    }
    mbar_init(&bar.sums, 4);
    mbar_init(&bar.drain, 1);
    for (int i = 0; i < kMaxRaw; ++i) {
      mbar_init(&bar.raw[i], 1);
      mbar_init(&bar.freed[i], 9);
    }
    mbar_init(&bar.loose[0], 1);
    mbar_init(&bar.loose[1], 1);
    fence_mbar_init();
    sh.abort = 0;
    sh.any[0] = sh.any[1] = 0;
  }
  if (wid == kMmaWarp) tmem_alloc(smem_u32(&sh.tmem), 512);
  // ---- queries: 16 threads a row, zeros behind the last
  {
    uint32_t mag = 0;
    for (int i = tid; i < N * 16; i += kTreeThreads) {
      const int x = i >> 4, c = i & 15;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (x < R) {
        const int y = unit * N + x, node = y / p.g;
        v = *reinterpret_cast<const uint4*>(p.q + (size_t)(hd.first + node) * p.q_stride + ((size_t)kvh * p.g + y - node * p.g) * kD + 8 * c);
        mag = mag2(mag2(mag2(mag2(mag, v.x), v.y), v.z), v.w);
        if (F::kPacked) v = make_uint4(to_half2(v.x, p.in_dtype), to_half2(v.y, p.in_dtype), to_half2(v.z, p.in_dtype), to_half2(v.w, p.in_dtype));
      }
      sts128(qs + (c >> 3) * Z::kQHalf + x * 128 + (((c & 7) ^ (x & 7)) << 4), v);
    }
    fence_async_shared();
    const int code = mag_code(mag, F::kPacked, p.in_dtype);
    // (by the split that takes the loose tokens: it alone has tiles in every sequence, however short)
    if (has_loose && code != KITTY_ST_OK) set_status(p.d_status, code);
  }
  // the ids of this block's first eight tiles of pages, for the warps that request them
  int first_ids = -1;
  if (wid == kFetchWarp || (!F::kPacked && wid == kBiasWarp)) {
    const int x = t0 * kTilePages + lane;
    if (x < pages && lane / kTilePages < n)
      first_ids = x < hd.prefix ? p.prefix_table[x] : p.block_table[(size_t)b * p.max_pages + x - hd.prefix];
  }
  if (tid < N) {
    sh.row[tid] = tid < R ? out_row(tid) : -1;
    sh.m[0][tid] = sh.m[1][tid] = kFloor;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sh.tmem, 0);
  if (has_loose) {  // which nodes each row sees, and which any row does
    const unsigned long long all = hd.n == 64 ? ~0ull : (1ull << hd.n) - 1;
    auto sees = [&](int node) { return (p.visible != nullptr ? p.visible[hd.first + node] : node == 63 ? ~0ull : (2ull << node) - 1) & all; };
    if (tid < N) sh.sees[tid] = tid < R ? sees((unit * N + tid) / p.g) : 0;
    if (tid >= 128 && tid < 128 + hd.n) {
      const unsigned long long s = sees(tid - 128);
      atomicOr(&sh.any[0], (uint32_t)s);
      atomicOr(&sh.any[1], (uint32_t)(s >> 32));
    }
    if (tid == 0) {
      int there = 2 | (hd.n > 32 ? 4 : 0);
      if (hd.loose > 0) {
        const int id = F::kPacked ? 0 : p.block_table[(size_t)b * p.max_pages + hd.pages];
        if (id >= 0 && (F::kPacked || id < p.pool_pages)) there |= 1;
        else set_status(p.d_status, KITTY_ST_BAD_PAGE);
      }
      sh.loose = there;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMaxNodes / (kTreeThreads / 32); ++k) {  // a row a lane
      const int j = wid * (kMaxNodes / (kTreeThreads / 32)) + k;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int x = 32 * half + lane;
        const uint32_t rows = __ballot_sync(0xFFFFFFFFu, x < N && ((sh.sees[x % N] >> j) & 1ull) != 0);
        if (lane == 0) sh.by[j][half] = rows;
      }
    }
    __syncthreads();
  }
  // loose part g (32 tokens: the tail, nodes 0.., nodes 32..): how many of them there are
  auto loose_count = [&](int g) { return g == 0 ? hd.loose : min(max(hd.n - 32 * (g - 1), 0), g < 3 ? 32 : 0); };
  // somebody sees token i of part g
  auto loose_seen = [&](int g, int i) {
    return i < loose_count(g) && (g == 0 || ((sh.any[g == 1 ? 0 : 1] >> i) & 1u) != 0);
  };
  // pages of tile i, or parts of the loose tokens, that are there
  auto there_of = [&](int i) { return has_loose && i == n - 1 ? sh.loose : (int)sh.flags[i % kFlags]; };
  const uint32_t quad = (uint32_t)(32 * (wid & 3)) << 16;
  int issued = 0;  // tiles whose copies this warp has requested

  if (wid < kSoftmaxWarps) {
    // =========================================================== softmax
    const int h = wid >> 2, g = wid & 3, id = 1 + h;
    const float sc = p.sm_log2;
    const float sc_page = F::kPacked ? sc * pow2(-key_exp<F>(lane, p.n_hi > 0)) : sc;
    const uint32_t shift_at = smem_u32(sh.shift[wid]);
    const int token = 32 * g + lane;
    const uint32_t prow0 = ps + token * 128, S = tmem + Z::kSCol + h * N + quad;
    const int node = (token - 32) & 63;  // of a loose token that is one (masked: in range for the others, too)
    constexpr int U = F::kPacked ? 16 : N < 32 ? N : 32;  // rows at a time
    // what is added to each row's scaled score: q.M of the page, less the reference
    auto fill = [&](int i, bool with_m) {
      __syncwarp();
#pragma unroll
      for (int c = lane; c < N; c += 32) {
        const float bias = F::kPacked ? sh.bias[i & 3][g][c] * sc : 0.f;
        sts32(shift_at + 4 * c, with_m ? bias - sh.m[h][c] : bias);  // read by lds128 alone
      }
      __syncwarp();
    };
    bool ok = true;
    for (int i = h; i < n; i += 2) {
      const int u = (i >> 1) & 1;
      ok = !F::kPacked || wait(bar.bias[i & 3], (i >> 2) & 1);
      fill(i, true);
      ok = ok && wait(bar.pempty[at4(i)], turn4(i) ^ 1) && wait(bar.sfull[h], u);
      const uint32_t prow = prow0 + at4(i) * Z::kP;
      tc_fence_after();
      const bool special = has_loose && i == n - 1;
      const bool there = (there_of(i) >> g) & 1, masks = special && there;
      uint32_t see[2] = {~0u, ~0u};  // rows that see this thread's token
      if (masks && (g > 0 || lane >= hd.loose)) {
        see[0] = g > 0 ? sh.by[node][0] : 0;
        see[1] = g > 0 ? sh.by[node][1] : 0;
      }
      const float scl = special ? sc : sc_page;
      // U rows' scores from tensor memory: scaled, shifted, masked
      auto scores = [&](int c0, uint32_t (&x)[U]) {
        tmem_load<U>(S + c0, x);
        const uint64_t scl2 = f2pack(scl, scl);
#pragma unroll
        for (int c = 0; c < U; c += 4) {
          const uint4 s4 = lds128(shift_at + 4 * (c0 + c));
          fma2(x[c], x[c + 1], scl2, s4.x, s4.y);
          fma2(x[c + 2], x[c + 3], scl2, s4.z, s4.w);
        }
        if (masks) {
          const uint32_t on = (c0 < 32 ? see[0] : see[1]) >> (c0 & 31);
#pragma unroll
          for (int c = 0; c < U; ++c)
            if (((on >> c) & 1u) == 0) x[c] = __float_as_uint(-INFINITY);
        }
      };
      bool moves = false, leave = false;
      for (int pass = 0;; ++pass) {
        // p of the tile by the references as they are (a token that is not there is not multiplied)
        float top = -INFINITY;
        if (there) {
#pragma unroll 1
          for (int c0 = 0; c0 < N; c0 += U) {
            uint32_t x[U];
            scores(c0, x);
#pragma unroll
            for (int c = 0; c < U; c += 2) top = fmaxf(fmaxf(top, __uint_as_float(x[c])), __uint_as_float(x[c + 1]));
#pragma unroll
            for (int c = 0; c < U; c += 8) {
              uint32_t w[4], rest[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float e0 = ex2a(__uint_as_float(x[c + 2 * k])), e1 = ex2a(__uint_as_float(x[c + 2 * k + 1]));
                if (F::kBf16) {
                  const __nv_bfloat162 y = __floats2bfloat162_rn(e0, e1);
                  w[k] = *reinterpret_cast<const uint32_t*>(&y);
                  const __nv_bfloat162 z = __floats2bfloat162_rn(e0 - __uint_as_float(w[k] << 16), e1 - __uint_as_float(w[k] & 0xFFFF0000u));
                  rest[k] = *reinterpret_cast<const uint32_t*>(&z);
                } else {
                  const __half2 y = __floats2half2_rn(e0, e1);
                  w[k] = h2_bits(y);
                  if (F::kPair) {
                    const float2 z = __half22float2(y);
                    rest[k] = h2_bits(__floats2half2_rn(e0 - z.x, e1 - z.y));
                  }
                }
              }
              const uint32_t at = prow + ((((c0 + c) / 8) ^ (token & 7)) << 4);
              sts128(at, make_uint4(w[0], w[1], w[2], w[3]));
              if (F::kPair) sts128(at + Z::kPHalf, make_uint4(rest[0], rest[1], rest[2], rest[3]));
            }
          }
        }
        // a score that passes its reference by too much (always to be set at the first tile): the
        // group moves the references, and the tile's p are formed again
        if (pass == 1 || !group_any(id, i == h || top > kSlack || !ok)) break;
        // (a move is of what the tiles before have left: their products and sums are done, then)
        if (i > h) ok = ok && wait(bar.pempty[at4(i - 2)], turn4(i - 2));
        leave = group_any(id, !ok);
        if (leave) break;
        fill(i, false);
#pragma unroll 1
        for (int c0 = 0; c0 < N; c0 += U) {
          uint32_t x[U];
          scores(c0, x);
#pragma unroll
          for (int c = 0; c < U; ++c) {
            const float mx = warp_max(there ? __uint_as_float(x[c]) : -INFINITY);
            if (lane == 0) sh.top[wid][c0 + c] = mx;
          }
        }
        group_sync(id);
        const int c = tid & 127;  // a thread a row
        if (c < N) {
          const float mx = fmaxf(fmaxf(sh.top[4 * h][c], sh.top[4 * h + 1][c]), fmaxf(sh.top[4 * h + 2][c], sh.top[4 * h + 3][c]));
          const float m = sh.m[h][c];
          const bool set = (i == h && mx > kFloor) || mx > m + kSlack;
          const float nm = set ? mx + kMargin : m;
          sh.m[h][c] = nm;
          sh.f[h][c] = i > h && set ? ex2a(m - nm) : 1.f;
          moves = i > h && set;
        }
        moves = group_any(id, moves);
        if (moves) {  // the outputs so far
          tc_fence_after();
          const uint32_t O = tmem + Z::kOCol + h * N + quad;
#pragma unroll 1
          for (int k0 = 0; k0 < N; k0 += 8) {
            uint32_t y[8];
            tmem_load<8>(O + k0, y);
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * sh.f[h][k0 + k]);
            tmem_st8(O + k0, y);
          }
          tmem_wait_st();
        }
        fill(i, true);
      }
      if (leave) {
        ok = false;
        break;
      }
      if (lane == 0 && g == 0) sh.moved[at4(i)] = moves;
      // the scores and their bias have been read, p is written
      tc_fence_before();
      fence_async_shared();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_s(a_of(bar.sempty[h]));
        if (F::kPacked) mbar_arrive_s(a_of(bar.bfree[i & 3]));
        mbar_arrive_s(a_of(bar.pfull[at4(i)]));
      }
    }
    // ---- the last products and sums; then the weights of the two pipelines' outputs
    const int last = n - 1 - ((n - 1 - h) & 1);  // this one's last tile, if it has one
    if (ok) ok = (last < 0 || wait(bar.pempty[at4(last)], turn4(last))) && wait(bar.sums, 0);
    tc_fence_after();
    if (ok && wid < 2 && tid < N) {
      const float l0 = sh.sum[0][tid], l1 = n > 1 ? sh.sum[1][tid] : 0.f;
      const float m0 = l0 != 0.f ? sh.m[0][tid] : -INFINITY, m1 = l1 != 0.f ? sh.m[1][tid] : -INFINITY, m = fmaxf(m0, m1);
      const float w0 = l0 != 0.f ? ex2a(m0 - m) : 0.f, w1 = l1 != 0.f ? ex2a(m1 - m) : 0.f;
      sh.weight[0][tid] = w0;
      sh.weight[1][tid] = w1;
      sh.total[tid] = (l0 != 0.f ? l0 * w0 : 0.f) + (l1 != 0.f ? l1 * w1 : 0.f);
      sh.m[0][tid] = m;
    }
    // all eight warps come here: both pipelines have ended, or none goes on
    uint32_t failed;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "barrier.cta.red.or.pred p, 5, 256, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(failed)
        : "r"((uint32_t)!ok)
        : "memory");
    if (failed == 0) {
      // ---- outputs or partials: a thread a channel, a warp 32 channels of each row of its half
      tc_fence_after();
      const float scale = F::kPacked ? pow2(-value_exp<F>(lane)) : 1.f;
      const int ch = 32 * g + lane;
      bool empty = false;
#pragma unroll 1
      for (int c = h * (N / 2); c < (h + 1) * (N / 2) && c < R; c += 8) {
        uint32_t x[8], x1[8];
        tmem_load<8>(tmem + Z::kOCol + c + quad, x);
        tmem_load<8>(tmem + Z::kOCol + N + c + quad, x1);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int y = c + k, row = sh.row[y];
          if (row < 0) continue;
          // (a weight of 0: that pipeline's outputs may be anything)
          const float l = sh.total[y], w0 = sh.weight[0][y], w1 = sh.weight[1][y];
          float o = 0.f;
          if (w0 != 0.f) o = (__uint_as_float(x[k]) * scale + (F::kPacked ? sh.mid[0][g][y] : 0.f)) * w0;
          if (w1 != 0.f) o += (__uint_as_float(x1[k]) * scale + (F::kPacked ? sh.mid[1][g][y] : 0.f)) * w1;
          if (p.direct) {
            const float v = l != 0.f ? o / l : 0.f;
            const size_t at = (size_t)row * kD + ch;
            if (p.out_dtype == KITTY_F32) static_cast<float*>(p.out)[at] = v;
            else if (p.out_dtype == KITTY_BF16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
            else static_cast<__half*>(p.out)[at] = __float2half_rn(v);
            empty = empty || l == 0.f;
          } else {
            float* part = p.ws + ((size_t)row * p.splits + split) * kPartialFloats;
            part[4 + ch] = o;
            if (ch == 0) *reinterpret_cast<float2*>(part) = make_float2(l != 0.f ? sh.m[0][y] : -INFINITY, l);
          }
        }
      }
      if (empty && ch == 0) set_status(p.d_status, KITTY_ST_EMPTY);
      tc_fence_before();
    } else if (lane == 0) {
      set_status(p.d_status, KITTY_ST_TIMEOUT);
    }
  } else if (wid < kBiasWarp) {
    // =========================================================== operands
    const bool keys = wid < kValueWarp;
    const int g = wid & 3;
    bool ok = true;
    if constexpr (F::kPacked) {
      const int h = (wid >> 2) & 1;
      int slot = h, turn = 0;
      for (int i = h; i < n; i += 2) {
        const int u = (i >> 1) & 1;
        const bool special = has_loose && i == n - 1;
        ok = wait(special ? bar.loose[0] : bar.raw[slot], special ? 0 : turn & 1) && wait(keys ? bar.kempty[h] : bar.vempty[h], u ^ 1);
        if (!keys) ok = ok && wait(bar.pempty[at4(i)], turn4(i) ^ 1);  // the middles' place
        if (!ok) break;
        tc_fence_after();
        const uint32_t to = tmem + (keys ? 0 : 128) + 64 * h + quad;
        if (!special) {
          const uint32_t raw = raws + slot * (kTilePages * p.blob);
          const int there = sh.flags[i % kFlags];
          if (keys) {
            if ((there >> g) & 1) put_keys<F::W>(raw + g * p.blob, to, spread + (wid - kKeyWarp) * Z::kSpread, p.n_hi, p.d_status);
          } else {
#pragma unroll 1
            for (int x = 0; x < kTilePages; ++x)
              if ((there >> x) & 1) put_values<F::V>(raw + x * p.blob, to + 16 * x, mids + at4(i) * 1024 + 256 * x, g, p.n_hi, F::W, p.d_status);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_s(a_of(bar.freed[slot]));
          slot += 2;
          if (slot >= p.raw_stages) {
            slot -= p.raw_stages;
            ++turn;
          }
        } else if (keys) {
          // a thread a token
          uint32_t mag = 0;
          const uint32_t src = loose + (32 * g + lane) * kLoosePitch;
          if (loose_count(g) > 0) {
#pragma unroll 1
            for (int x = 0; x < 4; ++x) {
              uint32_t w[16];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint4 v = lds128(src + 64 * x + 16 * k);
                mag = mag2(mag2(mag2(mag2(mag, v.x), v.y), v.z), v.w);
                w[4 * k] = to_half2(v.x, p.in_dtype);
                w[4 * k + 1] = to_half2(v.y, p.in_dtype);
                w[4 * k + 2] = to_half2(v.z, p.in_dtype);
                w[4 * k + 3] = to_half2(v.w, p.in_dtype);
              }
              tmem_st16(to + 16 * x, w);
            }
            const int code = mag_code(mag, true, p.in_dtype);
            if (code != KITTY_ST_OK && loose_seen(g, lane)) set_status(p.d_status, code);
          }
        } else {
          // a thread a channel; what no one sees, or fp16 cannot hold (beyond 16376), is 0
          const float up = pow2(value_exp<F>(lane));
          const uint32_t most = p.in_dtype == KITTY_BF16 ? 0x467Fu : 0x73FFu;
          uint32_t top = 0;  // the largest, as bits
#pragma unroll 1
          for (int x = 0; x < 6; ++x) {  // 16 tokens
            const int part = x >> 1, count = loose_count(part);
            if (count == 0) continue;
            const uint32_t seen = (part == 0 ? 0xFFFFFFFFu : sh.any[part - 1]) & (count < 32 ? (1u << count) - 1 : 0xFFFFFFFFu);
            const uint32_t on = seen >> (16 * (x & 1)), src = loose + (kLoose + 16 * x) * kLoosePitch + 2 * (32 * g + lane);
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              float f[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t v = ((on >> (2 * k + e)) & 1u) != 0 ? lds16(src + (2 * k + e) * kLoosePitch) : 0u;
                top = max(top, v & 0x7FFFu);
                f[e] = (v & 0x7FFFu) <= most ? bits16_to_f32((uint16_t)v, p.in_dtype) : 0.f;
              }
              w[k] = h2_bits(__floats2half2_rn(f[0] * up, f[1] * up));
            }
            tmem_st8(to + 8 * x, w);
            if (lane < 4) sts128(mids + at4(i) * 1024 + 256 * part + 64 * g + 16 * lane, make_uint4(0, 0, 0, 0));
          }
          if (top > most)
            set_status(p.d_status, top >= (p.in_dtype == KITTY_BF16 ? 0x7F80u : 0x7C00u) ? KITTY_ST_NONFINITE : KITTY_ST_RANGE);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_s(keys ? a_of(bar.kfull[h]) : a_of(bar.vfull[h]));
          if (!keys) mbar_arrive_s(a_of(bar.mfull[at4(i)]));
        }
      }
    } else if (has_loose) {
      // the loose tokens' rows, swizzled as the tiled loads leave the others: 8 lanes a row half
      const int i = n - 1, st = i & 1;
      ok = wait(bar.loose[keys ? 0 : 1], 0);
      const uint32_t to = ops + (2 * st + (keys ? 0 : 1)) * Z::kTile16;
      if (ok) {
        int code = KITTY_ST_OK;
        const bool in = (sh.loose & 1) != 0;
        const int id = in ? p.block_table[(size_t)b * p.max_pages + hd.pages] : 0;
        const uint16_t* page = reinterpret_cast<const uint16_t*>(p.pool) + (((size_t)id * p.Hkv + kvh) * 2 + (keys ? 0 : 1)) * kPage * kD;
        const uint16_t* nodes = (keys ? p.k : p.v) + (size_t)hd.first * (keys ? p.k_stride : p.v_stride) + (size_t)kvh * kD;
        const size_t stride = keys ? p.k_stride : p.v_stride;
#pragma unroll 1
        for (int k0 = 0; k0 < kLoose * 16; k0 += 3 * 256) {
          uint4 v[3];
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const int at = k0 + 256 * k + (tid & 255), t = at >> 4, c = at & 15, part = t >> 5;
            const bool on = t < kLoose && (part == 0 ? (t & 31) < hd.loose && in : loose_seen(part, t & 31));
            v[k] = on ? *reinterpret_cast<const uint4*>((part == 0 ? page + (size_t)t * kD : nodes + (size_t)(t - 32) * stride) + 8 * c)
                      : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const int at = k0 + 256 * k + (tid & 255), t = at >> 4, c = at & 15;
            if (t >= 32) {  // elements that are not numbers: reported, and 0, so that they reach no one
              const int e = mag_code(mag2(mag2(mag2(mag2(0, v[k].x), v[k].y), v[k].z), v[k].w), false, p.in_dtype);
              if (e != KITTY_ST_OK) {
                code = e;
                v[k] = make_uint4(numbers2(v[k].x, p.in_dtype), numbers2(v[k].y, p.in_dtype), numbers2(v[k].z, p.in_dtype),
                                  numbers2(v[k].w, p.in_dtype));
              }
            }
            if (t < kLoose) sts128(to + (c >> 3) * Z::kHalf16 + t * 128 + (((c & 7) ^ (t & 7)) << 4), v[k]);
          }
        }
        if (code != KITTY_ST_OK) set_status(p.d_status, code);
      }
      fence_async_shared();
      asm volatile("barrier.cta.sync %0, 256;" ::"r"(keys ? 3 : 4) : "memory");
      if (ok && (tid & 255) == 0) mbar_arrive_s(keys ? a_of(bar.kfull[st]) : a_of(bar.vfull[st]));
    }
    if (!ok && lane == 0) set_status(p.d_status, KITTY_ST_TIMEOUT);
    __syncwarp();
  } else if (wid == kMmaWarp) {
    // =========================================================== products
    constexpr uint32_t qk = mma_desc(F::kBf16, false, N);
    constexpr uint32_t pv = mma_desc(F::kBf16, true, N) | (F::kPacked ? 0u : 1u << 15);  // 16-bit Values: channels contiguous
    const uint64_t qdesc = smem_desc(qs, 16, 1024, kSwizzle128);
    const uint64_t pdesc = smem_desc(ps, Z::kPHalf, 1024, kSwizzle128);
    bool ok = true;
    int started = 0;  // pipelines whose outputs have been begun
    auto scores = [&](int i) {
      const int st = i & 1;
      ok = wait(bar.kfull[st], (i >> 1) & 1) && wait(bar.sempty[st], ((i >> 1) & 1) ^ 1);
      if (!ok) return;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t d = tmem + Z::kSCol + st * N;
#pragma unroll
        for (int k = 0; k < kD / 16; ++k) {
          const uint64_t qd = qdesc + (k >> 2) * (Z::kQHalf / 16) + 2 * (k & 3);
          if constexpr (F::kPacked) {
            mma_ts(d, tmem + 64 * st + 8 * k, qd, qk, k > 0);
          } else {
            const uint64_t kd = smem_desc(ops + 2 * st * Z::kTile16, 16, 1024, kSwizzle128);
            mma_ss(d, kd + (k >> 2) * (Z::kHalf16 / 16) + 2 * (k & 3), qd, qk, k > 0);
          }
        }
        mma_commit(a_of(bar.sfull[st]));
        mma_commit(a_of(bar.kempty[st]));
      }
      __syncwarp();
    };
    scores(0);
    for (int i = 0; ok && i < n; ++i) {
      const int st = i & 1;
      if (i + 1 < n) {
        scores(i + 1);
        if (!ok) break;
      }
      ok = wait(bar.vfull[st], (i >> 1) & 1) && wait(bar.pfull[at4(i)], turn4(i));
      if (!ok) break;
      tc_fence_after();
      const int there = there_of(i);
      if (elect_one()) {
        const uint32_t d = tmem + Z::kOCol + st * N, v = tmem + 128 + 64 * st;
        const uint64_t pd = pdesc + at4(i) * (Z::kP / 16);
        const uint64_t vd = smem_desc(ops + (2 * st + 1) * Z::kTile16, Z::kHalf16, 1024, kSwizzle128);
        auto product = [&](int k, bool acc) {  // 16 tokens
          if constexpr (F::kPacked) {
            mma_ts(d, v + 8 * k, pd + 128 * k, pv, acc);
          } else {
            mma_ss(d, vd + 128 * k, pd + 128 * k, pv, acc);
            mma_ss(d, vd + 128 * k, pd + Z::kPHalf / 16 + 128 * k, pv, true);
          }
        };
        const bool begun = (started >> st) & 1;
        if (there == 15) {
#pragma unroll
          for (int k = 0; k < 8; ++k) product(k, begun || k > 0);
        } else {
          bool acc = begun;
#pragma unroll 1
          for (int k = 0; k < 8; ++k)
            if ((there >> (k >> 1)) & 1) {
              product(k, acc);
              acc = true;
            }
        }
        mma_commit(a_of(bar.vempty[st]));
        mma_commit(a_of(bar.pempty[at4(i)]));
      }
      if (there != 0) started |= 1 << st;
      __syncwarp();
    }
    if (!ok && lane == 0) set_status(p.d_status, KITTY_ST_TIMEOUT);
    __syncwarp();
  } else if (!F::kPacked && (wid == kFetchWarp || wid == kBiasWarp)) {
    // =========================================================== tiled loads: a warp the Keys', one the Values'
    const bool values = wid != kFetchWarp;
    bool ok = true;
    int ids = -1;  // lane l: the id of page l of the eight tiles at hand
    for (int i = 0; i < n; ++i) {
      const int st = i & 1;
      const uint32_t full = values ? a_of(bar.vfull[st]) : a_of(bar.kfull[st]);
      ok = wait(values ? bar.vempty[st] : bar.kempty[st], ((i >> 1) & 1) ^ 1);
      if (!ok) break;
      if (has_loose && i == n - 1) {  // room for the loose tokens: this warp has followed every use of the stage
        if (elect_one()) mbar_arrive_s(a_of(bar.loose[values ? 1 : 0]));
        break;
      }
      if ((i & 7) == 0) {
        const int x = (t0 + i) * kTilePages + lane;
        ids = i == 0 ? first_ids : x >= pages ? -1 : x < hd.prefix ? p.prefix_table[x] : p.block_table[(size_t)b * p.max_pages + x - hd.prefix];
        if (ids < 0 || ids >= p.pool_pages) {
          if (!values && x < min(pages, (t0 + n) * kTilePages)) set_status(p.d_status, KITTY_ST_BAD_PAGE);
          ids = -1;
        }
      }
      int id[kTilePages], there = 0;
#pragma unroll
      for (int g = 0; g < kTilePages; ++g) {
        id[g] = __shfl_sync(0xFFFFFFFFu, ids, kTilePages * (i & 7) + g);
        there |= (id[g] >= 0 ? 1 : 0) << g;
      }
      if (elect_one()) {  // one thread requests all of a tile's boxes
        if (!values) sh.flags[i % kFlags] = (uint8_t)there;
        mbar_arrive_expect_tx_s(full, (uint32_t)(__popc(there) * kPage * kD * 2));
        const uint32_t to = ops + (2 * st + (values ? 1 : 0)) * Z::kTile16;
#pragma unroll
        for (int g = 0; g < kTilePages; ++g)
          if (id[g] >= 0) {
            const int y = (id[g] * p.Hkv + kvh) * 2 * kPage + (values ? kPage : 0);
            tma_load_2d(to + g * kPage * 128, &map, 0, y, full);
            tma_load_2d(to + Z::kHalf16 + g * kPage * 128, &map, 64, y, full);
          }
      }
      issued = i + 1;
      __syncwarp();
    }
    if (!ok && lane == 0) set_status(p.d_status, KITTY_ST_TIMEOUT);
    __syncwarp();
  } else if (wid == kFetchWarp) {
    // =========================================================== copies
    bool ok = true;
    if (F::kPacked && has_loose) {  // the loose tokens' rows first: nobody frees their place
      const int total = hd.loose + hd.n;
      if (lane == 0) mbar_arrive_expect_tx_s(a_of(bar.loose[0]), (uint32_t)(total * 2 * kD * 2));
      __syncwarp();
      for (int x = lane; x < 2 * total; x += 32) {
        const int t = x >> 1;
        const bool tail = t < hd.loose;
        const uint16_t* src;
        if (x & 1) src = tail ? p.tail_v + (((size_t)b * p.Hkv + kvh) * kPage + t) * kD : p.v + (size_t)(hd.first + t - hd.loose) * p.v_stride + (size_t)kvh * kD;
        else src = tail ? p.tail_k + (((size_t)b * p.Hkv + kvh) * kPage + t) * kD : p.k + (size_t)(hd.first + t - hd.loose) * p.k_stride + (size_t)kvh * kD;
        bulk_g2s_s(loose + ((x & 1) * kLoose + (tail ? t : 32 + t - hd.loose)) * kLoosePitch, src, kD * 2, a_of(bar.loose[0]));
      }
      __syncwarp();
    }
    int ids = -1, ids_at = 0, slot = 0, turn = 0;
    for (int i = 0; i < n; ++i) {
      const bool special = has_loose && i == n - 1;
      if (special) break;
      if (i == 0 || i - ids_at >= 8) {  // page ids of eight tiles
        ids_at = i;
        const int x = (t0 + i) * kTilePages + lane;
        ids = i == 0 ? first_ids : x >= pages || (i + lane / 4) >= n ? -1 : x < hd.prefix ? p.prefix_table[x] : p.block_table[(size_t)b * p.max_pages + x - hd.prefix];
      }
      const int id = __shfl_sync(0xFFFFFFFFu, ids, 4 * (i - ids_at) + (lane & 3));
      const bool in = id >= 0 && id < p.pool_pages;
      const int there = __ballot_sync(0xFFFFFFFFu, in) & 15;
      if (lane < 4 && !in && (t0 + i) * kTilePages + lane < pages) set_status(p.d_status, KITTY_ST_BAD_PAGE);
      if constexpr (F::kPacked) {
        ok = wait(bar.freed[slot], (turn & 1) ^ 1);
        if (!ok) break;
        const uint32_t full = a_of(bar.raw[slot]);
        if (lane == 0) {
          sh.flags[i % kFlags] = (uint8_t)there;
          mbar_arrive_expect_tx_s(full, (uint32_t)(__popc(there) * p.blob));
        }
        __syncwarp();
        if (lane < 4 && in)
          bulk_g2s_s(raws + (slot * kTilePages + lane) * p.blob, p.pool + ((size_t)id * p.Hkv + kvh) * p.blob, (uint32_t)p.blob, full);
        if (++slot == p.raw_stages) {
          slot = 0;
          ++turn;
        }
      }
      issued = i + 1;
      __syncwarp();
    }
    if (!ok && lane == 0) set_status(p.d_status, KITTY_ST_TIMEOUT);
    __syncwarp();
  } else if (wid < kSumWarp) {
    // =========================================================== q.M: a page a row of the product
    if constexpr (F::kPacked) {
      constexpr int T = N / 8;  // tiles of eight rows
      const int h = wid - kBiasWarp, r = lane >> 2, qq = lane & 3;
      // eight rows' 32 channels of the queries: a matrix of eight channels a quarter warp
      const uint32_t q_at[2] = {qs + (lane & 7) * 128 + (((lane >> 3) ^ (lane & 7)) << 4),
                                qs + (lane & 7) * 128 + (((4 + (lane >> 3)) ^ (lane & 7)) << 4)};
      bool ok = true;
      int slot = h, turn = 0;
      for (int i = h; i < n; i += 2) {
        const bool special = has_loose && i == n - 1;
        ok = (special || wait(bar.raw[slot], turn & 1)) && wait(bar.bfree[i & 3], ((i >> 2) & 1) ^ 1);
        if (!ok) break;
        if (special) {
          for (int x = lane; x < 4 * N; x += 32) (&sh.bias[i & 3][0][0])[x] = 0.f;
        } else {
          uint32_t M[16];
          const uint32_t at = raws + (slot * kTilePages + (r & 3)) * p.blob + 512 * F::W + 4 * F::W * p.n_hi + 256 + 64 * qq;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 v = r < 4 ? lds128(at + 16 * k) : make_uint4(0, 0, 0, 0);
            M[4 * k] = v.x;
            M[4 * k + 1] = v.y;
            M[4 * k + 2] = v.z;
            M[4 * k + 3] = v.w;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_s(a_of(bar.freed[slot]));
          slot += 2;
          if (slot >= p.raw_stages) {
            slot -= p.raw_stages;
            ++turn;
          }
#pragma unroll 1
          for (int nt = 0; nt < T; ++nt) {
            float x[4], y[4];
#pragma unroll
            for (int jp = 0; jp < 4; ++jp) {
              uint32_t q4[4];
              ldsm_x4(q_at[jp & 1] + (jp >> 1) * Z::kQHalf + nt * 1024, q4);
              const uint32_t a0[4] = {M[4 * jp], 0u, M[4 * jp + 1], 0u}, a1[4] = {M[4 * jp + 2], 0u, M[4 * jp + 3], 0u};
              if (jp == 0) {
                mma_rows8(x, M[0], M[1], q4[0], q4[1]);
                mma_rows8(y, M[2], M[3], q4[2], q4[3]);
                continue;
              }
              mma_f16(x, a0, q4[0], q4[1]);
              mma_f16(y, a1, q4[2], q4[3]);
            }
            if (r < 4) *reinterpret_cast<float2*>(&sh.bias[i & 3][r][8 * nt + 2 * qq]) = make_float2(x[0] + y[0], x[1] + y[1]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_s(a_of(bar.bias[i & 3]));
      }
      if (!ok && lane == 0) set_status(p.d_status, KITTY_ST_TIMEOUT);
    }
    __syncwarp();
  } else {
    // =========================================================== sums of p and of p * middles
    constexpr int T = N < 32 ? 2 : N / 16;  // tiles of eight rows of a warp
    const int h = (wid - kSumWarp) & 1, n0 = (wid - kSumWarp) / 2 * T, r = lane >> 2, qq = lane & 3;
    const bool mine = n0 * 8 < N;  // (16 rows are one warp's)
    bool ok = true;
    float c[T][4];  // (rows 8 .. 15 of the product are zeros)
#pragma unroll
    for (int nt = 0; nt < T; ++nt) c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.f;
    constexpr uint32_t one = F::kBf16 ? two(0x3F80) : two(0x3C00);
    // 16 tokens' p of 16 rows (two chunks of a token's 64): matrices of eight by eight
    uint32_t p_at[T / 2];
#pragma unroll
    for (int np = 0; np < T / 2; ++np)
      p_at[np] = ps + (8 * ((lane >> 3) & 1) + (lane & 7)) * 128 + (((n0 + 2 * np + (lane >> 4)) ^ (lane & 7)) << 4);
    // page g of the stage at `at`
    auto page_sums = [&](uint32_t at, uint4 a4) {
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        const uint32_t a[4] = {kt ? a4.z : a4.x, 0u, kt ? a4.w : a4.y, 0u};
#pragma unroll
        for (int pr = 0; pr < (F::kPair ? 2 : 1); ++pr) {
#pragma unroll
          for (int np = 0; np < T / 2; ++np) {
            uint32_t b4[4];
            ldsm_x4_t(p_at[np] + at + pr * Z::kPHalf + kt * 2048, b4);
            mma16<F::kBf16 ? KITTY_BF16 : KITTY_F16>(c[2 * np], a, b4[0], b4[1]);
            mma16<F::kBf16 ? KITTY_BF16 : KITTY_F16>(c[2 * np + 1], a, b4[2], b4[3]);
          }
        }
      }
    };
    for (int i = h; i < n; i += 2) {
      ok = (!F::kPacked || wait(bar.mfull[at4(i)], turn4(i))) && wait(bar.pfull[at4(i)], turn4(i));
      const uint32_t pi = at4(i) * Z::kP;
      if (!ok) break;
      const int there = there_of(i);
      if (i > h && sh.moved[at4(i)] != 0) {
#pragma unroll
        for (int nt = 0; nt < T; ++nt) {
          c[nt][0] *= sh.f[h][8 * ((n0 + nt) % (N / 8)) + 2 * qq];
          c[nt][1] *= sh.f[h][8 * ((n0 + nt) % (N / 8)) + 2 * qq + 1];
        }
      }
      auto middles = [&](int g) {  // and, in row 4, ones
        uint4 a4 = make_uint4(0, 0, 0, 0);
        if (F::kPacked && r < 4) a4 = lds128(mids + at4(i) * 1024 + 256 * g + 64 * r + 16 * qq);
        if (r == 4) a4 = make_uint4(one, one, one, one);
        return a4;
      };
#pragma unroll 1
      for (int g = 0; g < kTilePages; ++g)
        if (mine && ((there >> g) & 1)) page_sums(pi + g * 4096, middles(g));
      __syncwarp();
      if (lane == 0) mbar_arrive_s(a_of(bar.pempty[at4(i)]));
    }
    if (ok) {
#pragma unroll
      for (int nt = 0; nt < T; ++nt) {
        const int y = 8 * (n0 + nt) + 2 * qq;
        if (!mine) break;
        if (r < 4) *reinterpret_cast<float2*>(&sh.mid[h][r][y]) = make_float2(c[nt][0], c[nt][1]);
        if (r == 4) *reinterpret_cast<float2*>(&sh.sum[h][y]) = make_float2(c[nt][0], c[nt][1]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_s(a_of(bar.sums));
    } else if (lane == 0) {
      set_status(p.d_status, KITTY_ST_TIMEOUT);
    }
    __syncwarp();
  }

  __syncthreads();
  // after a wait that ran out: nothing may be in flight when the block's memory is given back
  if (*abort != 0 && elect_one()) {
    if (wid == kMmaWarp) {
      mma_commit(a_of(bar.drain));
      mbar_wait_bounded(&bar.drain, 0, kTreeWaitPolls);
    } else if (F::kPacked && wid == kFetchWarp) {
      if (has_loose) mbar_wait_bounded(&bar.loose[0], 0, kTreeWaitPolls);
      for (int k = max(0, issued - p.raw_stages); k < issued; ++k)
        mbar_wait_bounded(&bar.raw[k % p.raw_stages], (k / p.raw_stages) & 1, kTreeWaitPolls);
    } else if (!F::kPacked && (wid == kFetchWarp || wid == kBiasWarp)) {
      for (int k = max(0, issued - 2); k < issued; ++k)
        mbar_wait_bounded(wid == kFetchWarp ? &bar.kfull[k & 1] : &bar.vfull[k & 1], (k >> 1) & 1, kTreeWaitPolls);
    }
  }
  if (*abort != 0) __syncthreads();
  if (wid == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  end_behind();
}

// ------------------------------------------------------------- merge of the partials
// What each drafted token sees of a prefix that not all sequences see whole, as the prefix kernel
// takes it.  (Rows of no sequence: 0, set before.)
template <bool PACKED>
__global__ void __launch_bounds__(kMaxNodes) tree_prefix_rows_kernel(const TreeParams p, int32_t* rows) {
  const Held hd = held_of<PACKED>(p, blockIdx.x);
  if (hd.ok && (int)threadIdx.x < hd.n) rows[hd.first + threadIdx.x] = hd.prefix;
  if (hd.code != KITTY_ST_OK && threadIdx.x == 0) set_status(p.d_status, hd.code);
}

// A warp a row (query head of a drafted token), four channels a lane; the maxima of 32 partials, a
// lane a partial, and the outputs of eight requested at once.
template <bool PACKED>
__global__ void __launch_bounds__(128) tree_merge_kernel(const TreeParams p) {
  const int b = blockIdx.y, lane = threadIdx.x & 31, i = blockIdx.x * 4 + (threadIdx.x >> 5);
  const Held hd = held_of<PACKED>(p, b);
  if (!hd.ok || i >= hd.n * p.Hq) {
    // the call ends with this grid, so it waits for those before it even if no sequence has a row: the
    // prefix kernel attends rows of padding, too, and writes their partials
    grid_wait();
    return;
  }
  const size_t row = (size_t)hd.first * p.Hq + i;
  const float *pre = p.pre + row * p.slots * kPartialFloats, *own = p.ws + row * p.splits * kPartialFloats;
  const int n = p.slots + p.splits;
  auto part = [&](int x) { return x < p.slots ? pre + (size_t)x * kPartialFloats : own + (size_t)(x - p.slots) * kPartialFloats; };
  grid_wait();
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int x0 = 0; x0 < n; x0 += 32) {
    const float2 ml = x0 + lane < n ? *reinterpret_cast<const float2*>(part(x0 + lane)) : make_float2(-INFINITY, 0.f);
    float top = fmaxf(m, ml.x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    if (top == -INFINITY) continue;
    const float f = m == -INFINITY ? 0.f : ex2a(m - top), e = ml.x == -INFINITY ? 0.f : ex2a(ml.x - top);
    float more = e == 0.f ? 0.f : ml.y * e;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) more += __shfl_xor_sync(0xFFFFFFFFu, more, d);
    l = l * f + more;
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
    m = top;
    for (int s0 = x0; s0 < min(n, x0 + 32); s0 += 8) {
      float4 x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        x[k] = s0 + k < n ? reinterpret_cast<const float4*>(part(s0 + k) + 4)[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float w = __shfl_sync(0xFFFFFFFFu, e, (s0 + k) & 31);
        if (w != 0.f) {  // (0 behind the last)
          o.x = fmaf(x[k].x, w, o.x);
          o.y = fmaf(x[k].y, w, o.y);
          o.z = fmaf(x[k].z, w, o.z);
          o.w = fmaf(x[k].w, w, o.w);
        }
      }
    }
  }
  const bool some = l != 0.f;
  if (!some && lane == 0) set_status(p.d_status, KITTY_ST_EMPTY);
  const float r[4] = {some ? o.x / l : 0.f, some ? o.y / l : 0.f, some ? o.z / l : 0.f, some ? o.w / l : 0.f};
  const size_t at = row * kD + 4 * lane;
  if (p.out_dtype == KITTY_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(r[0], r[1], r[2], r[3]);
  } else {
    uint2 h;
    if (p.out_dtype == KITTY_BF16) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(r[0], r[1]), y = __floats2bfloat162_rn(r[2], r[3]);
      h = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    } else {
      h = make_uint2(h2_bits(__floats2half2_rn(r[0], r[1])), h2_bits(__floats2half2_rn(r[2], r[3])));
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = h;
  }
}

// ------------------------------------------------------------- plan
// Room for staged tiles beside the rest of a block's shared memory.
template <class F>
constexpr int staged_room() { return kSharedMost - (int)((sizeof(Shared<F::N>) + 127) / 128 * 128) - fixed_bytes<F>(); }

static_assert(2 * kTilePages * 7296 <= staged_room<PackedTree<4, 4, 64>>() && 2 * kTilePages * 4224 <= staged_room<PackedTree<2, 2, 64>>(),
              "two staged tiles of the largest pages");

struct TreePlan {
  int rows, units, splits;  // rows of a block, blocks of a (sequence, kv head), splits of its tiles
  double us;                // about how long that takes
  PrefixPlan pre;           // of the prefix kernel, where it attends the prefix (splits: 0: it does not)
};

// Rows of a block: the least of 16, 32, 64 that holds the largest tree's.
// Splits: a block has an SM to itself, so as many as make the last round of blocks end soonest, with
// a block's time its tiles' and a fixed part (us, measured on one block an SM: 2048 and 8192 tokens of
// 4, 8, 16 nodes x 4 heads, packed 34 and 82, 37 and 86, 47 and 111; 16-bit 37 and 98, 40 and 100, 50 and
// 128.  A fixed part of 4 or 10 instead chose the same or, on 16-bit pages, 8% more time).
TreePlan list_plan(const kitty_cfg* cfg, bool packed, int B, int max_nodes, int n_prefix, int max_pages) {
  const int rows = max_nodes * (cfg->num_q_heads / cfg->num_kv_heads);
  TreePlan pl = {16, 1, 1, 0.0, {0, 0, 0}};
  while (pl.rows < rows && pl.rows < 64) pl.rows *= 2;
  pl.units = (rows + pl.rows - 1) / pl.rows;
  const double tile_us = packed ? (pl.rows <= 32 ? 1.0 : 1.3) : (pl.rows <= 32 ? 1.3 : 1.6), fixed_us = 7.0;
  const double own = cfg->decode_total_pages > 0 && B > 0 ? (double)cfg->decode_total_pages / B : max_pages;
  const int tiles = (int)((n_prefix + std::min(own, (double)max_pages) + kTilePages - 1) / kTilePages) + 1;
  const long blocks = (long)pl.units * cfg->num_kv_heads * B;
  const int sms = sm_count();
  double best = 1e30;
  for (int s = 1; s <= std::min(tiles, kMaxSplits); ++s) {
    const double cost = (double)((blocks * s + sms - 1) / sms) * ((tiles + s - 1) / s * tile_us + fixed_us) + (s > 1 ? 2.0 : 0.0);
    if (cost < best - 1e-9) {
      best = cost;
      pl.splits = s;
      pl.us = cost;
    }
  }
  return pl;
}

// A shared prefix is either part of every sequence's tiles, or attended by the prefix kernel for all
// drafted tokens at once, 256 rows a block, and merged.  The second prepares a page's operands for
// four times the rows, and costs the prefix kernel's start and end and a launch or two more: its
// blocks' time (as its own plan has it) is weighed here; what the two grids overlap pays for the rest.
// Sequences of 12 nodes x 4 heads behind 4096 tokens, tiles against prefix kernel, us: 1 sequence 29
// against 37, 4 39 against 41, 8 51 against 47 (where the rule still takes the tiles), 16 74 against 60,
// 32 132 against 85, 64 259 against 136.
TreePlan tree_plan_of(const kitty_cfg* cfg, bool packed, int B, int n_tokens, int max_nodes, int n_prefix, int max_pages) {
  TreePlan all = list_plan(cfg, packed, B, max_nodes, n_prefix, max_pages);
  if (n_prefix == 0) return all;
  TreePlan own = list_plan(cfg, packed, B, max_nodes, 0, max_pages);
  own.pre = prefix_plan(cfg, packed, n_tokens, n_prefix, 0);
  const long blocks = (long)own.pre.units * own.pre.splits, sms = sm_count();
  const int pages = packed ? 3 : 4, tiles = (n_prefix + pages - 1) / pages;
  const double tile_us = n_tokens * (cfg->num_q_heads / cfg->num_kv_heads) > 128 ? 1.8 : 0.9;
  own.us += (double)((blocks + sms - 1) / sms) * ((tiles + own.pre.splits - 1) / own.pre.splits + 7) * tile_us;
  return own.us < all.us ? own : all;
}

size_t own_bytes(const kitty_cfg* cfg, const TreePlan& pl, int n_tokens) {
  return pl.splits > 1 || pl.pre.splits > 0 ? (size_t)n_tokens * cfg->num_q_heads * pl.splits * kPartialFloats * sizeof(float) : 0;
}
// The prefix's partials, then the own ones, then what each token sees of the prefix.
size_t prefix_bytes(const kitty_cfg* cfg, const TreePlan& pl, int n_tokens) {
  return (size_t)n_tokens * cfg->num_q_heads * pl.pre.slots * kPartialFloats * sizeof(float);
}
size_t partial_bytes(const kitty_cfg* cfg, const TreePlan& pl, int n_tokens) {
  return prefix_bytes(cfg, pl, n_tokens) + own_bytes(cfg, pl, n_tokens) + (pl.pre.splits > 0 ? (size_t)n_tokens * sizeof(int32_t) : 0);
}

bool rows_ok(const void* p, int64_t stride, int heads) {
  return p != nullptr && aligned16(p) && stride >= (int64_t)heads * kD && stride % 8 == 0;
}

int check_tree(const kitty_cfg* cfg, int B, int n_tokens, int max_nodes, int n_prefix, int max_pages) {
  const int rc = check_cfg(cfg, 32);
  if (rc != KITTY_OK) return rc;
  if (B < 0 || n_tokens < 0 || n_prefix < 0 || max_pages < 0 || max_nodes < 1) return KITTY_ERR_INVALID_ARG;
  // (rows are counted in 32 bits)
  return max_nodes > kMaxNodes || (uint64_t)n_tokens * cfg->num_q_heads > 0x7FFFFFFFull ? KITTY_ERR_UNSUPPORTED : KITTY_OK;
}

int workspace(const kitty_cfg* cfg, bool packed, int B, int n_tokens, int max_nodes, int n_prefix, int max_pages,
              size_t* bytes) {
  const int rc = check_tree(cfg, B, n_tokens, max_nodes, n_prefix, max_pages);
  if (rc != KITTY_OK) return rc;
  if (!bytes) return KITTY_ERR_INVALID_ARG;
  *bytes = B == 0 || n_tokens == 0 ? 0 : partial_bytes(cfg, tree_plan_of(cfg, packed, B, n_tokens, max_nodes, n_prefix, max_pages), n_tokens);
  return KITTY_OK;
}

template <class F>
int launch_tree(TreeParams& p, const CUtensorMap& map, cudaStream_t s) {
  using Z = Sizes<F>;
  static_assert(Z::kCols <= 512, "fits tensor memory");
  constexpr int kMost = staged_room<F>() + fixed_bytes<F>();
  // one block an SM: two would wait for each other's tensor memory
  static_assert(F::kPacked || fixed_bytes<F>() > 116 * 1024, "one block an SM");
  int smem = fixed_bytes<F>();
  if (F::kPacked) {
    p.raw_stages = kMaxRaw * kTilePages * p.blob <= staged_room<F>() ? kMaxRaw : 2;
    smem = std::max(smem + p.raw_stages * kTilePages * p.blob, 116 * 1024);
  }
  static std::atomic<uint64_t> opted_in{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KITTY_ERR_CUDA;
  const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t(1) << dev) : 0;
  if (bit == 0 || (opted_in.load() & bit) == 0) {
    if (cudaFuncSetAttribute(tree_kernel<F>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost) != cudaSuccess) {
      (void)cudaGetLastError();
      return KITTY_ERR_CUDA;
    }
    opted_in.fetch_or(bit);
  }
  cudaError_t e = launch_behind(tree_kernel<F>, dim3((unsigned)(p.units * p.Hkv) * (unsigned)p.B, (unsigned)p.splits), kTreeThreads,
                                (size_t)smem, s, p.slots > 0, p, map);
  if (e == cudaSuccess && !p.direct)
    e = launch_dependent(tree_merge_kernel<F::kPacked>, dim3((unsigned)((p.max_nodes * p.Hq + 3) / 4), (unsigned)p.B), 128, 0, s, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? KITTY_OK : KITTY_ERR_CUDA;
}

template <int W, int V>
int launch_packed(TreeParams& p, int rows, cudaStream_t s) {
  const CUtensorMap map = {};
  switch (rows) {
    case 16: return launch_tree<PackedTree<W, V, 16>>(p, map, s);
    case 32: return launch_tree<PackedTree<W, V, 32>>(p, map, s);
    default: return launch_tree<PackedTree<W, V, 64>>(p, map, s);
  }
}
template <bool BF>
int launch_plain(TreeParams& p, int rows, cudaStream_t s) {
  CUtensorMap map = {};
  const uint64_t lines = (uint64_t)p.pool_pages * p.Hkv * 2 * kPage;
  if (lines > 0x7FFFFFFFull) return KITTY_ERR_UNSUPPORTED;  // a row's coordinate is an int32
  if (lines > 0 && p.pool != nullptr && !pool_map(&map, p.pool, lines)) return KITTY_ERR_CUDA;
  switch (rows) {
    case 16: return launch_tree<PlainTree<BF, 16>>(p, map, s);
    case 32: return launch_tree<PlainTree<BF, 32>>(p, map, s);
    default: return launch_tree<PlainTree<BF, 64>>(p, map, s);
  }
}

// Checks of what both caches' calls share, and their part of p; 1: nothing to do.
int tree_params(const kitty_cfg* cfg, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                const void* v, int64_t v_stride, int32_t n_tokens, const int32_t* seq_start,
                const uint64_t* visible, int32_t max_nodes, const void* pool, int32_t pool_pages,
                const int32_t* prefix_table, int32_t n_prefix, const int32_t* prefix_pages,
                const int32_t* block_table, int32_t max_pages, float sm_scale, void* out, int32_t out_dtype,
                void* ws, size_t ws_bytes, int32_t B, int32_t* d_status, bool packed, TreePlan* plan, TreeParams* p) {
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
  const TreePlan pl = tree_plan_of(cfg, packed, B, n_tokens, max_nodes, n_prefix, max_pages);
  if (pl.pre.splits > 0 && (size_t)q_stride > kPrefixMaxStride) return KITTY_ERR_UNSUPPORTED;
  const size_t need = partial_bytes(cfg, pl, n_tokens);
  if (ws_bytes < need || (need > 0 && (!ws || !aligned16(ws)))) return KITTY_ERR_WORKSPACE;
  if ((uint64_t)pl.units * Hkv * B > 0x7FFFFFFFull || B > 65535) return KITTY_ERR_UNSUPPORTED;
  *plan = pl;
  p->units = pl.units;
  p->splits = pl.splits;
  p->slots = pl.pre.slots;
  p->direct = pl.splits == 1 && pl.pre.slots == 0;
  p->pre = static_cast<float*>(ws);
  p->ws = static_cast<float*>(ws) + prefix_bytes(cfg, pl, n_tokens) / sizeof(float);
  p->wait_polls = cfg->decode_wait_polls > 0 ? (uint32_t)cfg->decode_wait_polls : kTreeWaitPolls;
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

// The prefix's partials by the prefix kernel, if the plan has it so: p goes on without a prefix.
template <bool PACKED>
int attend_prefix(const kitty_cfg* cfg, const TreePlan& pl, TreeParams& p, cudaStream_t s) {
  if (pl.pre.splits == 0) return KITTY_OK;
  int32_t* rows = nullptr;
  if (p.prefix_pages != nullptr) {
    rows = reinterpret_cast<int32_t*>(p.ws + own_bytes(cfg, pl, p.n_tokens) / sizeof(float));
    if (cudaMemsetAsync(rows, 0, (size_t)p.n_tokens * sizeof(int32_t), s) != cudaSuccess) {
      (void)cudaGetLastError();
      return KITTY_ERR_CUDA;
    }
    const cudaError_t e = launch_behind(tree_prefix_rows_kernel<PACKED>, dim3((unsigned)p.B), kMaxNodes, 0, s, false, p, rows);
    if (e != cudaSuccess) return KITTY_ERR_CUDA;
  }
  PrefixArgs a = {};
  a.q = p.q;
  a.q_stride = p.q_stride;
  a.pool = p.pool;
  a.table = p.prefix_table;
  a.prefix_pages = rows;
  a.ws = const_cast<float*>(p.pre);
  a.d_status = p.d_status;
  a.sm_log2 = p.sm_log2;
  a.wait_polls = cfg->decode_wait_polls > 0 ? (uint32_t)cfg->decode_wait_polls : 1u << 22;
  a.pool_pages = p.pool_pages;
  a.n_prefix = p.n_prefix;
  a.B = p.n_tokens;
  a.Hq = p.Hq;
  a.Hkv = p.Hkv;
  a.g = p.g;
  a.n_hi = p.n_hi;
  a.blob = p.blob;
  a.in_dtype = p.in_dtype;
  a.splits = pl.pre.splits;
  a.slots = pl.pre.slots;
  p.n_prefix = 0;
  p.prefix_pages = nullptr;
  return prefix_launch(cfg, PACKED, a, pl.pre, s);
}

}  // namespace
}  // namespace kitty

using namespace kitty;

extern "C" int kitty_tree_workspace_bytes(const kitty_cfg* cfg, int32_t B, int32_t n_tokens, int32_t max_nodes,
                                          int32_t n_prefix, int32_t max_pages, size_t* bytes) {
  return workspace(cfg, true, B, n_tokens, max_nodes, n_prefix, max_pages, bytes);
}

extern "C" int kitty_f16kv_tree_workspace_bytes(const kitty_cfg* cfg, int32_t B, int32_t n_tokens,
                                                int32_t max_nodes, int32_t n_prefix, int32_t max_pages,
                                                size_t* bytes) {
  return workspace(cfg, false, B, n_tokens, max_nodes, n_prefix, max_pages, bytes);
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
  TreePlan pl = {};
  int rc = tree_params(cfg, q, q_stride, k, k_stride, v, v_stride, n_tokens, seq_start, visible, max_nodes,
                             pool, pool_pages, prefix_table, n_prefix, prefix_pages, block_table, max_pages,
                             sm_scale, out, out_dtype, workspace, workspace_bytes, B, d_status, true, &pl, &p);
  if (rc != KITTY_OK) return rc == 1 ? KITTY_OK : rc;
  if (!num_pages || !tail_len || !tail_k || !tail_v || !aligned16(tail_k) || !aligned16(tail_v))
    return KITTY_ERR_INVALID_ARG;
  p.num_pages = num_pages;
  p.tail_len = tail_len;
  p.tail_k = static_cast<const uint16_t*>(tail_k);
  p.tail_v = static_cast<const uint16_t*>(tail_v);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  rc = attend_prefix<true>(cfg, pl, p, s);
  if (rc != KITTY_OK) return rc;
  if (cfg->lo_bit == 2) return launch_packed<2, 2>(p, pl.rows, s);
  return v_bits(cfg) == 2 ? launch_packed<4, 2>(p, pl.rows, s) : launch_packed<4, 4>(p, pl.rows, s);
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
  TreePlan pl = {};
  int rc = tree_params(cfg, q, q_stride, k, k_stride, v, v_stride, n_tokens, seq_start, visible, max_nodes,
                             pool, pool_pages, prefix_table, n_prefix, prefix_pages, block_table, max_pages,
                             sm_scale, out, out_dtype, workspace, workspace_bytes, B, d_status, false, &pl, &p);
  if (rc != KITTY_OK) return rc == 1 ? KITTY_OK : rc;
  if (!ctx_len) return KITTY_ERR_INVALID_ARG;
  p.ctx_len = ctx_len;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  rc = attend_prefix<false>(cfg, pl, p, s);
  if (rc != KITTY_OK) return rc;
  return cfg->in_dtype == KITTY_BF16 ? launch_plain<true>(p, pl.rows, s) : launch_plain<false>(p, pl.rows, s);
}
