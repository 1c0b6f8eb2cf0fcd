// Attention of drafted tokens over a sequence's cache and over each other, on the fifth-generation
// tensor cores (sm_103a).
//
//   out[t][hq] = softmax(sm_scale * q . [K_prefix; K_b; K_tree]) . [V_prefix; V_b; V_tree]
//
// Rows.  The query heads of a kv head over the nodes of a sequence's tree, node by node: n * g
// rows that see the same cached tokens.  One block takes up to N of them (N = 16, 32, 64, 128 by
// the largest tree) and a share of the sequence's tiles of 128 tokens.  Tokens are the
// products' 128 rows and query rows their N columns, so that a product costs what the rows
// need: 16 rows an eighth of 128.  Per tile
//   S^T = K Q^T         128 x N x 128, fp32 in tensor memory
//   p = 2^(s - m)       a thread a token: its scores from tensor memory, p to shared memory
//   O^T += V^T P^T      128 channels x N x 128 tokens, fp32 in tensor memory
// The reference m of a row is set 2^4 below its maximum over the first tile and moves only when a
// score passes it by more than 2^15: what p loses below 2^-25 is 2^-29 of the largest then.
// A row decides by its own scores, so its bytes do not depend on the others.
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
// fp16; 16-bit pages: p to two halves.
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
constexpr int kSoftmaxWarps = 8;  // two groups of four, each with half of the rows
constexpr int kKeyWarp = 8, kValueWarp = 12, kMmaWarp = 16, kFetchWarp = 17, kBiasWarp = 18, kSumWarp = 19;
constexpr int kTreeThreads = 640;
constexpr int kMaxRaw = 4;        // staged tiles of packed pages
constexpr int kFlags = 16;        // tiles whose page flags are kept
constexpr int kLoose = 96;        // loose tokens: 32 of the tail, 64 nodes
constexpr int kLoosePitch = 272;
constexpr uint32_t kTreeWaitPolls = 1u << 22;
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
  int units, splits, raw_stages;
};

// Packed pages: Key planes of W bits, Values of V bits; N rows.
template <int W_, int V_, int N_>
struct PackedTree {
  static constexpr bool kPacked = true, kBf16 = false, kPair = false;
  static constexpr int W = W_, V = V_, N = N_;
  static constexpr int kOps = N == 128 ? 1 : 2;  // stages of the Key and Value operands
  static constexpr int kVCol = 64 * kOps, kSCol = 128 * kOps;
};
// 16-bit pages.
template <bool BF, int N_>
struct PlainTree {
  static constexpr bool kPacked = false, kBf16 = BF, kPair = true;
  static constexpr int W = 0, V = 0, N = N_;
  static constexpr int kOps = 2;
  static constexpr int kVCol = 0, kSCol = 0;
};
template <class F>
struct Sizes {
  static constexpr int N = F::N, C = N / 2;           // rows; columns of a softmax group
  static constexpr int kQHalf = N * 128, kQ = 2 * kQHalf;
  static constexpr int kPBlock = kTile * 128;          // 64 rows of 128 tokens
  static constexpr int kPHalf = kPBlock * (N > 64 ? 2 : 1), kP = kPHalf * (F::kPair ? 2 : 1);
  static constexpr int kOCol = F::kSCol + 2 * N, kCols = kOCol + N;
  static constexpr int kHalf16 = kTile * 128, kTile16 = 2 * kHalf16;  // a 16-bit tile of Keys or Values
  static constexpr int kSpread = F::kPacked ? 512 * F::W : 0;         // a page's low codes in base-plane order
  static constexpr int kFixed = kQ + 2 * kP + (F::kPacked ? 2 * kLoose * kLoosePitch + 4 * kSpread + F::kOps * 1024
                                                         : 2 * F::kOps * kTile16);
};

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
__device__ __forceinline__ bool wait_lanes(bool need, uint32_t a, uint32_t parity, uint32_t polls, volatile int* abort) {
  bool done = !need;
  for (uint32_t i = 0;; ++i) {
    done = done || mbar_try(a, parity);
    if (__all_sync(0xFFFFFFFFu, done)) return true;
    const bool stop = i >= polls || *abort != 0;
    if (__any_sync(0xFFFFFFFFu, stop)) break;
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
__device__ __forceinline__ void tmem_st_frag(uint32_t a, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
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
#pragma unroll 2
  for (int js = 0; js < nx; ++js) {
    const uint32_t ids = lds32(kch + 16 * js + 4 * qq);
#pragma unroll
    for (int mt = 0; mt < W / 2; ++mt) {
      // rotated back by two bits, byte 2e + h holds the column parity e, half h; ids: 2h + e
      uint32_t x = lds32(plane + 2 * W * js + 4 * mt);
      x = __funnelshift_r(x, x, 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t c = (ids >> (8 * i)) & 127u, byte = (x >> (8 * (2 * (i & 1) + (i >> 1)))) & 255u;
        // word of channel c: lane (r, (c & 7) / 2), k-step c / 16 (W = 4: and mt); its byte there
        sts8(mine + 16 * W * ((c & 7) >> 1) + 2 * W * (c >> 4) + 4 * mt + 2 * (c & 1) + ((c >> 3) & 1), byte);
      }
    }
  }
  __syncwarp();
}

// A page's Keys, staged at raw, to the 32 lanes of tensor memory at `to`: 64 columns of channel pairs.
// (For spread words bytes are not rotated: they are rotated as they are taken.)
template <int W>
__device__ __forceinline__ void put_keys(uint32_t raw, uint32_t to, uint32_t spread, int n_hi, int32_t* d_status) {
  const int lane = threadIdx.x & 31, qq = lane & 3;
  const uint32_t ks = raw + 512 * W + 4 * W * n_hi, sq = ks + 4 * qq;
  const bool boosted = n_hi > 0;
  if (boosted) spread_low<W>(raw, spread, n_hi);
#pragma unroll
  for (int jc = 0; jc < 8; jc += 4) {  // four k-steps: 32 columns
    uint32_t w[2 * W], lo[2 * W];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
      const uint4 a = lds128(raw + 16 * W * lane + 2 * W * jc + 16 * i);
      w[4 * i] = a.x;
      w[4 * i + 1] = a.y;
      w[4 * i + 2] = a.z;
      w[4 * i + 3] = a.w;
      if (boosted) {
        const uint4 c = lds128(spread + 16 * W * lane + 2 * W * jc + 16 * i);
        lo[4 * i] = c.x;
        lo[4 * i + 1] = c.y;
        lo[4 * i + 2] = c.z;
        lo[4 * i + 3] = c.w;
      }
    }
    uint32_t a[2][16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t S[2] = {lds32(sq + 32 * (jc + j)), lds32(sq + 32 * (jc + j) + 16)};
      const uint32_t T[2] = {h2mul(S[0], two(0xCC00)), h2mul(S[1], two(0xCC00))};  // -16 S
      if (W == 2) {
        if (!boosted) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x = h ? __funnelshift_r(w[j], w[j], 8) : w[j];
            uint32_t* o0 = &a[0][2 * (2 * j + h)];
            uint32_t* o1 = &a[1][2 * (2 * j + h)];
            o0[0] = h2fma((x & two(0x000C)) | k16, S[h], T[h]);
            o0[1] = h2fma((x & two(0x0030)) | k16, S[h], T[h]);
            o1[0] = h2fma((x & two(0x00C0)) | k16, S[h], T[h]);
            o1[1] = h2fma((x & two(0x0300)) | k16, S[h], T[h]);
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
            o0[0] = h2fma((xa & two(0x003C)) | k16, S[h], T[h]);
            o0[1] = h2fma((xb & two(0x003C)) | k16, S[h], T[h]);
            o1[0] = h2fma((xa & two(0x03C0)) | k16, S[h], T[h]);
            o1[1] = h2fma((xb & two(0x03C0)) | k16, S[h], T[h]);
          }
        }
      } else {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const uint32_t x0 = w[(2 * j + mt) % (2 * W)];
          const uint32_t l0 = boosted ? __funnelshift_l(lo[(2 * j + mt) % (2 * W)], lo[(2 * j + mt) % (2 * W)], 2) : 0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x = h ? __funnelshift_r(x0, x0, 8) : x0;
            uint32_t* o = &a[mt][2 * (2 * j + h)];
            o[0] = h2fma((x & two(0x003C)) | k16, S[h], T[h]);
            o[1] = h2fma((x & two(0x03C0)) | k16, S[h], T[h]);
            if (boosted) {  // + S / 16 * low code, rounded once
              const uint32_t l = h ? __funnelshift_r(l0, l0, 8) : l0, s = h2mul(S[h], two(0x2C00));
              o[0] = h2fma(h2add((l & two(0x003C)) | k16, two(0xCC00)), s, o[0]);
              o[1] = h2fma(h2add((l & two(0x03C0)) | k16, two(0xCC00)), s, o[1]);
            }
          }
        }
      }
    }
    tmem_st_frag(to + 8 * jc, a[0]);
    tmem_st_frag(to + 8 * jc + (16u << 16), a[1]);
  }
  const uint2 s4 = lds64(ks + 8 * lane);  // steps that times 16 leave fp16
  const float2 s0 = __half22float2(bits_h2(s4.x)), s1 = __half22float2(bits_h2(s4.y));
  if (!(fmaxf(fmaxf(s0.x, s0.y), fmaxf(s1.x, s1.y)) <= 4094.f)) set_status(d_status, KITTY_ST_RANGE);
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

// Two pages' Values of channel group G (staged at raw, one `stride` behind the other): their
// centered codes times steps to 16 + 16 lanes of tensor memory at `to` (16 columns a page), the
// groups' middles to `mids` (a page's [group][64 bytes], 256 bytes a page).
template <int V>
__device__ __forceinline__ void put_values(uint32_t raw, int stride, uint32_t to, uint32_t mids, int G, int n_hi, int W,
                                           int there, int32_t* d_status) {
  const int lane = threadIdx.x & 31, r = lane >> 2, qq = lane & 3;
  uint32_t a[2][16];
  uint32_t top = 0;
#pragma unroll
  for (int page = 0; page < 2; ++page) {
    const uint32_t vb = raw + page * stride + 512 * W + 4 * W * n_hi + 512 + n_hi, vs = vb + 512 * V, vm = vs + 256;
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
      if ((there >> page) & 1) top = __vmaxu2(top, S[i]);
      uint32_t* o0 = &a[0][2 * (4 * page + i)];
      uint32_t* o1 = &a[1][2 * (4 * page + i)];
      if (V == 2) {
        const uint32_t x = h ? __funnelshift_r(w[kt], w[kt], 8) : w[kt];
        // 16 + 1.5 * 2^e, e = -4, -2, 0, 2
        o0[0] = h2mul(h2add((x & two(0x000C)) | k16, two(0xCC06)), S[i]);
        o0[1] = h2mul(h2add((x & two(0x0030)) | k16, two(0xCC18)), S[i]);
        o1[0] = h2mul(h2add((x & two(0x00C0)) | k16, two(0xCC60)), S[i]);
        o1[1] = h2mul(h2add((x & two(0x0300)) | k16, two(0xCD80)), S[i]);
      } else {
#pragma unroll
        for (int mc = 0; mc < 2; ++mc) {
          const uint32_t y = w[(2 * kt + mc) % V], x = h ? __funnelshift_r(y, y, 8) : y;
          uint32_t* o = mc ? o1 : o0;
          // 16 + 7.5 * 2^e, e = -4, 0
          o[0] = h2mul(h2add((x & two(0x003C)) | k16, two(0xCC1E)), S[i]);
          o[1] = h2mul(h2add((x & two(0x03C0)) | k16, two(0xCDE0)), S[i]);
        }
      }
    }
    if (r == 0)
      sts128(mids + 256 * page + 64 * G + 16 * qq,
             make_uint4(h2fma(S[0], mid, M[0]), h2fma(S[1], mid, M[1]), h2fma(S[2], mid, M[2]), h2fma(S[3], mid, M[3])));
  }
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

struct Bars {
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2];  // operands
  uint64_t sfull[2], sempty[2], bias[2], pfull[2], pempty[2], sums, drain;
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
  float m[N], f[2][N];         // reference of each row; factor of its move, by tile parity
  int moved[2][2];             // by tile parity and softmax group
  alignas(16) float bias[2][4][N];   // q.M of each page, by tile parity
  alignas(16) float shift[kSoftmaxWarps][N / 2];
  float top[kSoftmaxWarps][N / 2];   // maxima of a warp's tokens
  float sum[N], mid[4][N];
  int row[N];                  // output row (token, query head); -1: none
  unsigned long long sees[N];
};


template <class F>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_kernel(const TreeParams p, const __grid_constant__ CUtensorMap map) {
  using Z = Sizes<F>;
  constexpr int N = F::N, C = Z::C;
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
  if (!hd.ok || R <= 0) return;
  const int pages = hd.prefix + hd.pages, tiles = (pages + kTilePages - 1) / kTilePages + 1;
  const int t0 = (int)((long)tiles * split / p.splits), n = (int)((long)tiles * (split + 1) / p.splits) - t0;
  // row x of the block: output row; node
  auto out_row = [&](int x) {
    const int i = unit * N + x, node = i / p.g;
    return (hd.first + node) * p.Hq + kvh * p.g + (i - node * p.g);
  };
  if (n == 0) {
    if (tid < R) p.ws[((size_t)out_row(tid) * p.splits + split) * kPartialFloats] = -INFINITY;
    return;
  }
  const bool has_loose = t0 + n == tiles;
  volatile int* abort = &sh.abort;
  const uint32_t base = (smem_u32(dyn) + 1023u) & ~1023u;
  const uint32_t qs = base, ps = qs + Z::kQ, ops = ps + 2 * Z::kP;  // ops: 16-bit tiles (Keys, then Values)
  const uint32_t loose = ops, spread = loose + 2 * kLoose * kLoosePitch, mids = spread + 4 * Z::kSpread;
  const uint32_t raws = mids + F::kOps * 1024;
  Bars& bar = sh.bars;
  auto a_of = [&](uint64_t& x) { return smem_u32(&x); };
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.kfull[i], F::kPacked ? 4 : 1);
      mbar_init(&bar.vfull[i], F::kPacked ? 4 : 1);
      mbar_init(&bar.kempty[i], 1);
      mbar_init(&bar.vempty[i], F::kPacked ? 2 : 1);
      mbar_init(&bar.sfull[i], 1);
      mbar_init(&bar.sempty[i], kSoftmaxWarps);
      mbar_init(&bar.bias[i], 1);
      mbar_init(&bar.pfull[i], kSoftmaxWarps);
      mbar_init(&bar.pempty[i], 2);
    }
    mbar_init(&bar.sums, 1);
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
    if (split == 0 && code != KITTY_ST_OK) set_status(p.d_status, code);
  }
  if (tid < N) {
    sh.row[tid] = tid < R ? out_row(tid) : -1;
    sh.m[tid] = kFloor;
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
    const int h = wid >> 2, g = wid & 3, id = 1 + h, col = h * C;
    const float sc = p.sm_log2;
    const float sc_page = F::kPacked ? sc * pow2(-key_exp<F>(lane, p.n_hi > 0)) : sc;
    const uint32_t shift_at = smem_u32(sh.shift[wid]);
    const int token = 32 * g + lane;
    const uint32_t prow = ps + (N > 64 ? h * Z::kPBlock : 0) + token * 128;
    bool ok = true;
    int i = 0;
    for (; i < n; ++i) {
      const int st = i & 1;
      ok = wait_lanes(lane < (F::kPacked ? 3 : 2), lane == 0 ? a_of(bar.sfull[st]) : lane == 1 ? a_of(bar.pempty[st]) : a_of(bar.bias[st]),
                      lane == 1 ? ((i >> 1) & 1) ^ 1 : (i >> 1) & 1, p.wait_polls, abort);
      tc_fence_after();
      const bool special = has_loose && i == n - 1;
      const bool there = (there_of(i) >> g) & 1;
      const float scl = special ? sc : sc_page;
      const uint32_t S = tmem + F::kSCol + st * N + col + quad;
      uint32_t x[C];
      tmem_load<C>(S, x);
      // y = x * scl + shift of the row, masked
      const bool in = lane < loose_count(g);
      const int node = (token - 32) & 63;  // of a loose token that is one (masked: in range for the others, too)
      auto scores = [&](bool with_m) {
        for (int c = lane; c < C; c += 32) {
          const float bias = F::kPacked ? sh.bias[st][g][col + c] * sc : 0.f;
          sts32(shift_at + 4 * c, with_m ? bias - sh.m[col + c] : bias);  // read by lds128 alone
        }
        __syncwarp();
        const uint64_t scl2 = f2pack(scl, scl);
#pragma unroll
        for (int c = 0; c < C; c += 4) {
          const uint4 s4 = lds128(shift_at + 4 * c);
          uint64_t e;
          asm("mov.b64 %0, {%1, %2};" : "=l"(e) : "r"(x[c]), "r"(x[c + 1]));
          uint64_t s2;
          asm("mov.b64 %0, {%1, %2};" : "=l"(s2) : "r"(s4.x), "r"(s4.y));
          asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(e) : "l"(e), "l"(scl2), "l"(s2));
          asm("mov.b64 {%0, %1}, %2;" : "=r"(x[c]), "=r"(x[c + 1]) : "l"(e));
          asm("mov.b64 %0, {%1, %2};" : "=l"(e) : "r"(x[c + 2]), "r"(x[c + 3]));
          asm("mov.b64 %0, {%1, %2};" : "=l"(s2) : "r"(s4.z), "r"(s4.w));
          asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(e) : "l"(e), "l"(scl2), "l"(s2));
          asm("mov.b64 {%0, %1}, %2;" : "=r"(x[c + 2]), "=r"(x[c + 3]) : "l"(e));
        }
        if (!there) {
#pragma unroll
          for (int c = 0; c < C; ++c) x[c] = __float_as_uint(-INFINITY);
        } else if (special) {
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const bool on = g == 0 || ((sh.sees[col + c] >> node) & 1ull) != 0;
            if (!in || !on) x[c] = __float_as_uint(-INFINITY);
          }
        }
        __syncwarp();
      };
      scores(true);
      float top = -INFINITY;
#pragma unroll
      for (int c = 0; c < C; c += 2) top = fmaxf(fmaxf(top, __uint_as_float(x[c])), __uint_as_float(x[c + 1]));
      bool slow = group_any(id, i == 0 || top > kSlack || !ok);
      if (slow) {
        if (group_any(id, !ok)) {
          ok = false;
          break;
        }
        tmem_load<C>(S, x);
        scores(false);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const float mx = warp_max(__uint_as_float(x[c]));
          if (lane == 0) sh.top[wid][c] = mx;
        }
        group_sync(id);
        bool moves = false;
        const int c = tid & 127;  // a thread a row
        if (c < C) {
          const float mx = fmaxf(fmaxf(sh.top[4 * h][c], sh.top[4 * h + 1][c]), fmaxf(sh.top[4 * h + 2][c], sh.top[4 * h + 3][c]));
          const float m = sh.m[col + c];
          const bool set = (i == 0 && mx > kFloor) || mx > m + kSlack;
          const float nm = set ? mx + kMargin : m;
          sh.m[col + c] = nm;
          sh.f[st][col + c] = i > 0 && set ? ex2a(m - nm) : 1.f;
          moves = i > 0 && set;
        }
        moves = group_any(id, moves);
        if (moves) {  // the outputs so far, once the products so far are done
          ok = wait_lanes(lane == 0, a_of(bar.pempty[1 - st]), ((i - 1) >> 1) & 1, p.wait_polls, abort);
          tc_fence_after();
          const uint32_t O = tmem + Z::kOCol + col + quad;
#pragma unroll 1
          for (int c = 0; c < C; c += 8) {
            uint32_t y[8];
            tmem_load<8>(O + c, y);
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * sh.f[st][col + c + k]);
            tmem_st8(O + c, y);
          }
          tmem_wait_st();
          if (group_any(id, !ok)) {
            ok = false;
            break;
          }
        }
        if (lane == 0 && g == 0) sh.moved[st][h] = moves;
        tmem_load<C>(S, x);
        scores(true);
      } else if (lane == 0 && g == 0) {
        sh.moved[st][h] = 0;
      }
      // the scores and their bias have been read
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_s(a_of(bar.sempty[st]));
#pragma unroll
      for (int c = 0; c < C; c += 8) {
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
        const int chunk = ((N > 64 ? 0 : col) + c) / 8;
        const uint32_t at = prow + st * Z::kP + ((chunk ^ (token & 7)) << 4);
        sts128(at, make_uint4(w[0], w[1], w[2], w[3]));
        if (F::kPair) sts128(at + Z::kPHalf, make_uint4(rest[0], rest[1], rest[2], rest[3]));
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive_s(a_of(bar.pfull[st]));
    }
    // ---- outputs or partials: a thread a channel, a warp 32 channels of each row of its group
    if (ok)
      ok = wait_lanes(lane < 2, lane == 0 ? a_of(bar.pempty[(n - 1) & 1]) : a_of(bar.sums), lane == 0 ? ((n - 1) >> 1) & 1 : 0, p.wait_polls, abort);
    if (ok) {
      tc_fence_after();
      const float scale = F::kPacked ? pow2(-value_exp<F>(lane)) : 1.f;
      const int ch = 32 * g + lane;
      bool empty = false;
#pragma unroll
      for (int c = 0; c < C; c += 8) {
        if (col + c >= R) break;
        uint32_t x[8];
        tmem_load<8>(tmem + Z::kOCol + col + c + quad, x);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int y = col + c + k, row = sh.row[y];
          if (row < 0) continue;
          const float l = sh.sum[y];
          const float o = l != 0.f ? __uint_as_float(x[k]) * scale + (F::kPacked ? sh.mid[g][y] : 0.f) : 0.f;
          if (p.splits == 1) {
            const float v = l != 0.f ? o / l : 0.f;
            const size_t at = (size_t)row * kD + ch;
            if (p.out_dtype == KITTY_F32) static_cast<float*>(p.out)[at] = v;
            else if (p.out_dtype == KITTY_BF16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
            else static_cast<__half*>(p.out)[at] = __float2half_rn(v);
            empty = empty || l == 0.f;
          } else {
            float* part = p.ws + ((size_t)row * p.splits + split) * kPartialFloats;
            part[4 + ch] = o;
            if (ch == 0) *reinterpret_cast<float2*>(part) = make_float2(l != 0.f ? sh.m[y] : -INFINITY, l);
          }
        }
      }
      if (empty && ch == 0) set_status(p.d_status, KITTY_ST_EMPTY);
      tc_fence_before();
    } else if (lane == 0) {
      set_status(p.d_status, KITTY_ST_TIMEOUT);
    }
  } else if (wid < kMmaWarp) {
    // =========================================================== operands
    const bool keys = wid < kValueWarp;
    const int g = wid & 3;
    bool ok = true;
    if constexpr (F::kPacked) {
      int slot = 0, turn = 0;
      for (int i = 0; i < n; ++i) {
        const int st = i % F::kOps, use = i / F::kOps;
        const bool special = has_loose && i == n - 1;
        const uint32_t empty = keys ? a_of(bar.kempty[st]) : a_of(bar.vempty[st]);
        ok = wait_lanes(lane < 2, lane == 0 ? empty : special ? a_of(bar.loose[0]) : a_of(bar.raw[slot]),
                        lane == 0 ? (use & 1) ^ 1 : special ? 0 : turn & 1, p.wait_polls, abort);
        if (!ok) break;
        tc_fence_after();
        const uint32_t to = tmem + (keys ? 0 : F::kVCol) + 64 * st + quad;
        if (!special) {
          const uint32_t raw = raws + slot * (kTilePages * p.blob);
          const int there = sh.flags[i % kFlags];
          if (keys) {
            if ((there >> g) & 1) put_keys<F::W>(raw + g * p.blob, to, spread + g * Z::kSpread, p.n_hi, p.d_status);
          } else {
#pragma unroll 1
            for (int x = 0; x < 2; ++x)
              if ((there >> (2 * x)) & 3)
                put_values<F::V>(raw + 2 * x * p.blob, p.blob, to + 32 * x, mids + st * 1024 + 512 * x, g, p.n_hi, F::W, there >> (2 * x), p.d_status);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_s(a_of(bar.freed[slot]));
          if (++slot == p.raw_stages) {
            slot = 0;
            ++turn;
          }
        } else if (keys) {
          // a thread a token
          uint32_t mag = 0;
          const uint32_t src = loose + (32 * g + lane) * kLoosePitch;
          if (loose_count(g) > 0) {
#pragma unroll
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
          // a thread a channel; what no one sees, or fp16 cannot hold, is 0
          const float up = pow2(value_exp<F>(lane));
          int code = KITTY_ST_OK;
#pragma unroll 1
          for (int x = 0; x < 3; ++x) {
            const int count = loose_count(x);
            if (count == 0) continue;
            const uint32_t seen = x == 0 ? 0xFFFFFFFFu : sh.any[x - 1];
            const uint32_t src = loose + (kLoose + 32 * x) * kLoosePitch + 2 * (32 * g + lane);
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float f[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int t = 2 * k + e;
                const bool on = t < count && ((seen >> t) & 1u) != 0;
                f[e] = on ? bits16_to_f32((uint16_t)lds16(src + t * kLoosePitch), p.in_dtype) : 0.f;
                if (!(fabsf(f[e]) <= 16376.f)) {
                  if (code != KITTY_ST_NONFINITE) code = fabsf(f[e]) <= 3.4028235e38f ? KITTY_ST_RANGE : KITTY_ST_NONFINITE;
                  f[e] = 0.f;
                }
              }
              w[k] = h2_bits(__floats2half2_rn(f[0] * up, f[1] * up));
            }
            tmem_st16(to + 16 * x, w);
            if (lane < 4) sts128(mids + st * 1024 + 256 * x + 64 * g + 16 * lane, make_uint4(0, 0, 0, 0));
          }
          if (code != KITTY_ST_OK) set_status(p.d_status, code);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_s(keys ? a_of(bar.kfull[st]) : a_of(bar.vfull[st]));
      }
    } else if (has_loose) {
      // the loose tokens' rows, swizzled as the tiled loads leave the others: 8 lanes a row half
      const int i = n - 1, st = i & 1;
      ok = wait_lanes(lane == 0, a_of(bar.loose[keys ? 0 : 1]), 0, p.wait_polls, abort);
      const uint32_t to = ops + (2 * st + (keys ? 0 : 1)) * Z::kTile16;
      if (ok) {
        int code = KITTY_ST_OK;
        const bool in = (sh.loose & 1) != 0;
        const int id = in ? p.block_table[(size_t)b * p.max_pages + hd.pages] : 0;
        const uint16_t* page = reinterpret_cast<const uint16_t*>(p.pool) + (((size_t)id * p.Hkv + kvh) * 2 + (keys ? 0 : 1)) * kPage * kD;
        const uint16_t* nodes = (keys ? p.k : p.v) + (size_t)hd.first * (keys ? p.k_stride : p.v_stride) + (size_t)kvh * kD;
        const size_t stride = keys ? p.k_stride : p.v_stride;
#pragma unroll 1
        for (int k0 = 0; k0 < kLoose * 16; k0 += 4 * 128) {
          uint4 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int at = k0 + 128 * k + 32 * g + lane, t = at >> 4, c = at & 15, part = t >> 5;
            const bool on = t < kLoose && (part == 0 ? (t & 31) < hd.loose && in : loose_seen(part, t & 31));
            v[k] = on ? *reinterpret_cast<const uint4*>((part == 0 ? page + (size_t)t * kD : nodes + (size_t)(t - 32) * stride) + 8 * c)
                      : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int at = k0 + 128 * k + 32 * g + lane, t = at >> 4, c = at & 15;
            if (t >= 32) {  // not a number: reported, and kept from those that do not see it
              const int e = mag_code(mag2(mag2(mag2(mag2(0, v[k].x), v[k].y), v[k].z), v[k].w), false, p.in_dtype);
              if (e != KITTY_ST_OK) {
                code = e;
                v[k] = make_uint4(0, 0, 0, 0);
              }
            }
            if (t < kLoose) sts128(to + (c >> 3) * Z::kHalf16 + t * 128 + (((c & 7) ^ (t & 7)) << 4), v[k]);
          }
        }
        if (code != KITTY_ST_OK) set_status(p.d_status, code);
      }
      fence_async_shared();
      group_sync(keys ? 3 : 4);
      if (ok && g == 0 && lane == 0) mbar_arrive_s(keys ? a_of(bar.kfull[st]) : a_of(bar.vfull[st]));
    }
    if (!ok && lane == 0) set_status(p.d_status, KITTY_ST_TIMEOUT);
    __syncwarp();
  } else if (wid == kMmaWarp) {
    // =========================================================== products
    constexpr uint32_t qk = mma_desc(F::kBf16, false, N);
    constexpr uint32_t pv = mma_desc(F::kBf16, true, N) | (F::kPacked ? 0u : 1u << 15);  // 16-bit Values: channels contiguous
    const uint64_t qdesc = smem_desc(qs, 16, 1024, kSwizzle128);
    const uint64_t pdesc = smem_desc(ps, Z::kPBlock, 1024, kSwizzle128);
    bool ok = true, started = false;
    auto scores = [&](int i) {
      const int st = i & 1, op = i % F::kOps;
      ok = wait_lanes(lane < 2, lane == 0 ? a_of(bar.kfull[op]) : a_of(bar.sempty[st]),
                      lane == 0 ? (i / F::kOps) & 1 : ((i >> 1) & 1) ^ 1, p.wait_polls, abort);
      if (!ok) return;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t d = tmem + F::kSCol + st * N;
#pragma unroll
        for (int k = 0; k < kD / 16; ++k) {
          const uint64_t qd = qdesc + (k >> 2) * (Z::kQHalf / 16) + 2 * (k & 3);
          if constexpr (F::kPacked) {
            mma_ts(d, tmem + 64 * op + 8 * k, qd, qk, k > 0);
          } else {
            const uint64_t kd = smem_desc(ops + 2 * op * Z::kTile16, 16, 1024, kSwizzle128);
            mma_ss(d, kd + (k >> 2) * (Z::kHalf16 / 16) + 2 * (k & 3), qd, qk, k > 0);
          }
        }
        mma_commit(a_of(bar.sfull[st]));
        mma_commit(a_of(bar.kempty[op]));
      }
      __syncwarp();
    };
    scores(0);
    for (int i = 0; ok && i < n; ++i) {
      const int st = i & 1, op = i % F::kOps;
      if (i + 1 < n) {
        scores(i + 1);
        if (!ok) break;
      }
      ok = wait_lanes(lane < 2, lane == 0 ? a_of(bar.pfull[st]) : a_of(bar.vfull[op]), lane == 0 ? (i >> 1) & 1 : (i / F::kOps) & 1,
                      p.wait_polls, abort);
      if (!ok) break;
      tc_fence_after();
      const int there = there_of(i);
      if (elect_one()) {
        const uint32_t d = tmem + Z::kOCol;
        const uint64_t pd = pdesc + st * (Z::kP / 16);
        bool acc = started;
#pragma unroll 1
        for (int g = 0; g < kTilePages; ++g) {
          if (!((there >> g) & 1)) continue;
#pragma unroll
          for (int k = 2 * g; k < 2 * g + 2; ++k) {
            if constexpr (F::kPacked) {
              mma_ts(d, tmem + F::kVCol + 64 * op + 8 * k, pd + 128 * k, pv, acc);
            } else {
              const uint64_t vd = smem_desc(ops + (2 * op + 1) * Z::kTile16, Z::kHalf16, 1024, kSwizzle128) + 128 * k;
              mma_ss(d, vd, pd + 128 * k, pv, acc);
              mma_ss(d, vd, pd + Z::kPHalf / 16 + 128 * k, pv, true);
            }
            acc = true;
          }
        }
        mma_commit(a_of(bar.vempty[op]));
        mma_commit(a_of(bar.pempty[st]));
      }
      started = started || there != 0;
      __syncwarp();
    }
    if (!ok && lane == 0) set_status(p.d_status, KITTY_ST_TIMEOUT);
    __syncwarp();
  } else if (!F::kPacked && (wid == kFetchWarp || wid == kBiasWarp)) {
    // =========================================================== tiled loads: a warp the Keys', one the Values'
    const bool values = wid == kBiasWarp;
    bool ok = true;
    int ids = -1;  // lane l: the id of page l of the eight tiles at hand
    for (int i = 0; i < n; ++i) {
      const int st = i & 1;
      const uint32_t full = values ? a_of(bar.vfull[st]) : a_of(bar.kfull[st]);
      ok = wait_lanes(true, values ? a_of(bar.vempty[st]) : a_of(bar.kempty[st]), ((i >> 1) & 1) ^ 1, p.wait_polls, abort);
      if (!ok) break;
      if (has_loose && i == n - 1) {  // room for the loose tokens: this warp has followed every use of the stage
        if (elect_one()) mbar_arrive_s(a_of(bar.loose[values ? 1 : 0]));
        break;
      }
      if ((i & 7) == 0) {
        const int x = (t0 + i) * kTilePages + lane;
        ids = x >= pages ? -1 : x < hd.prefix ? p.prefix_table[x] : p.block_table[(size_t)b * p.max_pages + x - hd.prefix];
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
        ids = x >= pages || (i + lane / 4) >= n ? -1 : x < hd.prefix ? p.prefix_table[x] : p.block_table[(size_t)b * p.max_pages + x - hd.prefix];
      }
      const int id = __shfl_sync(0xFFFFFFFFu, ids, 4 * (i - ids_at) + (lane & 3));
      const bool in = id >= 0 && id < p.pool_pages;
      const int there = __ballot_sync(0xFFFFFFFFu, in) & 15;
      if (lane < 4 && !in && (t0 + i) * kTilePages + lane < pages) set_status(p.d_status, KITTY_ST_BAD_PAGE);
      if constexpr (F::kPacked) {
        ok = wait_lanes(lane == 0, a_of(bar.freed[slot]), (turn & 1) ^ 1, p.wait_polls, abort);
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
  } else if (wid == kBiasWarp) {
    // =========================================================== q.M
    if constexpr (F::kPacked) {
      const int r = lane >> 2, qq = lane & 3;
      bool ok = true;
      int slot = 0, turn = 0;
      const uint32_t km = 512 * F::W + 4 * F::W * p.n_hi + 256;
      for (int i = 0; i < n; ++i) {
        const int st = i & 1;
        const bool special = has_loose && i == n - 1;
        ok = wait_lanes(lane < (special ? 1 : 2), lane == 0 ? a_of(bar.sempty[st]) : a_of(bar.raw[slot]),
                        lane == 0 ? ((i >> 1) & 1) ^ 1 : turn & 1, p.wait_polls, abort);
        if (!ok) break;
        if (special) {
          for (int x = lane; x < 4 * N; x += 32) (&sh.bias[st][0][0])[x] = 0.f;
        } else {
          uint32_t M[16];
          const uint32_t at = raws + (slot * kTilePages + (r & 3)) * p.blob + km + 64 * qq;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 v = lds128(at + 16 * k);
            M[4 * k] = r < 4 ? v.x : 0;
            M[4 * k + 1] = r < 4 ? v.y : 0;
            M[4 * k + 2] = r < 4 ? v.z : 0;
            M[4 * k + 3] = r < 4 ? v.w : 0;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_s(a_of(bar.freed[slot]));
#pragma unroll 2
          for (int nt = 0; nt < N / 8; ++nt) {
            float c[4] = {}, d[4] = {};
            const int row = 8 * nt + (lane & 7);
#pragma unroll
            for (int jp = 0; jp < 4; ++jp) {
              uint32_t q4[4];
              ldsm_x4(qs + (jp >> 1) * Z::kQHalf + row * 128 + (((4 * (jp & 1) + (lane >> 3)) ^ (row & 7)) << 4), q4);
              const uint32_t a0[4] = {M[4 * jp], 0u, M[4 * jp + 1], 0u}, a1[4] = {M[4 * jp + 2], 0u, M[4 * jp + 3], 0u};
              mma_f16(c, a0, q4[0], q4[1]);
              mma_f16(d, a1, q4[2], q4[3]);
            }
            if (r < 4) *reinterpret_cast<float2*>(&sh.bias[st][r][8 * nt + 2 * qq]) = make_float2(c[0] + d[0], c[1] + d[1]);
          }
          if (++slot == p.raw_stages) {
            slot = 0;
            ++turn;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_s(a_of(bar.bias[st]));
      }
      if (!ok && lane == 0) set_status(p.d_status, KITTY_ST_TIMEOUT);
    }
    __syncwarp();
  } else {
    // =========================================================== sums of p, of p * middles
    const int r = lane >> 2, qq = lane & 3;
    float c[N / 8][4];
#pragma unroll
    for (int nt = 0; nt < N / 8; ++nt) c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.f;
    constexpr uint32_t one = F::kBf16 ? two(0x3F80) : two(0x3C00);
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int st = i & 1, op = i % F::kOps;
      ok = wait_lanes(lane < (F::kPacked ? 2 : 1), lane == 0 ? a_of(bar.pfull[st]) : a_of(bar.vfull[op]),
                      lane == 0 ? (i >> 1) & 1 : (i / F::kOps) & 1, p.wait_polls, abort);
      if (!ok) break;
      const int there = there_of(i);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (i > 0 && sh.moved[st][h]) {
#pragma unroll
          for (int nt = h * (N / 16); nt < (h + 1) * (N / 16); ++nt) {
            c[nt][0] *= sh.f[st][8 * nt + 2 * qq];
            c[nt][1] *= sh.f[st][8 * nt + 2 * qq + 1];
          }
        }
#pragma unroll 1
      for (int g = 0; g < kTilePages; ++g) {
        if (!((there >> g) & 1)) continue;
        uint4 a4 = make_uint4(0, 0, 0, 0);
        if (F::kPacked && r < 4) a4 = lds128(mids + op * 1024 + 256 * g + 64 * r + 16 * qq);
        if (r == 4) a4 = make_uint4(one, one, one, one);
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
          const uint32_t a[4] = {kt ? a4.z : a4.x, 0u, kt ? a4.w : a4.y, 0u};
          const int token = 32 * g + 16 * kt + 8 * ((lane >> 3) & 1) + (lane & 7);
#pragma unroll
          for (int pr = 0; pr < (F::kPair ? 2 : 1); ++pr) {
#pragma unroll
            for (int np = 0; np < N / 16; ++np) {
              const int chunk = 2 * np + (lane >> 4);
              uint32_t b4[4];
              ldsm_x4_t(ps + st * Z::kP + pr * Z::kPHalf + (chunk >> 3) * Z::kPBlock + token * 128 + (((chunk & 7) ^ (token & 7)) << 4), b4);
              mma16<F::kBf16 ? KITTY_BF16 : KITTY_F16>(c[2 * np], a, b4[0], b4[1]);
              mma16<F::kBf16 ? KITTY_BF16 : KITTY_F16>(c[2 * np + 1], a, b4[2], b4[3]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_s(a_of(bar.pempty[st]));
        if (F::kPacked) mbar_arrive_s(a_of(bar.vempty[op]));
      }
    }
    if (ok) {
#pragma unroll
      for (int nt = 0; nt < N / 8; ++nt) {
        if (r < 4) *reinterpret_cast<float2*>(&sh.mid[r][8 * nt + 2 * qq]) = make_float2(c[nt][0], c[nt][1]);
        if (r == 4) *reinterpret_cast<float2*>(&sh.sum[8 * nt + 2 * qq]) = make_float2(c[nt][0], c[nt][1]);
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
}

// ------------------------------------------------------------- merge of the splits
// A warp a row (query head of a drafted token), four channels a lane; eight partials requested at
// once, with the row's maxima, a lane a split.
template <bool PACKED>
__global__ void __launch_bounds__(128) tree_merge_kernel(const TreeParams p) {
  const int b = blockIdx.y, lane = threadIdx.x & 31, i = blockIdx.x * 4 + (threadIdx.x >> 5);
  const Held hd = held_of<PACKED>(p, b);
  if (!hd.ok || i >= hd.n * p.Hq) return;
  const size_t row = (size_t)hd.first * p.Hq + i;
  const float* part = p.ws + row * p.splits * kPartialFloats;
  grid_wait();
  const float2 ml = lane < p.splits ? *reinterpret_cast<const float2*>(part + lane * kPartialFloats) : make_float2(-INFINITY, 0.f);
  float m = ml.x;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
  const float e = ml.x == -INFINITY ? 0.f : ex2a(ml.x - m);
  float l = e == 0.f ? 0.f : ml.y * e;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < p.splits; s0 += 8) {
    float4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      x[k] = s0 + k < p.splits ? reinterpret_cast<const float4*>(part + (s0 + k) * kPartialFloats + 4)[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float w = __shfl_sync(0xFFFFFFFFu, e, (s0 + k) & 31);
      if (s0 + k < p.splits && w != 0.f) {
        o.x = fmaf(x[k].x, w, o.x);
        o.y = fmaf(x[k].y, w, o.y);
        o.z = fmaf(x[k].z, w, o.z);
        o.w = fmaf(x[k].w, w, o.w);
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
struct TreePlan {
  int rows, units, splits;  // rows of a block, blocks of a (sequence, kv head), splits of its tiles
};

// Rows of a block: the least of 16, 32, 64, 128 (16-bit pages: 64) that holds the largest tree's.
// Splits: a block has an SM to itself, so as many as make the last round of blocks end soonest, with
// a block's time its tiles' and a fixed part.
TreePlan tree_plan_of(const kitty_cfg* cfg, bool packed, int B, int max_nodes, int n_prefix, int max_pages) {
  const int rows = max_nodes * (cfg->num_q_heads / cfg->num_kv_heads);
  TreePlan pl = {16, 1, 1};
  while (pl.rows < rows && pl.rows < (packed ? 128 : 64)) pl.rows *= 2;
  pl.units = (rows + pl.rows - 1) / pl.rows;
  const double tile_us = packed ? (pl.rows <= 32 ? 0.5 : pl.rows == 64 ? 0.7 : 1.1) : 1.5, fixed_us = 4.0;
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
    }
  }
  return pl;
}

size_t partial_bytes(const kitty_cfg* cfg, const TreePlan& pl, int n_tokens) {
  return pl.splits > 1 ? (size_t)n_tokens * cfg->num_q_heads * pl.splits * kPartialFloats * sizeof(float) : 0;
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

int workspace(const kitty_cfg* cfg, bool packed, int B, int n_tokens, int max_nodes, int n_prefix, int max_pages,
              size_t* bytes) {
  const int rc = check_tree(cfg, B, n_tokens, max_nodes, n_prefix, max_pages);
  if (rc != KITTY_OK) return rc;
  if (!bytes) return KITTY_ERR_INVALID_ARG;
  *bytes = B == 0 || n_tokens == 0 ? 0 : partial_bytes(cfg, tree_plan_of(cfg, packed, B, max_nodes, n_prefix, max_pages), n_tokens);
  return KITTY_OK;
}

template <class F>
int launch_tree(TreeParams& p, const CUtensorMap& map, cudaStream_t s) {
  using Z = Sizes<F>;
  static_assert(Z::kCols <= 512, "fits tensor memory");
  constexpr int kMost = 227 * 1024 - (int)((sizeof(Shared<F::N>) + 127) / 128 * 128);
  constexpr int kFixed = 1024 + Z::kFixed;
  static_assert(kFixed + (F::kPacked ? 4 * (F::W == 2 ? 4224 : F::V == 2 ? 6272 : 7296) : 0) <= kMost, "one stage at least");
  // one block an SM: two would wait for each other's tensor memory
  static_assert(kFixed + (int)sizeof(Shared<F::N>) > 100 * 1024 || F::kPacked, "one block an SM");
  int smem = kFixed;
  if (F::kPacked) {
    p.raw_stages = std::min(kMaxRaw, (kMost - kFixed) / (kTilePages * p.blob));
    smem = std::max(kFixed + p.raw_stages * kTilePages * p.blob, 116 * 1024);
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
                                (size_t)smem, s, false, p, map);
  if (e == cudaSuccess && p.splits > 1)
    e = launch_dependent(tree_merge_kernel<F::kPacked>, dim3((unsigned)((p.max_nodes * p.Hq + 3) / 4), (unsigned)p.B), 128, 0, s, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? KITTY_OK : KITTY_ERR_CUDA;
}

template <int W, int V>
int launch_packed(TreeParams& p, int rows, cudaStream_t s) {
  const CUtensorMap map = {};
  switch (rows) {
    case 16: return launch_tree<PackedTree<W, V, 16>>(p, map, s);
    case 32: return launch_tree<PackedTree<W, V, 32>>(p, map, s);
    case 64: return launch_tree<PackedTree<W, V, 64>>(p, map, s);
    default: return launch_tree<PackedTree<W, V, 128>>(p, map, s);
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
                void* ws, size_t ws_bytes, int32_t B, int32_t* d_status, bool packed, int* rows, TreeParams* p) {
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
  const TreePlan pl = tree_plan_of(cfg, packed, B, max_nodes, n_prefix, max_pages);
  const size_t need = partial_bytes(cfg, pl, n_tokens);
  if (ws_bytes < need || (need > 0 && (!ws || !aligned16(ws)))) return KITTY_ERR_WORKSPACE;
  if ((uint64_t)pl.units * Hkv * B > 0x7FFFFFFFull || B > 65535) return KITTY_ERR_UNSUPPORTED;
  *rows = pl.rows;
  p->units = pl.units;
  p->splits = pl.splits;
  p->ws = static_cast<float*>(ws);
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
  int rows = 0;
  const int rc = tree_params(cfg, q, q_stride, k, k_stride, v, v_stride, n_tokens, seq_start, visible, max_nodes,
                             pool, pool_pages, prefix_table, n_prefix, prefix_pages, block_table, max_pages,
                             sm_scale, out, out_dtype, workspace, workspace_bytes, B, d_status, true, &rows, &p);
  if (rc != KITTY_OK) return rc == 1 ? KITTY_OK : rc;
  if (!num_pages || !tail_len || !tail_k || !tail_v || !aligned16(tail_k) || !aligned16(tail_v))
    return KITTY_ERR_INVALID_ARG;
  p.num_pages = num_pages;
  p.tail_len = tail_len;
  p.tail_k = static_cast<const uint16_t*>(tail_k);
  p.tail_v = static_cast<const uint16_t*>(tail_v);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cfg->lo_bit == 2) return launch_packed<2, 2>(p, rows, s);
  return v_bits(cfg) == 2 ? launch_packed<4, 2>(p, rows, s) : launch_packed<4, 4>(p, rows, s);
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
  int rows = 0;
  const int rc = tree_params(cfg, q, q_stride, k, k_stride, v, v_stride, n_tokens, seq_start, visible, max_nodes,
                             pool, pool_pages, prefix_table, n_prefix, prefix_pages, block_table, max_pages,
                             sm_scale, out, out_dtype, workspace, workspace_bytes, B, d_status, false, &rows, &p);
  if (rc != KITTY_OK) return rc == 1 ? KITTY_OK : rc;
  if (!ctx_len) return KITTY_ERR_INVALID_ARG;
  p.ctx_len = ctx_len;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cfg->in_dtype == KITTY_BF16 ? launch_plain<true>(p, rows, s) : launch_plain<false>(p, rows, s);
}
