// Attention of a whole batch's queries to the pages that its sequences share, on the
// fifth-generation tensor cores (sm_103a).
//
// Rows.  All query heads of a kv head over all sequences attend the same Keys and Values:
// R = B * Hq / Hkv rows.  One block takes up to 256 of them, as two tiles of 128 (the two
// "lanes" below), and a contiguous split of the prefix; with R <= 128 both lanes hold the
// same 128 rows and take alternate tiles of the split.  Per tile of kTok tokens and lane:
//   S = Q K^T          tcgen05.mma, 128 x kTok x 128, fp32 in tensor memory
//   p = 2^(s - m)      one thread a row: its scores from tensor memory, the running maximum
//                      and sum in registers, p back over S as the next product's operand
//   O += P V           tcgen05.mma with P in tensor memory, fp32 in tensor memory
// m is not the maximum itself: it is set 2^4 below the first tile's, and moves only when a score
// passes it by more than 2^15, so that O is hardly ever rescaled (a rescale costs the lane about
// a tile's time) and p <= 32768 stays inside fp16.  It is set below because p has fp16's range
// downwards, too: what is 2^-25 and less becomes 0, and 15000 tokens of 2^-19 of one large one
// each are 3% of its sum.  Here they would have to be 2^-29 of it.
// Warps: 4 a lane for the softmax, one a lane issuing products, the rest loading.  While one
// lane's softmax runs, the tensor cores work on the other's products.
//
// Packed pages (tiles of three pages).  A loading warp takes one page's Keys or Values of
// each tile, staged by bulk copies, and writes operands to shared memory in fp16:
//   Keys    step * code, exact (a step has 7 significant bits, a code 2 or 4); the page's
//           channel minima as one more row, so that Q K^T also gives q.M, which the
//           softmax adds to the page's 32 scores;
//   Values  step * (code - half the largest code), exact, transposed; the middles of each
//           token's four groups (minimum + half the largest code * step) as four more
//           channels, which the end adds to the channels of their group; and a channel of
//           ones, whose column of O is the sum of the rounded p.
// So the roundings are p to fp16, a group's middle to fp16 (2^-11 of it at most, once) and, for
// 8-bit boosted Keys, step * code to fp16; with the sum taken over the rounded p, theirs shift
// an output by at most 2^-11 of sum p |v - out|.  Why middles: codes from 0 and minima, which
// are exact, are sums that grow with the context and cancel, and the products' fp32
// accumulation rounds them one way: 16000 tokens a block left outputs off by 3.6e-3 of their
// RMS, all to one side.  Centered, both sums stay near the output's size.
//
// What bounds it.  Packed, 128 sequences of 64/8 heads behind 32768 tokens (32 x 4 blocks of 86
// tiles): 1.7 us a tile of both lanes; of the issue slots of the SMs in use 64% are taken (97.8 M
// warp instructions, near half of them writing operands), the tensor pipe is busy 50%, memory
// 2%.  Two blocks that share a tile's operands through a cluster would halve the writing for
// batches of more than 256 rows; that is not done.  A few tiles a block: fixed costs, about
// 7 tiles' time from launch to the last partial (first loads and queries, cold instructions, a
// row's 528 bytes out).  16-bit pages: 2 us a tile, 64 sequences behind 8192 tokens 29 us
// (8 x 8 blocks), the tensor pipe's two products per probability and the softmax by turns.
//
// 16-bit pages (tiles of four pages) come by tiled TMA loads, swizzled, the Values as they
// lie (N contiguous).  There is no room for a channel of ones beside 128 scores, and one bf16
// p would leave an error of 2^-9: p is a (high, rest) pair, its sum taken in registers.
//
// Masks.  Sequence b sees its first prefix_pages[b] pages.  Its rows' probabilities are 0 for
// later pages, and the products with those pages' Values leave its rows alone (the
// product's lane mask), so nothing in them can reach it.
#include "prefix.h"

#include <algorithm>
#include <atomic>

#include "grid_dep.cuh"
#include "host_common.h"
#include "kitty_common.cuh"
#include "partials.h"
#include "tcgen05.cuh"

namespace kitty {
namespace {

constexpr int kRows = 256;                // rows of a block: two lanes of 128
constexpr int kQBytes = kRows * kD * 2;   // the queries' operand: [channel half][row][128 bytes]
constexpr int kQHalf = kRows * 128;
constexpr int kStages = 2;                // of Keys and of Values
constexpr int kFlags = 8;                 // tiles whose page flags are kept
constexpr uint32_t kPrefixWaitPolls = 1u << 22;
constexpr int kSoftmaxWarps = 8;
constexpr int kMmaWarp = 8;               // and the next: one a lane
constexpr int kLoadWarp = 10;
constexpr float kFloor = -1.0e30f;        // a row without a score yet
constexpr float kSlack = 15.f;            // log2 units that a score may pass m by
constexpr float kMargin = -4.f;           // m against the maximum, when it is set

// Packed pages: Key planes of W bits, Values of V bits.
template <int W_, int V_>
struct PackedFmt {
  static constexpr bool kPacked = true, kBf16 = false, kPair = false;
  static constexpr int W = W_, V = V_, kPages = 3, kTok = 96;
  static constexpr int kS = 112;          // columns of S: 96 scores, 3 of q.M (16 is the granule)
  static constexpr int kO = 144;          // columns of O: 128 channels, 4 group middles, the sum of p
  static constexpr int kKHalf = kS * 128, kKBytes = 2 * kKHalf;
  static constexpr int kSlab = kO * 64;   // a page's Values: [channel][64 bytes]
  static constexpr int kVBytes = kPages * kSlab;
  // two warps for a page's Keys (64 channels each), one for its Values, and one that fetches
  static constexpr int kLoadWarps = 3 * kPages + 1;
  static constexpr int kRaw = W == 2 ? 4 : 2;                // staged tiles
  static constexpr int kRawK = 512 * W + 128 * 4 * W + 512 + 128;  // at n_hi = 128
  static constexpr int kRawV = 512 * V + 512;
  static constexpr int kRawBytes = kPages * kRaw * (kRawK + kRawV);
};

// 16-bit pages.
template <bool BF>
struct PlainFmt {
  static constexpr bool kPacked = false, kBf16 = BF, kPair = true;
  static constexpr int kPages = 4, kTok = 128, kS = 128, kO = 128;
  static constexpr int kKHalf = kTok * 128, kKBytes = 2 * kKHalf, kVBytes = kKBytes;
  static constexpr int W = 0, kSlab = 0, kLoadWarps = 2, kRaw = 1, kRawK = 0, kRawV = 0, kRawBytes = 0;
};

template <class F>
__host__ __device__ constexpr int threads_of() { return 32 * (kLoadWarp + F::kLoadWarps); }
template <class F>
__host__ __device__ constexpr int smem_of() { return 1024 + kQBytes + kStages * (F::kKBytes + F::kVBytes) + F::kRawBytes; }

struct Bars {
  uint64_t kfull[kStages], kempty[kStages], vfull[kStages], vempty[kStages];
  uint64_t sfull[2], pready[2], ofull[2], qready[2], drain[2], turn[2];
  uint64_t raw[6][4], freed[6][4], based[3];  // items: a tile's pages' Keys, then their Values
};

struct Shared {
  Bars bars;
  uint32_t tmem;
  int abort;
  int maxpages, minpages;          // that a row of the block sees
  int row[kRows];                  // partials' row (sequence, query head); -1: padding
  uint8_t got[kFlags][4];               // packed pages that were fetched, by tile
  alignas(4) uint8_t valid[kFlags][4];  // page ids in range, by tile
  alignas(16) uint32_t off[2][4][4];  // by lane and page: rows that do not see it, 32 a word
};

// Whole warp: waits for each lane's phase (need: it has one), at most `polls` polls; false when
// it, or another warp of the block, has given up.  Several barriers in one wait, a lane each,
// cost no more than one: a wait that is over already takes 100 to 200 cycles.
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

__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, uint32_t polls, volatile int* abort) {
  return wait_lanes(true, smem_u32(bar), parity, polls, abort);
}

__device__ __forceinline__ float ex2a(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
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
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"((uint16_t)v) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint32_t h2mul(uint32_t a, uint32_t b) { return h2_bits(__hmul2(bits_h2(a), bits_h2(b))); }

// Both halves' codes of class K of a plane word as fp16 integers.  2-bit planes: class
// K = token or channel block 0..3, at bits 2K + 2; 4-bit planes: K = 0, 1, at bits 4K + 2.  A
// code under the exponent of 1024 reads 1024 + code * 2^shift; one fused multiply-add
// takes both off, exactly.  CENTERED: minus half the largest code, as exact.
template <int BITS, int K, bool CENTERED = false>
__device__ __forceinline__ uint32_t codes(uint32_t x) {
  constexpr int shift = BITS * K + 2;
  constexpr uint32_t mask = (((1u << BITS) - 1u) << shift) * 0x00010001u;
  const uint32_t y = (x & mask) | 0x64006400u;
  constexpr uint32_t inv = ((15u - shift) << 10) * 0x00010001u;             // 2^-shift
  constexpr uint32_t half = CENTERED ? ((1u << BITS) - 1u) << (shift - 1) : 0u;  // in the mantissa's units
  constexpr uint32_t off = ((25u - shift) << 10 | 0x8000u | half) * 0x00010001u;  // -1024 * 2^-shift - half
  return h2_bits(__hfma2(bits_h2(y), bits_h2(inv), bits_h2(off)));
}

// A stored step so large that a step times a code may leave fp16.
template <int BITS>
__device__ __forceinline__ bool step_too_large(uint32_t pair) {
  const float2 f = __half22float2(bits_h2(pair));
  return !(fmaxf(f.x, f.y) * (float)(1 << BITS) <= 65504.f);
}

// Channels 64 half .. of a page's Key part (staged at raw, as in the page up to the channel
// list) to rows 32 page .. of the stage, and their minima to row kTok + page.  Lane (r, qq)
// holds tokens r, r + 8, r + 16, r + 24 of the channels 16j + 8h + 2qq + {0, 1}: pairs of
// channels, and the eight rows of a warp's store lie in different swizzled 16-byte columns.
// `based`: called between the base plane and the boosted channels; returns when both halves
// are at that point (false: given up).
template <class F, class Based>
__device__ __forceinline__ bool put_keys(uint32_t raw, uint32_t stage, int page, int half, int n_hi, int32_t* d_status, Based based) {
  constexpr int W = F::W;
  const int lane = threadIdx.x & 31, r = lane >> 2, qq = lane & 3;
  const uint32_t ks = raw + 512 * W + 4 * W * n_hi, km = ks + 256, kch = km + 256;
  const uint32_t dst = stage + half * F::kKHalf, row = dst + (32 * page + r) * 128 + 16 * r;  // + swizzle
  uint32_t w[2 * W];  // this lane's words of the half: one (W = 2) or two a j
#pragma unroll
  for (int i = 0; i < W / 2; ++i) {
    const uint4 v = lds128(raw + 16 * W * lane + 8 * W * half + 16 * i);
    w[4 * i] = v.x;
    w[4 * i + 1] = v.y;
    w[4 * i + 2] = v.z;
    w[4 * i + 3] = v.w;
  }
  const uint32_t sq = ks + 128 * half + 4 * qq;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t S = lds32(sq + 32 * j + 16 * h);
      const uint32_t at = (row ^ (16 * (2 * j + h))) + 4 * qq;
#pragma unroll
      for (int mt = 0; mt < W / 2; ++mt) {
        const uint32_t y = w[W / 2 * j + mt], x = h ? __funnelshift_r(y, y, 8) : y;
        if (W == 2) {
          sts32(at, h2mul(codes<2, 0>(x), S));
          sts32(at + 1024, h2mul(codes<2, 1>(x), S));
          sts32(at + 2 * 1024, h2mul(codes<2, 2>(x), S));
          sts32(at + 3 * 1024, h2mul(codes<2, 3>(x), S));
        } else {
          sts32(at + 2048 * mt, h2mul(codes<4, 0>(x), S));
          sts32(at + 2048 * mt + 1024, h2mul(codes<4, 1>(x), S));
        }
      }
    }
  }
  {  // minima of channels 64 half + 2 lane, + 1; their steps' range (boosted: times 2^W at most)
    const int c = 64 * half + 2 * lane, m = F::kTok + page;
    const uint32_t v = lds32(km + 4 * ((((c >> 1) & 3) * 8 + (c >> 4)) * 2 + ((c >> 3) & 1)));
    sts32(dst + m * 128 + (((lane >> 2) ^ (m & 7)) << 4) + 4 * (lane & 3), v);
    if (step_too_large<W>(lds32(ks + 2 * c))) set_status(d_status, KITTY_ST_RANGE);
  }
  if (n_hi == 0) return true;
  if (!based()) return false;
  // Boosted channels again, from both planes: step * high + step / 2^W * low.  This lane's
  // columns of the extra plane are pairs too, of any two channels: their words of the base
  // plane lie in the lanes of the same tokens.  The halves take alternate groups of 16.
  const uint32_t part = W == 2 ? 0x34003400u : 0x2C002C00u;  // 1/4, 1/16
  const int nx = n_hi / 16;
  const uint32_t lo_plane = raw + 512 * W + 2 * W * nx * lane, hi_plane = raw + 64 * W * r;
  const uint32_t row0 = stage + (32 * page + r) * 128 + 16 * r;
#pragma unroll 1
  for (int js = half; js < nx; js += 2) {
    const uint32_t ids = lds32(kch + 16 * js + 4 * qq);
    uint32_t lo[2];
    lo[0] = lds32(lo_plane + 2 * W * js);
    lo[1] = W == 4 ? lds32(lo_plane + 2 * W * js + 4) : 0;
    uint32_t at[4], st[4], hi[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t c = (ids >> (8 * i)) & 127u;
      st[i] = lds16(ks + 2 * c);
      const uint32_t from = hi_plane + 8 * W * (c & 6) + 2 * W * (c >> 4);
#pragma unroll
      for (int mt = 0; mt < W / 2; ++mt) {
        const uint32_t x = lds32(from + 4 * mt);
        hi[i][mt] = __funnelshift_r(x, x, (c & 8) + 16 * (c & 1));  // the channel's codes in the low half
      }
      at[i] = (row0 ^ ((2 * c) & 0x7Eu)) + (c >> 6) * F::kKHalf;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t s = __byte_perm(st[2 * h], st[2 * h + 1], 0x5410), sl = h2mul(s, part);
      auto put = [&](int tau, uint32_t ch, uint32_t cl) {
        const uint32_t v = h2_bits(__hfma2(bits_h2(ch), bits_h2(s), bits_h2(h2mul(cl, sl))));
        sts16(at[2 * h] + 1024 * tau, v);
        sts16(at[2 * h + 1] + 1024 * tau, v >> 16);
      };
#pragma unroll
      for (int mt = 0; mt < W / 2; ++mt) {
        const uint32_t xh = __byte_perm(hi[2 * h][mt], hi[2 * h + 1][mt], 0x5410);
        const uint32_t xl = h ? __funnelshift_r(lo[mt], lo[mt], 8) : lo[mt];
        if (W == 2) {
          put(0, codes<2, 0>(xh), codes<2, 0>(xl));
          put(1, codes<2, 1>(xh), codes<2, 1>(xl));
          put(2, codes<2, 2>(xh), codes<2, 2>(xl));
          put(3, codes<2, 3>(xh), codes<2, 3>(xl));
        } else {
          put(2 * mt, codes<4, 0>(xh), codes<4, 0>(xl));
          put(2 * mt + 1, codes<4, 1>(xh), codes<4, 1>(xl));
        }
      }
    }
  }
  return true;
}

// A page's Value part (staged at raw: plane, steps, minima) to its slab, channels as rows of
// 32 tokens, the four groups' middles as rows 128 .. 131.  (Rolled over pairs of groups: loading
// warps, softmax and products share one instruction cache; with everything unrolled the
// first page of a block took 4000 to 8700 cycles, each later one 2200 to 3300.)
template <class F>
__device__ __forceinline__ void put_values(uint32_t raw, uint32_t slab, int32_t* d_status) {
  constexpr int V = F::V;
  const int lane = threadIdx.x & 31, r = lane >> 2, qq = lane & 3;
  const uint32_t vs = raw + 512 * V, vm = vs + 256;
  const uint32_t sw = (r >> 1) & 3;
#pragma unroll 1
  for (int G0 = 0; G0 < 4; G0 += 2) {
    uint32_t w[2 * V];  // of two groups: one (V = 2) or two a kt
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const uint4 v = lds128(raw + 16 * V * lane + 4 * V * G0 + 16 * i);
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
#pragma unroll
    for (int G = 0; G < 2; ++G) {
      const uint4 s4 = lds128(vs + 64 * (G0 + G) + 16 * qq);
      const uint32_t S[4] = {s4.x, s4.y, s4.z, s4.w};
      const uint32_t row = slab + (32 * (G0 + G) + r) * 64 + 16 * sw;
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t s = S[2 * kt + h], at = (row ^ (16 * (2 * kt + h))) + 4 * qq;
#pragma unroll
          for (int mc = 0; mc < V / 2; ++mc) {
            const uint32_t y = w[V * G + V / 2 * kt + mc], x = h ? __funnelshift_r(y, y, 8) : y;
            if (V == 2) {
              sts32(at, h2mul(codes<2, 0, true>(x), s));
              sts32(at + 512, h2mul(codes<2, 1, true>(x), s));
              sts32(at + 1024, h2mul(codes<2, 2, true>(x), s));
              sts32(at + 1536, h2mul(codes<2, 3, true>(x), s));
            } else {
              sts32(at + 1024 * mc, h2mul(codes<4, 0, true>(x), s));
              sts32(at + 1024 * mc + 512, h2mul(codes<4, 1, true>(x), s));
            }
          }
        }
      }
    }
  }
  if (r < 4) {  // group r's middles of the tokens of column qq
    const uint4 m4 = lds128(vm + 64 * r + 16 * qq), s4 = lds128(vs + 64 * r + 16 * qq);
    const uint32_t m[4] = {m4.x, m4.y, m4.z, m4.w}, S[4] = {s4.x, s4.y, s4.z, s4.w};
    const uint32_t half = V == 2 ? 0x3E003E00u : 0x47804780u;  // 1.5, 7.5
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sts32(slab + (kD + r) * 64 + ((i ^ sw) << 4) + 4 * qq, h2_bits(__hfma2(bits_h2(S[i]), bits_h2(half), bits_h2(m[i]))));
  }
  if (step_too_large<V>(lds32(vs + 4 * lane)) || step_too_large<V>(lds32(vs + 128 + 4 * lane)))
    set_status(d_status, KITTY_ST_RANGE);
}

// Eight queries' channels (16 bytes) in the operand's type; a negative scale is taken as
// its magnitude and the negated query.
template <class F>
__device__ __forceinline__ uint4 query16(uint4 v, int in_dtype, bool negate) {
  uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (F::kPacked && in_dtype == KITTY_BF16)
      x[i] = h2_bits(__floats2half2_rn(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xFFFF0000u)));
    if (negate) x[i] ^= 0x80008000u;
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

__device__ __forceinline__ uint64_t pair64(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}

// Two probabilities in the operand's type; kPair: (high, rest).
template <class F>
__device__ __forceinline__ uint32_t pack_probs(float e0, float e1, uint32_t& rest) {
  if (!F::kBf16) {
    const __half2 h = __floats2half2_rn(e0, e1);
    if (F::kPair) {
      const float2 f = __half22float2(h);
      rest = h2_bits(__floats2half2_rn(e0 - f.x, e1 - f.y));
    }
    return h2_bits(h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(e0, e1);
  const uint32_t hi = *reinterpret_cast<const uint32_t*>(&h);
  const __nv_bfloat162 r = __floats2bfloat162_rn(e0 - __uint_as_float(hi << 16), e1 - __uint_as_float(hi & 0xFFFF0000u));
  rest = *reinterpret_cast<const uint32_t*>(&r);
  return hi;
}

template <class F>
__global__ void __launch_bounds__(threads_of<F>(), 1) prefix_kernel(const PrefixArgs p,
                                                                    const __grid_constant__ CUtensorMap map) {
  extern __shared__ uint8_t dyn[];
  __shared__ Shared sh;
  grid_trigger();  // the own pages' blocks may fill the SMs that are free, or get free
  const int tid = threadIdx.x, lane = tid & 31;
  const int wid = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // the compiler sees a warp-uniform role
  const int R = p.B * p.g, units = (R + kRows - 1) / kRows;
  const int kvh = blockIdx.x / units, unit = blockIdx.x - kvh * units, split = blockIdx.y;
  const bool both = R > 128;  // two lanes of rows; else the lanes share the rows and alternate
  volatile int* abort = &sh.abort;

  const uint32_t base = (smem_u32(dyn) + 1023u) & ~1023u;
  const uint32_t kst = base + kQBytes, vst = kst + kStages * F::kKBytes, raws = vst + kStages * F::kVBytes;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.bars.kfull[i], F::kPacked ? 2 * F::kPages : 1);
      mbar_init(&sh.bars.vfull[i], F::kPacked ? F::kPages : 1);
      mbar_init(&sh.bars.kempty[i], both ? 2 : 1);
      mbar_init(&sh.bars.vempty[i], both ? 2 : 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.bars.sfull[i], 1);
      mbar_init(&sh.bars.pready[i], 128);
      mbar_init(&sh.bars.ofull[i], 1);
      mbar_init(&sh.bars.qready[i], 128);
      mbar_init(&sh.bars.drain[i], 1);
      mbar_init(&sh.bars.turn[i], 1);
    }
    for (int i = 0; i < 3; ++i) mbar_init(&sh.bars.based[i], 2);
    fence_mbar_init();
    sh.abort = 0;
    sh.maxpages = 0;
    sh.minpages = p.n_prefix;
  }
  // ---- packed pages: what a loading warp takes.  The two schedulers that issue products get
  // a Key and a Value warp each, the others two Key warps and one more (measured against
  // three other orders at 128 x 32768: 184.6 us a call, the others 187.6 to 197.3).
  const int tiles = (p.n_prefix + F::kPages - 1) / F::kPages;
  const int t0 = (int)((long)tiles * split / p.splits), t1 = (int)((long)tiles * (split + 1) / p.splits);
  const int role = wid >= kLoadWarp ? (int)((0x8930547621ull >> (4 * (wid - kLoadWarp))) & 15) : 12;
  // page of the tile; 0, 1: halves of the Keys, 2: Values, 3: fetch, 4: not a loading warp
  const int lg = role % 3, part = role / 3;
  const bool values = part == 2;
  constexpr int kRaw = F::kRaw;
  const uint32_t key_bytes = F::kPacked ? 512 * F::W + 4 * F::W * p.n_hi + 512 + p.n_hi : 0;
  // item i of a slot: a page's Keys (i < 3) or Values
  auto raw_at = [&](int i, int slot) {
    return raws + (i < 3 ? (i * kRaw + slot) * F::kRawK : 3 * kRaw * F::kRawK + ((i - 3) * kRaw + slot) * F::kRawV);
  };
  uint32_t in_flight = 0;    // of this lane's item: bit: the slot awaits a copy
  int ids = -1, ids_at = 0;  // lane l: the id of this lane's page of tile ids_at + l / 3
  // The fetching warp: lane i < 6 requests item i of a tile, or arrives for it without one.
  auto fetch = [&](int tile) {
    if (tile == 0 || tile - ids_at >= 10) {
      ids_at = tile;
      const int t = t0 + tile + lane / 3, page = t * F::kPages + lane % 3;
      ids = lane < 30 && t < t1 && page < p.n_prefix ? p.table[page] : -1;
    }
    const int id = __shfl_sync(0xFFFFFFFFu, ids, 3 * (tile - ids_at) + lane % 3), slot = tile % kRaw;
    const bool in = id >= 0 && id < p.pool_pages;
    if (lane < 3) sh.got[tile % kFlags][lane] = in;
    __syncwarp();
    if (lane < 6) {
      const uint32_t bar = smem_u32(&sh.bars.raw[lane][slot]);
      if (in) {
        const uint32_t bytes = lane < 3 ? key_bytes : F::kRawV;
        mbar_arrive_expect_tx_s(bar, bytes);
        bulk_g2s_s(raw_at(lane, slot), p.pool + ((size_t)id * p.Hkv + kvh) * p.blob + (lane < 3 ? 0 : key_bytes), bytes, bar);
        in_flight |= 1u << slot;
      } else {
        mbar_arrive_s(bar);
        in_flight &= ~(1u << slot);
      }
    }
    __syncwarp();
  };
  if (F::kPacked && part == 3) {  // the first copies, before anything else
    if (lane < 6) {
      for (int k = 0; k < kRaw; ++k) {
        mbar_init(&sh.bars.raw[lane][k], 1);
        mbar_init(&sh.bars.freed[lane][k], lane < 3 ? 2 : 1);
      }
      fence_mbar_init();
    }
    __syncwarp();
    for (int tile = 0; tile < min(t1 - t0, kRaw); ++tile) fetch(tile);
  }
  // ---- the rows: what each sees of the prefix, its partials' place
  const int in_unit = unit * kRows + (both ? tid : (tid & 127));  // row of the kv head
  const bool real = tid < kRows && in_unit < R;
  int my_pages = p.n_prefix, b = 0;
  size_t part_row = 0;
  if (real) {
    b = in_unit / p.g;
    part_row = (size_t)b * p.Hq + (size_t)kvh * p.g + (in_unit - b * p.g);
    if (p.prefix_pages != nullptr) my_pages = p.prefix_pages[b];
  }
  if (tid < kRows) sh.row[tid] = real ? (int)part_row : -1;
  if (F::kPacked && tid < kStages * F::kPages * 4) {  // the row of ones behind each slab's middles
    const uint32_t at = vst + (tid / (4 * F::kPages)) * F::kVBytes + (tid / 4 % F::kPages) * F::kSlab + (kD + 4) * 64;
    sts128(at + 16 * (tid & 3), make_uint4(0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u));
    fence_async_shared();
  }
  if (wid == kMmaWarp) tmem_alloc(smem_u32(&sh.tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int page_end = p.n_prefix, full_pages = p.n_prefix;  // pages that some row, every row, of the block sees
  if (p.prefix_pages != nullptr) {
    if (real) {
      if (my_pages < 0 || my_pages > p.n_prefix) {
        set_status(p.d_status, KITTY_ST_BAD_LEN);
        my_pages = 0;
      }
      atomicMax(&sh.maxpages, my_pages);
      atomicMin(&sh.minpages, my_pages);
    }
    __syncthreads();
    page_end = __shfl_sync(0xFFFFFFFFu, sh.maxpages, 0);
    full_pages = __shfl_sync(0xFFFFFFFFu, sh.minpages, 0);
  }
  const int n = max(0, min(t1, (page_end + F::kPages - 1) / F::kPages) - t0);  // tiles of this block
  const int steps = both ? 2 * n : n;  // step s: lane s & 1, tile s / 2 or s
  const int slot0 = both ? split : 2 * split + (tid >> 7);
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sh.tmem, 0);
  int loads = 0;  // 16-bit pages: tiles that this warp has requested
  auto s_col = [&](int a) { return tmem + (uint32_t)(a * F::kS); };
  auto all_valid = [&](int tile) {
    constexpr uint32_t mask = F::kPages == 4 ? 0x01010101u : 0x00010101u;
    return (*reinterpret_cast<const volatile uint32_t*>(sh.valid[tile % kFlags]) & mask) == mask;
  };
  auto o_col = [&](int a) { return tmem + (uint32_t)(2 * F::kS + a * F::kO); };

  // five warpgroups at 96 registers: the two of the softmax take 136, the others 64
  if (F::kPacked) {
    if (wid < kSoftmaxWarps) asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
  }
  if (wid < kSoftmaxWarps) {
    // =========================================================== softmax
    const int a = wid >> 2;
    const uint32_t lanes = (uint32_t)(32 * (wid & 3)) << 16;
    const uint32_t S = s_col(a) + lanes, O = o_col(a) + lanes;
    const float sc = fabsf(p.sm_log2);
    if (n > 0) {  // the lane's queries: 16 threads a row, 8 rows at a time
      const int c = lane & 15, at = (c >> 3) * kQHalf;
      uint4 v[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int x = sh.row[32 * wid + 2 * k + (lane >> 4)];
        v[k] = x >= 0 ? *reinterpret_cast<const uint4*>(p.q + (size_t)x * kD + 8 * c) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int rr = 32 * wid + 2 * k + (lane >> 4);
        sts128(base + at + rr * 128 + (((c & 7) ^ (rr & 7)) << 4), query16<F>(v[k], p.in_dtype, p.sm_log2 < 0.f));
      }
      fence_async_shared();
      mbar_arrive_s(smem_u32(&sh.bars.qready[wid >> 2]));
    }
    float m = kFloor;
    float2 sum = make_float2(0.f, 0.f);  // 16-bit pages: two partial sums of p
    bool any = false;                    // this row has seen a page
    bool ok = true;
    int i = 0;
    for (int s = a; s < steps; s += 2, ++i) {
      if (!wait_phase(&sh.bars.sfull[a], i & 1, p.wait_polls, abort)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const int tile = both ? s >> 1 : s, page0 = (t0 + tile) * F::kPages;
      // the tile's scores, all at once, in registers
      uint32_t x[F::kPages][32], bias[F::kPages];
#pragma unroll
      for (int g = 0; g < F::kPages; ++g) {
        if (F::kPacked) tmem_ld1(S + F::kTok + g, bias[g]);
        else bias[g] = 0;
        tmem_ld32(S + 32 * g, x[g]);
      }
      // the pages that this row sees; the rows that do not, for the products' masks
      const bool full = page0 + F::kPages <= full_pages && all_valid(tile);
      bool on[F::kPages];
#pragma unroll
      for (int g = 0; g < F::kPages; ++g) on[g] = true;
      if (!full) {
#pragma unroll
        for (int g = 0; g < F::kPages; ++g) {
          on[g] = page0 + g < my_pages && sh.valid[tile % kFlags][g] != 0;
          const uint32_t off = __ballot_sync(0xFFFFFFFFu, !on[g]);
          if (lane == 0) sh.off[a][g][wid & 3] = off;
          any = any || on[g];
        }
      } else {
        any = true;
      }
#pragma unroll
      for (int g = 0; g < F::kPages; ++g) {
        tmem_wait_ld(x[g]);
        if (F::kPacked) pin(bias[g]);
      }
      float mx = kFloor;  // this row's maximum, scaled
#pragma unroll
      for (int g = 0; g < F::kPages; ++g) {
        float pm = fmaxf(__uint_as_float(x[g][0]), __uint_as_float(x[g][1]));
#pragma unroll
        for (int k = 2; k < 32; k += 2) pm = fmaxf(fmaxf(pm, __uint_as_float(x[g][k])), __uint_as_float(x[g][k + 1]));
        pm = (pm + __uint_as_float(bias[g])) * sc;
        mx = fmaxf(mx, full || on[g] ? pm : kFloor);
      }
      if (i == 0) {
        m = mx + kMargin;
      } else if (__any_sync(0xFFFFFFFFu, mx > m + kSlack)) {
        // each row by its own maximum: what it gives does not depend on its neighbours'
        const float nm = mx > m + kSlack ? mx + kMargin : m, f = nm > m ? ex2a(m - nm) : 1.f;
#pragma unroll 1
        for (int c = 0; c < F::kO; c += 16) {
          uint32_t y[16];
          tmem_ld16(O + c, y);
          tmem_wait_ld(y);
#pragma unroll
          for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * f);
          tmem_st16(O + c, y);
        }
        sum = make_float2(sum.x * f, sum.y * f);
        m = nm;
      }
      uint64_t acc = f2pack(sum.x, sum.y);
#pragma unroll
      for (int g = 0; g < F::kPages; ++g) {
        const float shift = fmaf(__uint_as_float(bias[g]), sc, -m);
        const uint64_t sc2 = f2pack(sc, sc), shift2 = f2pack(shift, shift);
        uint32_t P[16], rest[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          uint64_t e2;
          asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(e2) : "l"(pair64(x[g][2 * k], x[g][2 * k + 1])), "l"(sc2), "l"(shift2));
          float e0, e1;
          f2unpack(e2, e0, e1);
          e0 = ex2a(e0);
          e1 = ex2a(e1);
          if (!full) {  // what a row does not see may hold anything
            e0 = on[g] ? e0 : 0.f;
            e1 = on[g] ? e1 : 0.f;
          }
          if (!F::kPacked) asm("add.rn.f32x2 %0, %0, %1;" : "+l"(acc) : "l"(f2pack(e0, e1)));
          P[k] = pack_probs<F>(e0, e1, rest[k]);
        }
        // over the page's own scores, which this thread has taken
        tmem_st16(S + 32 * g, P);
        if (F::kPair) tmem_st16(S + 32 * g + 16, rest);
      }
      f2unpack(acc, sum.x, sum.y);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive_s(smem_u32(&sh.bars.pready[a]));
    }
    // ---- this lane's partials: 32 channels at a time through the lane's own queries' memory
    // (its products have read them), so that a row's 128 bytes are written together
    if (ok && i > 0) ok = wait_phase(&sh.bars.ofull[a], 0, p.wait_polls, abort);
    float total = sum.x + sum.y;
    if (ok && i > 0) {
      tc_fence_after();
      if (F::kPacked) {
        uint32_t t;
        tmem_ld1(O + kD + 4, t);
        tmem_wait_ld(t);
        total = __uint_as_float(t);
      }
      const uint32_t buf = base + 32 * wid * 128;  // 4096 bytes: 32 rows of 128, swizzled
      const int sub = lane >> 3, c4 = lane & 7;
#pragma unroll 1
      for (int c = 0; c < kD; c += 32) {
        uint32_t x[32], vmin = 0;
        if (F::kPacked) tmem_ld1(O + kD + c / 32, vmin);
        tmem_ld32(O + c, x);
        tmem_wait_ld(x);
        if (F::kPacked) pin(vmin);
        const float add = __uint_as_float(vmin);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint4 v;
          v.x = __float_as_uint(__uint_as_float(x[4 * k]) + add);
          v.y = __float_as_uint(__uint_as_float(x[4 * k + 1]) + add);
          v.z = __float_as_uint(__uint_as_float(x[4 * k + 2]) + add);
          v.w = __float_as_uint(__uint_as_float(x[4 * k + 3]) + add);
          sts128(buf + lane * 128 + ((k ^ (lane & 7)) << 4), v);
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int rr = 4 * k + sub, x = sh.row[32 * wid + rr];
          const uint4 v = lds128(buf + rr * 128 + ((c4 ^ (rr & 7)) << 4));
          if (x >= 0)
            *reinterpret_cast<uint4*>(p.ws + ((size_t)x * p.slots + slot0) * kPartialFloats + 4 + c + 4 * c4) = v;
        }
        __syncwarp();
      }
      tc_fence_before();
    }
    if (real)
      *reinterpret_cast<float2*>(p.ws + (part_row * p.slots + slot0) * kPartialFloats) = make_float2(ok && any ? m : -INFINITY, total);
    if (!ok && lane == 0) set_status(p.d_status, KITTY_ST_TIMEOUT);
  } else if (wid < kLoadWarp) {
    // =========================================================== products
    // One warp a lane, so that one lane's waits do not hold up the other's products; the whole
    // warp runs this and one elected lane issues, so that descriptors stay in uniform
    // registers.  The lanes take turns, a step's products in one piece: one lane's scores are
    // then done half a period before the other's, and its softmax runs beside the other's
    // products (without turns the two fell into phase, products and softmax by turns: 5000
    // cycles a tile).
    constexpr uint32_t qk = mma_desc(F::kBf16, false, F::kS), pv = mma_desc(F::kBf16, !F::kPacked, F::kO);
    const int a = wid - kMmaWarp, both_shift = both ? 1 : 0;
    const uint64_t qdesc = smem_desc(base + a * (128 * 128), 16, 1024, kSwizzle128), kdesc = smem_desc(kst, 16, 1024, kSwizzle128);
    const uint64_t vdesc = F::kPacked ? smem_desc(vst, 16, 512, kSwizzle64) : smem_desc(vst, F::kKHalf, 1024, kSwizzle128);
    const uint32_t scol = s_col(a), ocol = o_col(a);
    bool started = false, ok = true;
    // S of step s, by the elected lane; then the operands of its tile's Keys, and of the
    // Values of the step before on this lane, are free
    auto scores = [&](int s) {
      const int st = (s >> both_shift) % kStages;
      const uint64_t kb = kdesc + st * (F::kKBytes / 16);
#pragma unroll
      for (int k = 0; k < kD / 16; ++k) {
        // the other lane's turn, early enough that its products follow without a gap
        if (k == kD / 32) mbar_arrive_s(smem_u32(&sh.bars.turn[1 - a]));
        mma_ss(scol, qdesc + (k >> 2) * (kQHalf / 16) + 2 * (k & 3), kb + (k >> 2) * (F::kKHalf / 16) + 2 * (k & 3), qk, k > 0);
      }
      mma_commit(smem_u32(&sh.bars.sfull[a]));
      mma_commit(smem_u32(&sh.bars.kempty[st]));
      if (s >= 2) mma_commit(smem_u32(&sh.bars.vempty[((s - 2) >> both_shift) % kStages]));
    };
    if (a < steps) {
      const int tile = a >> both_shift;  // lane 1 after lane 0
      ok = wait_lanes(lane < 2 + a, lane == 0 ? smem_u32(&sh.bars.qready[a]) : lane == 1 ? smem_u32(&sh.bars.kfull[tile]) : smem_u32(&sh.bars.turn[a]),
                      0, p.wait_polls, abort);
      tc_fence_after();
      if (ok && elect_one()) scores(a);
      __syncwarp();
    }
    for (int s = a; ok && s < steps; s += 2) {
      const int tile = s >> both_shift, st = tile % kStages, page0 = (t0 + tile) * F::kPages;
      const bool more = s + 2 < steps;
      // this step's probabilities and Values, and the turn (the other lane's arrivals: one with
      // each of its scores, one with each end without)
      const uint32_t bar = smem_u32(lane == 0 ? &sh.bars.pready[a] : lane == 1 ? &sh.bars.vfull[st] : &sh.bars.turn[a]);
      const int phase = lane == 0 ? s >> 1 : lane == 1 ? tile / kStages : (s + a) >> 1;
      ok = wait_lanes(lane < (steps > 1 ? 3 : 2), bar, phase & 1, p.wait_polls, abort);
      if (!ok) break;
      tc_fence_after();
      const uint64_t vb = vdesc + st * (F::kVBytes / 16);
      if (page0 + F::kPages <= full_pages && all_valid(tile)) {
        // every row of the block sees every page of the tile
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 2 * F::kPages; ++k) {
            const uint64_t vk = vb + (F::kPacked ? ((k >> 1) * F::kSlab + 32 * (k & 1)) / 16 : 16 * k * 128 / 16);
            mma_ts(ocol, scol + 16 * k - 8 * (k & 1), vk, pv, started || k > 0);
            if (F::kPair) mma_ts(ocol, scol + 16 * k - 8 * (k & 1) + 16, vk, pv, true);
          }
        }
        started = true;
      } else {
#pragma unroll 1
        for (int g = 0; g < F::kPages; ++g) {
          const uint4 o4 = *reinterpret_cast<const uint4*>(sh.off[a][g]);
          if (__any_sync(0xFFFFFFFFu, (o4.x & o4.y & o4.z & o4.w) == 0xFFFFFFFFu)) continue;  // no row sees it, or no page
          const uint32_t off[4] = {o4.x, o4.y, o4.z, o4.w};
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t pa = scol + 32 * g + 8 * k;
              const uint64_t vk = vb + (F::kPacked ? (g * F::kSlab + 32 * k) / 16 : (32 * g + 16 * k) * 128 / 16);
              mma_ts_masked(ocol, pa, vk, pv, started || k > 0, off);
              if (F::kPair) mma_ts_masked(ocol, pa + 16, vk, pv, true, off);
            }
          }
          __syncwarp();
          started = true;
        }
      }
      __syncwarp();
      if (more) {
        const int next = (s + 2) >> both_shift;
        ok = wait_phase(&sh.bars.kfull[next % kStages], (next / kStages) & 1, p.wait_polls, abort);
        if (!ok) break;
        tc_fence_after();
      }
      if (elect_one()) {
        if (more) {
          scores(s + 2);
        } else {
          mma_commit(smem_u32(&sh.bars.ofull[a]));
          mbar_arrive_s(smem_u32(&sh.bars.turn[1 - a]));
        }
      }
      __syncwarp();
    }
    if (!ok && lane == 0) set_status(p.d_status, KITTY_ST_TIMEOUT);
    __syncwarp();
  } else if constexpr (F::kPacked) {
    // =========================================================== packed pages
    bool ok = true;
    if (part == 3) {
      int tile = min(t1 - t0, kRaw);
      for (; tile < n; ++tile) {  // a slot is free when its item's readers are through
        const int slot = tile % kRaw, turn = tile / kRaw - 1;
        ok = wait_lanes(lane < 6, smem_u32(&sh.bars.freed[lane < 6 ? lane : 0][slot]), turn & 1, p.wait_polls, abort);
        if (!ok) break;
        fetch(tile);
      }
      // copies that nobody waited for: after a wait that ran out, or past the last seen page
      if (lane < 6)
        for (int k = 0; k < kRaw; ++k)
          if ((in_flight >> k) & 1u) {
            const int last = (tile - 1 - k) / kRaw;  // the slot's latest use
            mbar_wait_bounded(&sh.bars.raw[lane][k], last & 1, kPrefixWaitPolls);
          }
      __syncwarp();
    } else {
      uint32_t based_phase = 0;
      for (int tile = 0; tile < n; ++tile) {
        const int slot = tile % kRaw, st = tile % kStages, item = values ? 3 + lg : lg;
        const bool seen = (t0 + tile) * F::kPages + lg < page_end;
        // the staged page, and the stage's last readers
        const uint32_t empty = smem_u32(values ? &sh.bars.vempty[st] : &sh.bars.kempty[st]);
        ok = wait_lanes(lane < 2, lane == 0 ? smem_u32(&sh.bars.raw[item][slot]) : empty,
                        lane == 0 ? (tile / kRaw) & 1 : ((tile / kStages) & 1) ^ 1, p.wait_polls, abort);
        if (!ok) break;
        const bool got = sh.got[tile % kFlags][lg] != 0, in = got && seen;
        if (!got && seen && part == 0 && lane == 0) set_status(p.d_status, KITTY_ST_BAD_PAGE);
        auto based = [&]() {
          __syncwarp();
          if (lane == 0) mbar_arrive_s(smem_u32(&sh.bars.based[lg]));
          return wait_phase(&sh.bars.based[lg], based_phase, p.wait_polls, abort);
        };
        if (in) {
          const uint32_t raw = raw_at(item, slot);
          if (values) {
            put_values<F>(raw, vst + st * F::kVBytes + lg * F::kSlab, p.d_status);
          } else {
            ok = put_keys<F>(raw, kst + st * F::kKBytes, lg, part, p.n_hi, p.d_status, based);
            based_phase ^= 1u;
          }
          if (!ok) break;
        }
        if (part == 0 && lane == 0) sh.valid[tile % kFlags][lg] = in;
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_s(smem_u32(values ? &sh.bars.vfull[st] : &sh.bars.kfull[st]));
          mbar_arrive_s(smem_u32(&sh.bars.freed[item][slot]));
        }
      }
    }
    if (!ok && lane == 0) set_status(p.d_status, KITTY_ST_TIMEOUT);
    __syncwarp();
  } else {
    // =========================================================== 16-bit pages
    const bool values = wid == kLoadWarp + 1;
    uint64_t *full = values ? sh.bars.vfull : sh.bars.kfull, *empty = values ? sh.bars.vempty : sh.bars.kempty;
    const uint32_t st0 = values ? vst : kst;
    bool ok = true;
    int tile = 0;  // loads issued
    for (; tile < n; ++tile) {
      const int st = tile % kStages;
      ok = wait_phase(&empty[st], ((tile / kStages) & 1) ^ 1, p.wait_polls, abort);
      if (!ok) break;
      const int page = (t0 + tile) * F::kPages + lane;
      const int id = lane < F::kPages && page < page_end ? p.table[page] : -1;
      const bool in = id >= 0 && id < p.pool_pages;
      const int count = __popc(__ballot_sync(0xFFFFFFFFu, in));
      const uint32_t bar = smem_u32(&full[st]);
      if (lane < F::kPages) {
        if (!values) sh.valid[tile % kFlags][lane] = in;
        if (!in && page < page_end) set_status(p.d_status, KITTY_ST_BAD_PAGE);
      }
      __syncwarp();  // the flags, before the arrival that publishes them
      if (lane == 0) mbar_arrive_expect_tx_s(bar, (uint32_t)(count * kPage * kD * 2));
      __syncwarp();
      if (in) {
        const int y = (id * p.Hkv + kvh) * 2 * kPage + (values ? kPage : 0);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          tma_load_2d(st0 + st * F::kKBytes + h * F::kKHalf + lane * kPage * 128, &map, 64 * h, y, bar);
      }
    }
    if (!ok && lane == 0) set_status(p.d_status, KITTY_ST_TIMEOUT);
    __syncwarp();
    loads = tile;
  }
  __syncthreads();
  // after a wait that ran out: nothing may be in flight when the block's memory is given back
  if (*abort != 0 && elect_one()) {
    if (wid >= kMmaWarp && wid < kLoadWarp) {
      mma_commit(smem_u32(&sh.bars.drain[wid - kMmaWarp]));
      mbar_wait_bounded(&sh.bars.drain[wid - kMmaWarp], 0, kPrefixWaitPolls);
    } else if (!F::kPacked && wid >= kLoadWarp) {
      for (int k = max(0, loads - kStages); k < loads; ++k)
        mbar_wait_bounded(wid == kLoadWarp ? &sh.bars.kfull[k % kStages] : &sh.bars.vfull[k % kStages],
                          (k / kStages) & 1, kPrefixWaitPolls);
    }
  }
  if (*abort != 0) __syncthreads();  // both lanes' products have ended
  if (wid == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Splits of the prefix.  A block has an SM to itself; the SMs that no block takes, or that get
// free, attend the sequences' own pages meanwhile.  So more splits shorten the longest block,
// but each costs SM time for its start and end and a partial a row, written and read.  In us,
// measured on GB300 by forcing the splits of five shapes (the model's choice was the fastest
// or within 2% of it at all five; one block on every SM, the choice without the own pages'
// share: 64 x 8192 tokens 34.3 against 30.1 us, on 16-bit pages 41.3 against 31.9 us,
// 128 x 32768 177 against 165 us):
constexpr double kTileUs = 1.8;    // a tile of both lanes (1.7 packed, 2 on 16-bit pages)
constexpr double kPathTiles = 7;   // start and end of a block, in tiles, on the critical path ..
constexpr double kBlockTiles = 8.5;  // .. and of its SM's time
PrefixPlan plan_for(int Hkv, int rows, int tiles, int sms, double own_us) {
  PrefixPlan pl = {Hkv * ((rows + kRows - 1) / kRows), 1, 1};
  const double tile = rows > 128 ? 1.0 : 0.5;  // lanes that share their rows halve a block's tiles
  const double per_split = (double)Hkv * rows * 1056.0 / 6.0e6;
  double best = 1e30;
  for (int s = 1; s <= std::min(tiles, 64); ++s) {
    const int blocks = pl.units * s, waves = (blocks + sms - 1) / sms;
    const double per = tile * ((tiles + s - 1) / s);
    const double path = waves * (per + kPathTiles) * kTileUs;
    const double all = (blocks * (per + kBlockTiles) * kTileUs + own_us) / sms;
    const double cost = std::max(path, all) + s * per_split;
    if (cost < best - 1e-9) {
      best = cost;
      pl.splits = s;
    }
  }
  pl.slots = rows > 128 ? pl.splits : 2 * pl.splits;
  return pl;
}

// SM time of the own pages' kernel, us: per (sequence, kv head) a start and its pages (from
// the same measurements).  Pages by the plan's hint; without one, up to 4: a block table's
// width says little of how much of it is filled, and a guess too high leaves the prefix on too
// few SMs (all of it), one too low costs about 1 us a needless split.
double own_us_of(const kitty_cfg* cfg, bool packed, int B, int max_pages) {
  const double pages = cfg->decode_total_pages > 0 ? (double)cfg->decode_total_pages / B : std::min(4.0, 0.5 * max_pages);
  const int g = cfg->num_q_heads / cfg->num_kv_heads;
  return (double)B * cfg->num_kv_heads * ((g + 7) / 8) * (packed ? 1.0 + 0.16 * pages : 2.5 + 0.5 * pages);
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The 16-bit pool as rows of 128 channels; boxes of 32 rows by 64 channels, swizzled.
bool pool_map(CUtensorMap* map, const void* pool, uint64_t rows) {
  static std::atomic<EncodeTiled> encode{nullptr};
  EncodeTiled f = encode.load();
  if (f == nullptr) {
    void* sym = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &sym, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      return false;
    f = reinterpret_cast<EncodeTiled>(sym);
    encode.store(f);
  }
  const cuuint64_t dims[2] = {kD, rows}, strides[1] = {kD * 2};
  const cuuint32_t box[2] = {64, kPage}, ones[2] = {1, 1};
  return f(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(pool), dims, strides, box, ones,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class F>
int launch(const PrefixArgs& a, const PrefixPlan& pl, const CUtensorMap& map, cudaStream_t s) {
  static_assert(smem_of<F>() <= 227 * 1024 - 1024, "fits beside the static part");
  static_assert(2 * (F::kS + F::kO) <= 512, "fits tensor memory");
  static std::atomic<uint64_t> opted_in{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KITTY_ERR_CUDA;
  const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t(1) << dev) : 0;
  if (bit == 0 || (opted_in.load() & bit) == 0) {
    if (cudaFuncSetAttribute(prefix_kernel<F>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_of<F>()) != cudaSuccess)
      return KITTY_ERR_CUDA;
    opted_in.fetch_or(bit);
  }
  const cudaError_t e = launch_behind(prefix_kernel<F>, dim3((unsigned)pl.units, (unsigned)pl.splits),
                                      threads_of<F>(), (size_t)smem_of<F>(), s, false, a, map);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? KITTY_OK : KITTY_ERR_CUDA;
}

}  // namespace

PrefixPlan prefix_plan(const kitty_cfg* cfg, bool packed, int B, int n_prefix, int max_pages) {
  if (n_prefix <= 0 || B <= 0) return {0, 0, 0};
  const int pages = packed ? PackedFmt<2, 2>::kPages : PlainFmt<true>::kPages;
  return plan_for(cfg->num_kv_heads, B * (cfg->num_q_heads / cfg->num_kv_heads), (n_prefix + pages - 1) / pages, sm_count(),
                  own_us_of(cfg, packed, B, max_pages));
}

int prefix_launch(const kitty_cfg* cfg, bool packed, const PrefixArgs& args, const PrefixPlan& pl, cudaStream_t s) {
  CUtensorMap map = {};
  if (packed) {
    if (cfg->lo_bit == 2) return launch<PackedFmt<2, 2>>(args, pl, map, s);
    return v_bits(cfg) == 2 ? launch<PackedFmt<4, 2>>(args, pl, map, s) : launch<PackedFmt<4, 4>>(args, pl, map, s);
  }
  const uint64_t rows = (uint64_t)args.pool_pages * args.Hkv * 2 * kPage;
  if (rows == 0) return KITTY_ERR_INVALID_ARG;
  if (rows > 0x7FFFFFFFull) return KITTY_ERR_UNSUPPORTED;  // a row's coordinate is an int32
  if (!pool_map(&map, args.pool, rows)) return KITTY_ERR_CUDA;
  return cfg->in_dtype == KITTY_BF16 ? launch<PlainFmt<true>>(args, pl, map, s) : launch<PlainFmt<false>>(args, pl, map, s);
}

}  // namespace kitty
