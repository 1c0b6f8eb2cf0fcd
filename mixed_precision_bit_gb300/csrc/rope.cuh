// Per-head RMS norm and position rotation of one 128-channel head row held by 16
// lanes, eight channels a lane: shared by the pass over queries and keys and by
// the appends that rotate on the way into a cache.
//
//   norm    n = x * rsqrt(sum x^2 / 128 + eps) * w                 (w given)
//   rotate  (a, b) -> A (a cos t - b sin t, b cos t + a sin t),   t = position * f_j,
//           over the pairs (j, j + rot/2) or (2j, 2j + 1) of the first rot channels
//
// Everything is held in fp32 and rounded once, to the 16-bit output.
//
// Angles.  A position times a frequency in fp32 is off by up to half a radian's
// 2^-24th of the product, 0.004 at position 65536: as much as a bf16 step of the
// result.  The table holds each frequency as a fraction of a turn in 64-bit fixed
// point instead (f / 2 pi * 2^64, mod 2^64): position * entry mod 2^64 is the angle's
// exact fraction of a turn, one integer product, for any int32 position (negative
// ones too); its top 32 bits as a signed number are the angle in half turns times
// 2^31.
#pragma once

#include "kitty_common.cuh"

namespace kitty {

constexpr int kRowLanes = 16;             // lanes of one head row, eight channels each

// A rotation as the kernels take it.
struct RopeParams {
  const uint64_t* turns;     // [rot / 2]
  const uint16_t* q_weight;  // [128] or null
  const uint16_t* k_weight;
  float amplitude, eps;
  int rot, interleaved;
};

// (cos, sin) * amplitude of every pair at one position into shared memory, by the
// first rot / 2 threads of the block; the caller synchronizes.
__device__ __forceinline__ void rope_angles(const RopeParams& p, int64_t position, float2* cs) {
  if (threadIdx.x < p.rot / 2) {
    const uint64_t t = (uint64_t)position * p.turns[threadIdx.x];
    float s, c;
    sincospif((float)(int32_t)(uint32_t)(t >> 32) * 0x1p-31f, &s, &c);
    cs[threadIdx.x] = make_float2(c * p.amplitude, s * p.amplitude);
  }
}

// What a lane of a row holds, so that both channels of a pair are its own and no rotation
// needs a shuffle: four channels from c0 and four from c1.
//   half layout   lanes below rot / 8: c0 = 4 lane, c1 = c0 + rot / 2 (pair i: c0 + i, c1 + i)
//   interleaved   c0 = 8 lane, c1 = c0 + 4 (pairs c0, c0 + 1; c0 + 2, ..)
// and the channels past rot, eight a lane, in the other lanes.  Rot is a multiple of 16,
// so every four are 8-byte aligned.  In registers the first and second channels of the pairs
// are two words each (by byte permutations that the layout picks: a, b = first words of both
// fours, then their second words), so the arithmetic takes two pairs at a time.  c, s: the
// coefficients of pairs (0, 1), (2, 3); interleaved: of pairs (0, 2), (1, 3).
struct RopeLane {
  uint64_t c[2], s[2], ns[2];  // ns = -s
  int c0, c1;
  uint32_t first, second;  // the permutations
  bool on, interleaved;  // on: this lane's channels rotate
};

// Where a lane's channels are (nothing of it depends on the position).
__device__ __forceinline__ RopeLane rope_lane(const RopeParams& p) {
  RopeLane L;
  const int lane = threadIdx.x & (kRowLanes - 1), h = p.rot / 2;
  L.interleaved = p.interleaved != 0;
  L.on = L.interleaved ? 8 * lane < p.rot : 4 * lane < h;
  if (L.interleaved) L.c0 = 8 * lane;
  else L.c0 = L.on ? 4 * lane : p.rot + 8 * (lane - h / 4);
  L.c1 = !L.interleaved && L.on ? L.c0 + h : L.c0 + 4;
  L.first = L.interleaved ? 0x5410u : 0x3210u;
  L.second = L.interleaved ? 0x7632u : 0x7654u;
  return L;
}

// Its pairs' coefficients, from the block's table.
__device__ __forceinline__ void rope_coefficients(RopeLane& L, const float2* cs) {
  const float2* at = cs + (L.interleaved ? L.c0 / 2 : L.c0);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = L.on ? at[L.interleaved ? i : 2 * i] : make_float2(1.f, 0.f);
    const float2 b = L.on ? at[L.interleaved ? i + 2 : 2 * i + 1] : make_float2(1.f, 0.f);
    L.c[i] = f2pack(a.x, b.x);
    L.s[i] = f2pack(a.y, b.y);
    L.ns[i] = f2pack(-a.y, -b.y);
  }
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Both fours' words to (first, second) channels of the pairs, and back.
__device__ __forceinline__ uint4 rope_permute(uint4 x, const RopeLane& L) {
  return make_uint4(__byte_perm(x.x, x.z, L.first), __byte_perm(x.y, x.w, L.first),
                    __byte_perm(x.x, x.z, L.second), __byte_perm(x.y, x.w, L.second));
}

template <int DT>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
  if (DT == KITTY_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(bits_h2(w));
}
template <int DT>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if (DT == KITTY_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  return h2_bits(__floats2half2_rn(a, b));
}

// Eight 16-bit values of a lane: the four from c0 in x, y, the four from c1 in z, w.
__device__ __forceinline__ uint4 rope_get(const uint16_t* row, const RopeLane& L) {
  const uint2 a = *reinterpret_cast<const uint2*>(row + L.c0), b = *reinterpret_cast<const uint2*>(row + L.c1);
  return make_uint4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void rope_put(uint16_t* row, const RopeLane& L, uint4 v) {
  *reinterpret_cast<uint2*>(row + L.c0) = make_uint2(v.x, v.y);
  *reinterpret_cast<uint2*>(row + L.c1) = make_uint2(v.z, v.w);
}
// Weights of the lane's channels (any alignment; zeros without a weight).
__device__ __forceinline__ uint4 rope_weights(const uint16_t* w, const RopeLane& L) {
  if (w == nullptr) return make_uint4(0, 0, 0, 0);
  if ((reinterpret_cast<uintptr_t>(w) & 7u) == 0) return rope_get(w, L);
  auto two = [&](int c) { return (uint32_t)w[c] | ((uint32_t)w[c + 1] << 16); };
  return make_uint4(two(L.c0), two(L.c0 + 2), two(L.c1), two(L.c1 + 2));
}

// One row: x = this lane's eight channels in, normed and rotated out (weight: permuted).  Called
// by whole warps; rows are 16 lanes, so a warp takes two.  any: a row of the warp may be normed.
template <int DT>
__device__ __forceinline__ uint4 rope_row(uint4 x, const RopeLane& L, uint4 weight, bool any, bool norm, float eps) {
  const uint4 y = rope_permute(x, L);
  const uint32_t in[4] = {y.x, y.y, y.z, y.w}, w[4] = {weight.x, weight.y, weight.z, weight.w};
  uint64_t f[4];  // first channels of two pairs, of two more; second channels
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = unpack16<DT>(in[i]);
    f[i] = f2pack(v.x, v.y);
  }
  if (any) {
    uint64_t s2 = mul2(f[0], f[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) s2 = fma2(f[i], f[i], s2);
    float ss, s1;
    f2unpack(s2, ss, s1);
    ss += s1;
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
    const float r = rsqrtf(fmaf(ss, 1.0f / kD, eps));
    if (norm) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = unpack16<DT>(w[i]);
        f[i] = mul2(mul2(f[i], f2pack(r, r)), f2pack(v.x, v.y));
      }
    }
  }
  if (L.on) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t a = f[i], b = f[2 + i];
      f[i] = fma2(a, L.c[i], mul2(b, L.ns[i]));
      f[2 + i] = fma2(b, L.c[i], mul2(a, L.s[i]));
    }
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2unpack(f[i], lo, hi);
    o[i] = pack16<DT>(lo, hi);
  }
  return rope_permute(make_uint4(o[0], o[1], o[2], o[3]), L);  // its own inverse
}

// The rows of one token: H1 query rows and H2 key rows through rope_row, H2 value
// rows copied (v may be null).  Head h's row is at + 128 h in the inputs and the
// query output, at + h * stride in the key and value outputs.
struct TokenRows {
  const uint16_t *q, *k, *v;
  uint16_t *qo, *ko, *vo;
  size_t kv_stride;
  int H1, H2;
  __device__ int rows() const { return H1 + (v != nullptr ? 2 : 1) * H2; }
  __device__ const uint16_t* in(int i) const {
    const uint16_t* base = i < H1 ? q : i < H1 + H2 ? k - (ptrdiff_t)H1 * kD : v - (ptrdiff_t)(H1 + H2) * kD;
    return base + (ptrdiff_t)i * kD;
  }
  __device__ uint16_t* out(int i) const {
    if (i < H1) return qo + (size_t)i * kD;
    return i < H1 + H2 ? ko + (size_t)(i - H1) * kv_stride : vo + (size_t)(i - H1 - H2) * kv_stride;
  }
};

// A block of THREADS takes THREADS / 16 rows at a time and loads AHEAD rows a 16-lane group
// before it uses the first of them.  First round of a token's rows (nothing depends on its
// position yet).
template <int THREADS, int AHEAD>
__device__ __forceinline__ void rope_load(const TokenRows& t, const RopeLane& L, int r0, uint4 (&x)[AHEAD]) {
  const int n = t.rows();
#pragma unroll
  for (int u = 0; u < AHEAD; ++u) {
    const int i = r0 + threadIdx.x / kRowLanes + u * (THREADS / kRowLanes);
    x[u] = i < n ? rope_get(t.in(i), L) : make_uint4(0, 0, 0, 0);
  }
}

// Every row of a token, the first round's already in x.  All threads of the block,
// after the angles (cs) are visible to them.
template <int DT, int THREADS, int AHEAD>
__device__ __forceinline__ void rope_token(const RopeParams& p, RopeLane& L, const float2* cs, const TokenRows& t,
                                           uint4 (&x)[AHEAD]) {
  const int grp = threadIdx.x / kRowLanes, n = t.rows();
  rope_coefficients(L, cs);
  const uint4 wq = rope_permute(rope_weights(p.q_weight, L), L), wk = rope_permute(rope_weights(p.k_weight, L), L);
  const bool any = p.q_weight != nullptr || p.k_weight != nullptr;
  constexpr int kStep = THREADS / kRowLanes;
  for (int r0 = 0; r0 < n; r0 += AHEAD * kStep) {
    if (r0 > 0) rope_load<THREADS>(t, L, r0, x);
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int first = r0 + u * kStep;  // the block's rows of this step from here
      if (first >= n) break;
      const int i = first + grp;
      uint4 y = x[u];
      if (first < t.H1 + t.H2) {  // some row of the step rotates: whole warps take part
        const bool key = i >= t.H1;
        const bool norm = (key ? p.k_weight : p.q_weight) != nullptr;
        const uint4 z = rope_row<DT>(x[u], L, key ? wk : wq, any, norm, p.eps);
        if (i < t.H1 + t.H2) y = z;
      }
      if (i < n) rope_put(t.out(i), L, y);
    }
  }
}

}  // namespace kitty
