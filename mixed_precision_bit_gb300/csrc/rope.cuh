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
constexpr int kRopeThreads = 128;         // eight rows at a time

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

// What a lane keeps for the rows it handles at one position: the coefficients of
// its own channels and of each one's partner in its pair,
//   y[i] = x[i] * c[i] + partner[i] * s[i],
// and where the partners are.  Half layout: rot / 2 is a multiple of 8, so all eight
// partners sit in one other lane of the row; interleaved: in the same lane.  Lanes
// past the rotated channels pass theirs through.
struct RopeLane {
  float c[8], s[8];
  int src;   // lane (of the warp) that holds the partners (half layout)
  bool on, interleaved;  // on: this lane's channels rotate
};

__device__ __forceinline__ RopeLane rope_lane(const RopeParams& p, const float2* cs) {
  RopeLane L;
  const int lane = threadIdx.x & 31, ch = (lane & (kRowLanes - 1)) * 8;
  L.interleaved = p.interleaved != 0;
  L.src = lane;
  L.on = ch < p.rot;
#pragma unroll
  for (int i = 0; i < 8; ++i) L.c[i] = L.s[i] = 0.f;
  if (L.on) {
    const int h = p.rot / 2;
    if (L.interleaved) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 a = cs[(ch + i) / 2];
        L.c[i] = L.c[i + 1] = a.x;
        L.s[i] = -a.y;
        L.s[i + 1] = a.y;
      }
    } else {
      const bool first = ch < h;
      L.src = first ? lane + h / 8 : lane - h / 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 a = cs[first ? ch + i : ch + i - h];
        L.c[i] = a.x;
        L.s[i] = first ? -a.y : a.y;
      }
    }
  }
  return L;
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

// Eight weights of this lane's channels (all 1 without a weight).
template <int DT>
__device__ __forceinline__ void rope_weights(const uint16_t* w, float (&f)[8]) {
  const int ch = (threadIdx.x & (kRowLanes - 1)) * 8;
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = w != nullptr ? load16<DT>(w + ch + i) : 1.f;
}

// One row: x = this lane's eight channels in, normed (weight != null) and rotated
// out.  Called by whole warps; rows are 16 lanes, so a warp takes two.
template <int DT>
__device__ __forceinline__ uint4 rope_row(uint4 x, const RopeLane& L, const float (&w)[8], bool norm,
                                          float eps) {
  float f[8];
  const uint32_t in[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = unpack16<DT>(in[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
  if (__any_sync(0xFFFFFFFFu, norm)) {  // the warp's two rows may be a query's and a key's
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
    const float r = rsqrtf(fmaf(ss, 1.0f / kD, eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = norm ? f[i] * r * w[i] : f[i];
  }
  float y[8];
  if (L.interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = fmaf(f[i], L.c[i], f[i ^ 1] * L.s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      y[i] = fmaf(f[i], L.c[i], __shfl_sync(0xFFFFFFFFu, f[i], L.src) * L.s[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = L.on ? y[i] : f[i];
  return make_uint4(pack16<DT>(y[0], y[1]), pack16<DT>(y[2], y[3]), pack16<DT>(y[4], y[5]),
                    pack16<DT>(y[6], y[7]));
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
    if (i < H1) return q + (size_t)i * kD;
    return i < H1 + H2 ? k + (size_t)(i - H1) * kD : v + (size_t)(i - H1 - H2) * kD;
  }
  __device__ uint16_t* out(int i) const {
    if (i < H1) return qo + (size_t)i * kD;
    return i < H1 + H2 ? ko + (size_t)(i - H1) * kv_stride : vo + (size_t)(i - H1 - H2) * kv_stride;
  }
};

// Rows a 16-lane group loads before it uses the first of them: with eight groups a
// block, 48 rows in one round of independent loads.
constexpr int kRopeAhead = 6;

// First round of a token's rows (nothing depends on its position yet).
__device__ __forceinline__ void rope_load(const TokenRows& t, int r0, uint4 (&x)[kRopeAhead]) {
  const int grp = threadIdx.x / kRowLanes, ch = (threadIdx.x & (kRowLanes - 1)) * 8, n = t.rows();
#pragma unroll
  for (int u = 0; u < kRopeAhead; ++u) {
    const int i = r0 + grp + u * (kRopeThreads / kRowLanes);
    x[u] = i < n ? *reinterpret_cast<const uint4*>(t.in(i) + ch) : make_uint4(0, 0, 0, 0);
  }
}

// Every row of a token, the first round's already in x.  All threads of the block,
// after the angles (cs) are visible to them.
template <int DT>
__device__ __forceinline__ void rope_token(const RopeParams& p, const float2* cs, const TokenRows& t,
                                           uint4 (&x)[kRopeAhead]) {
  const int grp = threadIdx.x / kRowLanes, ch = (threadIdx.x & (kRowLanes - 1)) * 8, n = t.rows();
  const RopeLane L = rope_lane(p, cs);
  float wq[8], wk[8];
  rope_weights<DT>(p.q_weight, wq);
  rope_weights<DT>(p.k_weight, wk);
  constexpr int kStep = kRopeThreads / kRowLanes;
  for (int r0 = 0; r0 < n; r0 += kRopeAhead * kStep) {
    if (r0 > 0) rope_load(t, r0, x);
#pragma unroll
    for (int u = 0; u < kRopeAhead; ++u) {
      const int first = r0 + u * kStep;  // the block's rows of this step: first .. first + 7
      if (first >= n) break;
      const int i = first + grp;
      uint4 y = x[u];
      if (first < t.H1 + t.H2) {  // some row of the step rotates: whole warps take part
        const bool key = i >= t.H1;
        const bool norm = (key ? p.k_weight : p.q_weight) != nullptr;
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = key ? wk[e] : wq[e];
        const uint4 z = rope_row<DT>(x[u], L, w, norm, p.eps);
        if (i < t.H1 + t.H2) y = z;
      }
      if (i < n) *reinterpret_cast<uint4*>(t.out(i) + ch) = y;
    }
  }
}

}  // namespace kitty
