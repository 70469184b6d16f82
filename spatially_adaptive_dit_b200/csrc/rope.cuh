// rope.cuh -- rotary positions on several axes, shared by the kernels that
// rotate rows (rope.cu) and that rotate them on the way into an 8-bit state
// (state8.cu).
//
// A row of d elements is cut into d / 8 slots of four pairs.  Pair p of a row
// turns by pos[axis(p)] * theta_axis^(-2 m / s) radians (m: the pair's place in
// its axis' segment of s elements); pairs behind the last segment do not turn.
// Interleaved pairs are neighbours, so a slot is 8 consecutive elements; pairs
// of halves are s / 2 apart, so a slot is two runs of 4 elements.
#pragma once

#include <cstdint>

#include "common.cuh"
#include "internal.h"

namespace sd {

constexpr int kMaxAxes = 4;
constexpr int kMaxPairs = 128;  // head dim up to 256

// One slot's constants side by side: lanes of a warp read different slots, and
// constant memory serves one address at a time, so few wide reads it is.
struct alignas(16) RopeSlot {
  double turn[4];    // theta^(-2 m / s) / (2 pi): turns per unit of position
  uint32_t axes;     // the pairs' axes, a byte each
  uint32_t runs;     // element offsets of the two runs of 4 elements / 4, a byte
                     // each, and above them the pairs that turn, a bit each
  __host__ __device__ static uint32_t pack(int lo, int hi) { return uint32_t(lo / 4) | uint32_t(hi / 4) << 8; }
  __host__ __device__ static int lo(uint32_t runs) { return int(runs & 255u) * 4; }
  __host__ __device__ static int hi(uint32_t runs) { return int(runs >> 8 & 255u) * 4; }
  __host__ __device__ static uint32_t turning(uint32_t runs) { return runs >> 16; }
};
struct RopeTable {
  RopeSlot slot[kMaxPairs / 4];
};

struct RopePos {
  const void* pos;  // [B or 1, tokens, axes] i32 or f32
  int f32;
  int64_t sb, st, sa;  // element strides
};

// Checks `rope` and `pos` against rows of d elements and fills the table and
// the position view.  *tokens: pos' token count.
safedit_status rope_setup(const safedit_rope* rope, const safedit_tensor* pos, int64_t B, int64_t d, RopeTable* tab,
                          RopePos* view, int64_t* tokens);

// cos and sin of the four angles of one slot at token i of batch b.  The
// angle is reduced to a fraction of a half turn in fp64 (a position of 2^20
// at frequency 1 leaves 2^-33 of it); what the fp32 argument of sincospif
// drops comes back as a first-order term, so both keep fp32 accuracy.
__device__ __forceinline__ void rope_angles(const RopeSlot& sl, const RopePos& v, int b, int64_t i, float sign,
                                            float (&c)[4], float (&s)[4]) {
  const uint32_t axes = sl.axes;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const double f = sl.turn[j];
    const int64_t at = int64_t(b) * v.sb + i * v.st + int64_t((axes >> (8 * j)) & 255u) * v.sa;
    const double x = v.f32 ? double(__ldg(static_cast<const float*>(v.pos) + at))
                           : double(__ldg(static_cast<const int32_t*>(v.pos) + at));
    double t = x * f;
    t = 2.0 * (t - rint(t));
    const float h = float(t);
    const float l = float(t - double(h)) * 3.14159274f;
    float sn, cs;
    sincospif(h, &sn, &cs);
    c[j] = fmaf(-l, sn, cs);
    s[j] = sign * fmaf(l, cs, sn);
    if (f == 0.0) {  // a pair that does not turn: no position reaches it, not even an infinite one
      c[j] = 1.f;
      s[j] = 0.f;
    }
  }
}

// Rotates the 8 elements of a slot in fp32: x[0..4) is the run at lo, x[4..8)
// the run at hi.  Pairs outside `turning` stay as they are: an infinity in one
// of their elements times the sine's 0 would make the other a NaN.
template <bool HALVES>
__device__ __forceinline__ void rope_turn(float (&x)[8], const float (&c)[4], const float (&s)[4],
                                          uint32_t turning = 15u) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (!(turning >> j & 1u)) continue;
    float& a = HALVES ? x[j] : x[2 * j];
    float& b = HALVES ? x[4 + j] : x[2 * j + 1];
    const float bs = -b * s[j], as = a * s[j];
    a = fmaf(a, c[j], bs);
    b = fmaf(b, c[j], as);
  }
}

// Pairs that do not turn back to what they were, x0.
template <bool HALVES>
__device__ __forceinline__ void rope_keep(float (&x)[8], const float (&x0)[8], uint32_t turning) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int a = HALVES ? j : 2 * j, b = HALVES ? 4 + j : 2 * j + 1;
    if (!(turning >> j & 1u)) x[a] = x0[a], x[b] = x0[b];
  }
}

// ---- slots in memory: 8 elements of f32, bf16 or f16 as raw 32-bit words
template <typename T>
struct SlotWords {
  static constexpr int N = sizeof(T) == 4 ? 8 : 4;
};

template <typename T, bool HALVES>
__device__ __forceinline__ void slot_load(uint32_t (&w)[SlotWords<T>::N], const T* row, int lo, int hi) {
  if constexpr (sizeof(T) == 4) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(row + lo)), b = __ldcs(reinterpret_cast<const uint4*>(row + hi));
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  } else if constexpr (HALVES) {
    const uint2 a = __ldcs(reinterpret_cast<const uint2*>(row + lo)), b = __ldcs(reinterpret_cast<const uint2*>(row + hi));
    w[0] = a.x, w[1] = a.y, w[2] = b.x, w[3] = b.y;
  } else {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(row + lo));
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  }
}

template <typename T>
__device__ __forceinline__ void slot_widen(const uint32_t (&w)[SlotWords<T>::N], float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(w[e]);
  } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
      x[2 * e] = f.x;
      x[2 * e + 1] = f.y;
    }
  }
}

}  // namespace sd
