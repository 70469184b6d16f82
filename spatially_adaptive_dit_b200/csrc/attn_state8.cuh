// attn_state8.cuh -- what the two kernels of the attention over an 8-bit state
// share: the call's parameters, the widening of codes, the masks' arithmetic
// and the record of a part of the keys.
//
//   K = k8 * ks, V = v8 * vs (one scale for each block of keys and head)
//   t_j = (scale log2 e) ks q . k8_j + pad_j log2 e,   p_j = 2^t_j
//   out = sum_j p_j vs_j v8_j / sum_j p_j
//
// Scales never touch a code: ks goes into the score's factor, and vs into the
// exponent of the weight w_j = 2^(t_j + lv_j - m), lv = log2 vs - base, m 2^6
// below the running maximum of t_j + lv_j, which it follows lazily, by more than
// 2^8 at a time.  So the weights that the tensor cores multiply with the codes
// are at most 2^14 whatever the scales' range; the row sum is
// sum_j w_j 2^-lv_j in fp32.  The base, the first scale in use to the nearest
// power of two, comes back with the result.  It keeps lv small: a far pad
// absorbs it as it does the score, and the sum must neither overflow nor vanish
// at scales near the ends of fp32.
// A weight is rounded to f16: 2^-11, or, below 2^-14, 2^-25 in all, which is
// 2^-31 of the row's largest p_j vs_j.  Where scales differ, that is no share of
// the values that a small one stands for (a block of zeros beside rows of 1e-5
// has a scale 2^25 times theirs).  So keys whose scale lies further than 2^8
// below the largest so far are "wide" (and, with few rows, those as far above the
// base: a far pad, which nothing takes off there, leaves lv as the weight).
// With few rows their weights go by the largest of their own 16 keys; in the
// tensor-core kernel a tile with such a key has its weights as a pair of bf16
// (2^-16, to the end of fp32) and its codes of V as bf16.  Then 2^-23 max(p) |V_j|
// of a key is all that is lost beside 2^-11 of its share.
// Codes of both types are exact in f16 and bf16, as is a bf16 query row in f16
// after a power of two has brought its largest element to 2^12 (elements 2^-29
// below it lose bits: 2^-36 of the row's largest), so the weights alone are
// rounded.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace sd {

struct State8Params {
  const __nv_bfloat16* q;
  int64_t q_sb, q_sh, q_sr;
  const uint8_t *k, *v;
  int64_t k_sb, k_sh, k_sr, v_sb, v_sh, v_sr;
  const float *ks, *vs;
  int64_t ks_sb, ks_sh, vs_sb, vs_sh;
  int block_log2;
  const int* idx;  // nullable
  int n_rows, Nq, Nk, H;
  float scale_log2;  // softmax scale * log2(e)
  const float* pad;  // nullable, [B, Nk]
  int64_t pad_sb;
  __nv_bfloat16* out;
  int64_t o_sb, o_sh, o_sr;
  int out_scattered;
  int* status;
  uint64_t wait_limit;
  // Schedule: units of query rows (n_tiles of them in a (b, h) slice).  Units
  // below n_full run whole; each later one as n_split parts over the keys,
  // whose records (of `tile_rows` rows, see PartView) are joined afterwards, or,
  // with few rows, as the n_split CTAs of a cluster (`cluster`), no records.
  // With at most 128 rows both query tiles of the tensor-core kernel hold the
  // same rows and take the key tiles in turn (`dual`, two records a part).
  int n_full, n_split, unit_rows, tile_rows, n_tiles, dual, cluster;
  float* part;
  int64_t n_records;
};

constexpr float kLog2eF = 1.4426950408889634f;
constexpr float kScaleSpread = 64.f;  // log2 of the widest spread of V scales in one slice
constexpr float kOneSlack = 24.f;     // and by how much more one of exactly 1 (of a block of zeros) may lie off
constexpr float kHeadroom = 6.f;      // log2 of what a row's largest weight is at least ..
constexpr float kLazyTop = 14.f;      // .. and at most, in f16's range
constexpr float kHalfSpread = 8.f;    // V scales this near the largest (and the base) take f16 weights

// pad in log2 units; a finite pad stays finite, so a row whose keys all carry
// the type's lowest value averages them instead of being empty.
__device__ __forceinline__ float pad_log2(float pad) {
  const float v = pad * kLog2eF;
  return (fabsf(v) == INFINITY && fabsf(pad) != INFINITY) ? copysignf(3.0e38f, v) : v;
}

// Two codes in the low half of `w` -> f16x2, exact.
template <bool E4M3>
__device__ __forceinline__ uint32_t widen_lo(uint32_t w) {
  uint32_t r;
  if constexpr (E4M3) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  } else {  // bytes biased by 128: 0x6400 | u is 1024 + u in f16
    const uint32_t m = __byte_perm(w, 0x64646464u, 0x4140);
    asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(0x64806480u));
  }
  return r;
}
template <bool E4M3>
__device__ __forceinline__ uint32_t widen_hi(uint32_t w) {
  uint32_t r;
  if constexpr (E4M3) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
  } else {
    const uint32_t m = __byte_perm(w, 0x64646464u, 0x4342);
    asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(0x64806480u));
  }
  return r;
}
// What the widening expects: int8 codes biased to 0..255, e4m3 as they are.
template <bool E4M3>
__device__ __forceinline__ uint32_t bias_codes(uint32_t w) {
  return E4M3 ? w : w ^ 0x80808080u;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Factor 2^f that brings a row's largest magnitude (its fp32 bits) to
// [2^12, 2^13), and its inverse times `scale`.
__device__ __forceinline__ float query_factor(uint32_t max_bits, float scale, float& undo) {
  int e = int(max_bits >> 23) - 127;
  if (max_bits == 0u) e = -88;  // a zero row
  int f = 12 - e;
  f = f > 126 ? 126 : f;
  undo = scale * __uint_as_float(uint32_t(127 - f) << 23);
  return __uint_as_float(uint32_t(127 + f) << 23);
}

// f16x2 -> bf16x2 (exact for codes), two floats -> the bf16 pair that they begin
// with and, in their place, what it leaves.
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t v) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
  return pack_bf16x2(f.x, f.y);
}
__device__ __forceinline__ uint32_t take_bf16x2(float& lo, float& hi) {
  const uint32_t r = pack_bf16x2(lo, hi);
  lo -= __uint_as_float(r << 16);
  hi -= __uint_as_float(r & 0xFFFF0000u);
  return r;
}

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2(float e) { return __uint_as_float(uint32_t(127 + int(e)) << 23); }
// The range of a slice's V scales, a scale's log2 at a time.
__device__ __forceinline__ void scale_range(float vs, float lv, float& lo, float& hi) {
  lo = fminf(lo, vs == 1.f ? kOneSlack : lv);
  hi = fmaxf(hi, vs == 1.f ? -kOneSlack : lv);
}
// The base of V scales from the log2 of the first one in use.
__device__ __forceinline__ float scale_base(float lv) { return fminf(fmaxf(rintf(lv), -120.f), 120.f); }
// A row sum l relative to a base -> relative to `a`, which it returns, and the
// factor of O that goes with it.  l takes what leaves it in range (at most 2^60),
// O the rest: a block of zeros may have taken it 2^-88 below 1 already.
__device__ __forceinline__ float leave_base(float base, float& l, float& o_factor) {
  const float a = fmaxf(base, -60.f);
  l *= pow2(-a);
  o_factor = pow2(base - a);
  return a;
}
// The reference of a row's sums is 2^(m + a), kept apart: m may be the size of a
// far pad, which absorbs a.
struct RowRef {
  float m = -INFINITY, a = 0.f;
  // The larger one.
  __device__ __forceinline__ void take(float m2, float a2) {
    if ((m2 - m) + (a2 - a) > 0.f) m = m2, a = a2;
  }
  // Weight of sums that refer to (m2, a2); 0 of those without a key.
  __device__ __forceinline__ float weight(float m2, float a2) const {
    return m2 == -INFINITY ? 0.f : ex2_approx((m2 - m) + (a2 - a));
  }
};

// A row came out as NaN: where its query row is finite, a NaN among the codes
// (or the pads) did it.  Looked at where results leave, so that the loops over
// keys need not look at every code.
__device__ __forceinline__ void report_nan(const State8Params& p, int b, int h, int qi, int D) {
  const uint16_t* row = reinterpret_cast<const uint16_t*>(p.q + b * p.q_sb + h * p.q_sh + int64_t(qi) * p.q_sr);
#pragma unroll 1
  for (int c = 0; c < D; ++c)
    if ((__ldg(row + c) & 0x7F80u) == 0x7F80u) return;
  set_status(p.status, SAFEDIT_ERR_INVALID_ARG);
}

// A part's record: O [rows][D] unnormalised, (m, l, a, -) [rows], and the range
// of V scales that it met (of all records behind one another).
struct PartView {
  float* o;
  float4* ml;
  float* range;
};
__host__ __device__ inline size_t part_floats(int64_t records, int rows, int D) {
  return size_t(records) * (size_t(rows) * (D + 4) + 2);
}
__device__ __forceinline__ PartView part_view(const State8Params& p, int64_t rec, int D) {
  PartView v;
  v.o = p.part + rec * p.tile_rows * D;
  v.ml = reinterpret_cast<float4*>(p.part + p.n_records * p.tile_rows * D) + rec * p.tile_rows;
  v.range = p.part + p.n_records * p.tile_rows * (D + 4) + rec * 2;
  return v;
}

// The tensor-core kernel over `ctas` CTAs (whole units and parts).
safedit_status launch_state8_tc(const safedit_tensor* k8, const safedit_tensor* v8, const State8Params& p,
                                int64_t ctas, cudaStream_t s);

}  // namespace sd
