// attn_state8.cu -- attention of gathered query rows over an 8-bit state.
#include <cmath>

#include "attn_state8.cuh"
#include "state8.cuh"

namespace sd {

// ------------------------------------------------------------- few rows
// One CTA: 8 or 16 query rows of a (b, h) slice and a range of the keys.
// Bound by reading the state once: a producer warp keeps a ring of TMA copies
// of 64 keys' codes of K and V in flight, and four warps take 16 keys each of
// a stage.  Codes go from shared memory into the
// registers of the warp-level multiplication as they lie: the order of a
// row's elements inside the product is free as long as both operands agree,
// so each lane loads runs of consecutive bytes and hands them out as if they
// were the tile's scattered elements.
// Keys are the rows of both products and queries the columns, eight to a tile
// (NQ = 1 or 2 tiles), so a single query wastes an eighth of what it would as
// one of 16 rows:
//   scores^T = K Q^T: lane (g = lane / 4, t = lane % 4) loads bytes
//     [t D/4, (t+1) D/4) of keys g and g + 8; step s multiplies bytes 4 s..+3.
//     It then holds keys g, g + 8 of queries 2 t, 2 t + 1;
//   out^T = V^T W^T: the weights' 8 x 8 blocks are transposed between the
//     lanes; the lane loads, of keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9, the
//     elements of column group g, and interleaves them by bytes.
// One row over 25600 keys of 48 slices (d = 96, 236 MB): 45 to 48 us, 5.1 TB/s,
// in clusters of eight (42 us and a join of 5 in nine parts), against 107 us with
// the codes straight from global memory into registers (a group of keys ahead was
// all that fitted).  A slice whose scales are wide throughout takes 53 us.
// The copies' 128-byte (d = 128) or 64-byte (d = 64) swizzle keeps those reads
// off each other's banks; rows of 96 bytes are so by themselves.
constexpr int kRowWarps = 4;                         // warps that multiply
constexpr int kRowThreads8 = kRowWarps * 32 + 32;    // and the producer
constexpr int kStageKeys = 16 * kRowWarps;
template <int D>
struct RowsCfg {
  static constexpr int TILE = kStageKeys * D;        // codes of K (or V) of a stage
  static constexpr int NST = D == 128 ? 4 : (D == 96 ? 5 : 6);  // stages
  static constexpr int CTAS = D == 64 ? 4 : 3;       // on an SM
  static constexpr int SMEM = 1024 + NST * 2 * TILE;
  static_assert(NST * 2 * TILE >= (kRowWarps + 1) * 16 * D * 4, "the warps' results fit the ring");
  static_assert(D % 2 == 0, "and the cluster reads the joined rows by pairs from a multiple of 8 bytes on");
};
constexpr uint64_t kRowsDrainNs = 1000000000ull;

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Column of element i (0 <= i < D / 8) of column group g.
template <int D>
__device__ __forceinline__ constexpr int value_col(int g, int i) {
  if constexpr (D == 96) return i < 8 ? g * 8 + i : 64 + g * 4 + (i - 8);
  else return g * (D / 8) + i;
}

// Shared-memory offset of byte `col` of row r of a tile.
template <int D>
__device__ __forceinline__ uint32_t code_at(int r, int col) {
  const uint32_t off = uint32_t(r * D + col);
  if constexpr (D == 128) return off ^ (((off >> 7) & 7u) << 4);
  else if constexpr (D == 64) return off ^ (((off >> 7) & 3u) << 4);
  else return off;
}

__device__ __forceinline__ uint32_t lds_u32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ void lds_u64(uint32_t at, uint32_t& a, uint32_t& b) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(at));
}
__device__ __forceinline__ void lds_u128(uint32_t at, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(at));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// The values at shared-memory address `at` of the cluster's CTA `rank`.
__device__ __forceinline__ float4 lds4_of(uint32_t at, uint32_t rank) {
  float4 v;
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
               "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at), "r"(rank)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 lds2_of(uint32_t at, uint32_t rank) {
  float2 v;
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %2, %3;\n\tld.shared::cluster.v2.f32 {%0, %1}, [a];\n\t}"
               : "=f"(v.x), "=f"(v.y)
               : "r"(at), "r"(rank)
               : "memory");
  return v;
}
__device__ __forceinline__ void rows_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

template <int D, int NQ, bool PAD, bool E4M3>
__global__ void __launch_bounds__(kRowThreads8, RowsCfg<D>::CTAS)
    attn_state8_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                            const __grid_constant__ State8Params p) {
  using C = RowsCfg<D>;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int NT = D / 16;       // tiles of 16 output columns
  constexpr int ROWS = 8 * NQ;     // query rows of the CTA
  constexpr bool CLEAR = PAD && E4M3;  // codes of masked keys may be NaN
  extern __shared__ __align__(16) uint8_t rows_smem[];
  __shared__ uint64_t full[C::NST], empty[C::NST];
  __shared__ int abort_word;
  __shared__ float sm_m[kRowWarps][ROWS], sm_l[kRowWarps][ROWS], sm_a[kRowWarps], sm_range[kRowWarps][2];
  __shared__ float4 cl_ml[ROWS];  // of all warps, for the cluster
  __shared__ __align__(8) float cl_range[2];
  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x, tile = blockIdx.y, bh = blockIdx.z;
  const int b = bh / p.H, h = bh - b * p.H;
  const int ns = (p.Nk + kStageKeys - 1) / kStageKeys;  // stages of the whole slice
  const int s_lo = int(int64_t(ns) * split / p.n_split), s_hi = int(int64_t(ns) * (split + 1) / p.n_split);
  const uint32_t ring = (smem_u32(rows_smem) + 1023u) & ~1023u;
  if (threadIdx.x == kRowWarps * 32) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), kRowWarps);
    }
    abort_word = 0;
    mbar_fence_init();
  }
  __syncthreads();
  const WaitCtl ctl{&abort_word, p.status, p.wait_limit};

  // queries 2 t and 2 t + 1 of each tile of eight
  float m[NQ][2], l[NQ][2];
  float lv_lo = INFINITY, lv_hi = -INFINITY;
  float base = NAN, lv_top = -INFINITY;  // of this warp's V scales (base: NaN before the first)
  bool ok = true;
  float o[NQ][NT][4];
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    m[q][0] = m[q][1] = -INFINITY;
    l[q][0] = l[q][1] = 0.f;
#pragma unroll
    for (int i = 0; i < NT; ++i) o[q][i][0] = o[q][i][1] = o[q][i][2] = o[q][i][3] = 0.f;
  }

  if (warp == kRowWarps) {
    // ------------------------------------------------ producer
    if (lane == 0) {
      int n = 0;
      for (int st = s_lo; st < s_hi; ++st, ++n) {
        const int i = n % C::NST;
        if (!wait_bounded(smem_u32(&empty[i]), uint32_t(((n / C::NST) & 1) ^ 1), ctl)) break;
        const uint32_t at = ring + uint32_t(i * 2 * C::TILE);
        mbar_arrive_expect_tx(smem_u32(&full[i]), 2 * C::TILE);
        tma_load_4d(at, &tmK, smem_u32(&full[i]), 0, st * kStageKeys, h, b);
        tma_load_4d(at + uint32_t(C::TILE), &tmV, smem_u32(&full[i]), 0, st * kStageKeys, h, b);
      }
      // every copy has landed before the CTA leaves
      for (int i = n > C::NST ? n - C::NST : 0; i < n; ++i)
        wait_drain(smem_u32(&full[i % C::NST]), uint32_t((i / C::NST) & 1), kRowsDrainNs);
    }
  } else {
    // ---- query row g of each tile of eight, f16, in the order of the key runs
    uint32_t bq[NQ][D / 16][2];
    float undo[NQ][2];  // of queries 2 t and 2 t + 1
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int r = tile * ROWS + 8 * q + g;
      int qi = -1;
      if (r < p.n_rows) {
        qi = p.idx ? __ldg(p.idx + r) : r;
        if (qi < 0 || qi >= p.Nq) {
          set_status(p.status, SAFEDIT_ERR_INDEX);
          qi = -1;
        }
      }
      uint32_t raw[D / 8];
#pragma unroll
      for (int c = 0; c < D / 8; ++c) raw[c] = 0u;
      if (qi >= 0) {
        const uint2* src =
            reinterpret_cast<const uint2*>(p.q + b * p.q_sb + h * p.q_sh + int64_t(qi) * p.q_sr + t * (D / 4));
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint2 x = __ldg(src + c);
          raw[2 * c] = x.x, raw[2 * c + 1] = x.y;
        }
      }
      uint32_t mb = 0u;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) mb = max(mb, max((raw[c] << 16) & 0x7FFF0000u, raw[c] & 0x7FFF0000u));
      mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
      mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 2));
      float un;
      const float f = query_factor(mb, p.scale_log2, un);
      undo[q][0] = __shfl_sync(0xffffffffu, un, 8 * t);
      undo[q][1] = __shfl_sync(0xffffffffu, un, 8 * t + 4);
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        bq[q][s][0] = pack_f16x2(__uint_as_float(raw[2 * s] << 16) * f, __uint_as_float(raw[2 * s] & 0xFFFF0000u) * f);
        bq[q][s][1] =
            pack_f16x2(__uint_as_float(raw[2 * s + 1] << 16) * f, __uint_as_float(raw[2 * s + 1] & 0xFFFF0000u) * f);
      }
    }
    const float* ksb = p.ks + b * p.ks_sb + h * p.ks_sh;
    const float* vsb = p.vs + b * p.vs_sb + h * p.vs_sh;
    const float* padb = PAD ? p.pad + b * p.pad_sb : nullptr;
    const int last_block = (p.Nk - 1) >> p.block_log2;
    bool bad = false;
    // scales and pads of the next stage are fetched a stage ahead: pads of keys
    // g, g + 8 and, where codes have to be cleared, 2 t, 2 t + 1, 2 t + 8, 2 t + 9
    float ks_n = 0.f, vs_n = 1.f, pad_n[2] = {0.f, 0.f}, padv_n[4] = {0.f, 0.f, 0.f, 0.f};
    auto pad_of = [&](int key) { return key < p.Nk ? __ldg(padb + key) : -INFINITY; };
    auto fetch = [&](int st) {
      const int key0 = st * kStageKeys + warp * 16;
      const int blk = min(key0 >> p.block_log2, last_block);
      ks_n = __ldg(ksb + blk);
      vs_n = __ldg(vsb + blk);
      if constexpr (PAD) {
        pad_n[0] = pad_of(key0 + g), pad_n[1] = pad_of(key0 + g + 8);
        if constexpr (CLEAR) {
#pragma unroll
          for (int e = 0; e < 4; ++e) padv_n[e] = pad_of(key0 + 2 * t + (e & 1) + 8 * (e >> 1));
        }
      }
    };
    if (s_lo < s_hi) fetch(s_lo);
    for (int st = s_lo, n = 0; st < s_hi; ++st, ++n) {
      const float ks = ks_n, vs = vs_n, pad[2] = {pad_n[0], pad_n[1]};
      const float padv[4] = {padv_n[0], padv_n[1], padv_n[2], padv_n[3]};
      if (st + 1 < s_hi) fetch(st + 1);
      const int i = n % C::NST;
      if (!wait_warp(smem_u32(&full[i]), uint32_t((n / C::NST) & 1), ctl)) {
        ok = false;
        break;
      }
      const int key0 = st * kStageKeys + warp * 16;
      // a group past the end, or of masked keys alone (its scales may be anything)
      bool live = key0 < p.Nk;
      if constexpr (PAD) live = __any_sync(0xffffffffu, pad[0] != -INFINITY || pad[1] != -INFINITY);
      if (live) {
        const uint32_t kt = ring + uint32_t(i * 2 * C::TILE), vt = kt + uint32_t(C::TILE);
        float lv = __log2f(vs);
        // finite, ks >= 0, vs > 0, by their bits
        bad |= __float_as_uint(ks) >= 0x7F800000u || __float_as_uint(vs) - 1u >= 0x7F7FFFFFu;
        scale_range(vs, lv, lv_lo, lv_hi);
        if (base != base) base = scale_base(lv);
        lv -= base;
        lv_top = fmaxf(lv_top, lv);
        const bool wide = lv < lv_top - kHalfSpread || lv > kHalfSpread;
        float s[NQ][4];
#pragma unroll
        for (int q = 0; q < NQ; ++q) s[q][0] = s[q][1] = s[q][2] = s[q][3] = 0.f;
        {
          uint32_t w[2][D / 16];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = warp * 16 + g + 8 * e;
            if constexpr (D == 96) {
#pragma unroll
              for (int c = 0; c < 3; ++c) lds_u64(kt + code_at<D>(r, t * 24 + c * 8), w[e][2 * c], w[e][2 * c + 1]);
            } else {
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                lds_u128(kt + code_at<D>(r, t * (D / 4) + c * 16), w[e][4 * c], w[e][4 * c + 1], w[e][4 * c + 2],
                         w[e][4 * c + 3]);
            }
          }
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint32_t x0 = bias_codes<E4M3>(w[0][c]), x1 = bias_codes<E4M3>(w[1][c]);
            const uint32_t a[4] = {widen_lo<E4M3>(x0), widen_lo<E4M3>(x1), widen_hi<E4M3>(x0), widen_hi<E4M3>(x1)};
#pragma unroll
            for (int q = 0; q < NQ; ++q) mma_16816(s[q], a, bq[q][c][0], bq[q][c][1]);
          }
        }
        // exponents against the queries' references; element e: key g + 8 (e / 2),
        // query 2 t + e % 2
        bool up = false;
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float f = undo[q][e & 1] * ks;
            if constexpr (PAD)
              s[q][e] = pad[e >> 1] == -INFINITY ? -INFINITY : fmaf(s[q][e], f, pad_log2(pad[e >> 1]));
            else
              s[q][e] *= f;
          }
          if (!PAD && key0 + 16 > p.Nk) {
            if (key0 + g >= p.Nk) s[q][0] = s[q][1] = -INFINITY;
            if (key0 + g + 8 >= p.Nk) s[q][2] = s[q][3] = -INFINITY;
          }
          // (as the exponents below, so that no weight leaves f16)
          up |= (fmaxf(s[q][0], s[q][2]) - m[q][0]) + lv > kLazyTop;
          up |= (fmaxf(s[q][1], s[q][3]) - m[q][1]) + lv > kLazyTop;
        }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float top = fmaxf(s[q][e], s[q][e + 2]) + lv;
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
              top -= kHeadroom;
              if (top > m[q][e]) {
                const float al = ex2_approx(m[q][e] - top);  // 0 from m = -inf
                m[q][e] = top;
                l[q][e] *= al;
#pragma unroll
                for (int c = 0; c < NT; ++c) {
                  o[q][c][e] *= al;
                  o[q][c][e + 2] *= al;
                }
              }
            }
        }
        const float inv = ex2_approx(-lv);
        uint32_t bp[NQ][2];
        // Wide: a group's weights go by their own largest, with the sums so far
        // brought to that and back (16 keys of one scale are a step of the product).
        float alone[NQ][2];
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float mm = m[q][e & 1] == -INFINITY ? 0.f : m[q][e & 1];
            s[q][e] = (s[q][e] - mm) + lv;
            w[e] = ex2_approx(s[q][e]);
          }
          l[q][0] = fmaf(w[0] + w[2], inv, l[q][0]);
          l[q][1] = fmaf(w[1] + w[3], inv, l[q][1]);
          if (wide) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float top = fmaxf(s[q][e], s[q][e + 2]);
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
              top = fmaxf(rintf(top - kHeadroom), -88.f);
              w[e] = ex2_approx(s[q][e] - top);
              w[e + 2] = ex2_approx(s[q][e + 2] - top);
              alone[q][e] = pow2(top);
#pragma unroll
              for (int c = 0; c < NT; ++c) {
                o[q][c][e] *= pow2(-top);
                o[q][c][e + 2] *= pow2(-top);
              }
            }
          }
          bp[q][0] = transpose_8x8(pack_f16x2(w[0], w[1]));
          bp[q][1] = transpose_8x8(pack_f16x2(w[2], w[3]));
        }
        uint32_t w[4][D / 32];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = warp * 16 + 2 * t + (e & 1) + 8 * (e >> 1);
          if constexpr (D == 128) {
            lds_u128(vt + code_at<D>(r, g * 16), w[e][0], w[e][1], w[e][2], w[e][3]);
          } else {
            lds_u64(vt + code_at<D>(r, g * 8), w[e][0], w[e][1]);
            if constexpr (D == 96) w[e][2] = lds_u32(vt + code_at<D>(r, 64 + g * 4));
          }
          if constexpr (CLEAR) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
              if (padv[e] == -INFINITY) w[e][c] = 0u;
          }
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = bias_codes<E4M3>(w[e][c]);
          // bytes of keys (0, 1) and (2, 3) side by side, column by column
          const uint32_t u0 = __byte_perm(x[0], x[1], 0x5140), u1 = __byte_perm(x[0], x[1], 0x7362);
          const uint32_t v0 = __byte_perm(x[2], x[3], 0x5140), v1 = __byte_perm(x[2], x[3], 0x7362);
          const uint32_t a0[4] = {widen_lo<E4M3>(u0), widen_hi<E4M3>(u0), widen_lo<E4M3>(v0), widen_hi<E4M3>(v0)};
          const uint32_t a1[4] = {widen_lo<E4M3>(u1), widen_hi<E4M3>(u1), widen_lo<E4M3>(v1), widen_hi<E4M3>(v1)};
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            mma_16816(o[q][2 * c], a0, bp[q][0], bp[q][1]);
            mma_16816(o[q][2 * c + 1], a1, bp[q][0], bp[q][1]);
          }
        }
        if (wide) {
#pragma unroll
          for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int c = 0; c < NT; ++c)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[q][c][e] *= alone[q][e & 1];
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&empty[i]));
    }
    if (bad) set_status(p.status, SAFEDIT_ERR_INVALID_ARG);
  }
  // A wait ran out: reported, nothing is written.  (A cluster's CTAs still meet:
  // the others read this one's results, which are then as unspecified as its own.)
  if (__syncthreads_or(!ok) && !p.cluster) return;

  // ---- the warps' results joined in shared memory
  float up = 1.f, base_a = 0.f;
  if (warp < kRowWarps) {
    if (base != base) base = 0.f;
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        base_a = leave_base(base, l[q][e], up);
        l[q][e] += __shfl_xor_sync(0xffffffffu, l[q][e], 4);
        l[q][e] += __shfl_xor_sync(0xffffffffu, l[q][e], 8);
        l[q][e] += __shfl_xor_sync(0xffffffffu, l[q][e], 16);
        if (g == 0) sm_m[warp][8 * q + 2 * t + e] = m[q][e], sm_l[warp][8 * q + 2 * t + e] = l[q][e];
      }
    if (lane == 0) sm_a[warp] = base_a, sm_range[warp][0] = lv_lo, sm_range[warp][1] = lv_hi;
  }
  __syncthreads();
  // each warp's scaled output to the ring (its copies have all landed), added
  // in the warps' order
  float* const sm_part = reinterpret_cast<float*>(rows_smem + (ring - smem_u32(rows_smem)));
  if (warp < kRowWarps) {
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * q + 2 * t + e;
        RowRef ref;
#pragma unroll
        for (int v = 0; v < kRowWarps; ++v) ref.take(sm_m[v][r], sm_a[v]);
        const float f = ref.weight(m[q][e], base_a) * up;
        float* row = sm_part + (warp * ROWS + r) * D;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          row[value_col<D>(g, 2 * i)] = o[q][i][e] * f;
          row[value_col<D>(g, 2 * i + 1)] = o[q][i][e + 2] * f;
        }
      }
  }
  __syncthreads();
  auto joined = [&](int e) {  // element e of [ROWS][D]
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) v += sm_part[w * ROWS * D + e];
    return v;
  };
  for (int w = 0; w < kRowWarps; ++w) lv_lo = fminf(lv_lo, sm_range[w][0]), lv_hi = fmaxf(lv_hi, sm_range[w][1]);
  RowRef ref;
  float lx = 0.f;  // of row threadIdx.x
  if (threadIdx.x < ROWS) {
    for (int w = 0; w < kRowWarps; ++w) ref.take(sm_m[w][threadIdx.x], sm_a[w]);
    for (int w = 0; w < kRowWarps; ++w)  // (scores of NaN leave m at -inf and l at NaN, which stays)
      lx = fmaf(ref.weight(sm_m[w][threadIdx.x], sm_a[w]), sm_l[w][threadIdx.x], lx);
  }
  if (p.cluster) {
    // ---- the parts joined by the cluster's CTAs: each takes its share of the
    // elements and adds the parts in their order
    float* const own = sm_part + kRowWarps * ROWS * D;
    for (int e = threadIdx.x; e < p.tile_rows * D; e += kRowThreads8) own[e] = joined(e);
    if (threadIdx.x < ROWS) cl_ml[threadIdx.x] = make_float4(ref.m, lx, ref.a, 0.f);
    if (threadIdx.x == 0) cl_range[0] = lv_lo, cl_range[1] = lv_hi;
    rows_cluster_sync();
    const uint32_t own_s = smem_u32(own), ml_s = smem_u32(cl_ml), range_s = smem_u32(cl_range);
    if (split == 0 && threadIdx.x == 0) {
      for (int s = 0; s < p.n_split; ++s) {
        const float2 range = lds2_of(range_s, s);
        lv_lo = fminf(lv_lo, range.x), lv_hi = fmaxf(lv_hi, range.y);
      }
      if (lv_hi - lv_lo > kScaleSpread) set_status(p.status, SAFEDIT_ERR_INVALID_ARG);
    }
    for (int e = split * kRowThreads8 + threadIdx.x; e < p.tile_rows * D / 2; e += p.n_split * kRowThreads8) {
      const int rr = e / (D / 2), c = (e - rr * (D / 2)) * 2, r = tile * ROWS + rr;
      if (r >= p.n_rows) break;
      const int qi = p.idx ? __ldg(p.idx + r) : r;
      if (qi < 0 || qi >= p.Nq) continue;
      RowRef all;
#pragma unroll 4
      for (int s = 0; s < p.n_split; ++s) {
        const float4 ml = lds4_of(ml_s + uint32_t(rr * 16), s);
        all.take(ml.x, ml.z);
      }
      float ls = 0.f, a0 = 0.f, a1 = 0.f;
#pragma unroll 4
      for (int s = 0; s < p.n_split; ++s) {
        const float4 ml = lds4_of(ml_s + uint32_t(rr * 16), s);
        const float2 x = lds2_of(own_s + uint32_t(e * 8), s);
        const float w = all.weight(ml.x, ml.z);
        ls = fmaf(w, ml.y, ls);
        a0 = fmaf(w, x.x, a0);
        a1 = fmaf(w, x.y, a1);
      }
      if (ls == 0.f && c == 0) set_status(p.status, SAFEDIT_ERR_MASKED_ROW);
      const float inv = ls == 0.f ? 0.f : 1.f / ls;
      a0 *= inv, a1 *= inv;
      if (a0 != a0 || a1 != a1) report_nan(p, b, h, qi, D);
      const int64_t orow = p.out_scattered ? int64_t(qi) : int64_t(r);
      *reinterpret_cast<uint32_t*>(p.out + b * p.o_sb + h * p.o_sh + orow * p.o_sr + c) = pack_bf16x2(a0, a1);
    }
    rows_cluster_sync();  // nobody leaves while another still reads it
    return;
  }
  if (p.n_split > 1) {
    const PartView pv = part_view(p, (int64_t(bh) * p.n_tiles + tile) * p.n_split + split, D);
    for (int e = threadIdx.x; e < p.tile_rows * D; e += kRowThreads8) pv.o[e] = joined(e);
    if (threadIdx.x < p.tile_rows) pv.ml[threadIdx.x] = make_float4(ref.m, lx, ref.a, 0.f);
    if (threadIdx.x == 0) pv.range[0] = lv_lo, pv.range[1] = lv_hi;
    return;
  }
  if (threadIdx.x == 0 && lv_hi - lv_lo > kScaleSpread) set_status(p.status, SAFEDIT_ERR_INVALID_ARG);
  __syncthreads();  // every sm_l has been read
  if (threadIdx.x < ROWS) sm_l[0][threadIdx.x] = lx;
  __syncthreads();
  for (int e = threadIdx.x; e < ROWS * D / 2; e += kRowThreads8) {
    const int rr = e / (D / 2), c = (e - rr * (D / 2)) * 2, r = tile * ROWS + rr;
    if (r >= p.n_rows) break;
    const int qi = p.idx ? __ldg(p.idx + r) : r;
    if (qi < 0 || qi >= p.Nq) continue;
    const float ls = sm_l[0][rr];
    if (ls == 0.f && c == 0) set_status(p.status, SAFEDIT_ERR_MASKED_ROW);
    const float inv = ls == 0.f ? 0.f : 1.f / ls;
    const float a0 = joined(rr * D + c) * inv, a1 = joined(rr * D + c + 1) * inv;
    if (a0 != a0 || a1 != a1) report_nan(p, b, h, qi, D);
    const int64_t orow = p.out_scattered ? int64_t(qi) : int64_t(r);
    *reinterpret_cast<uint32_t*>(p.out + b * p.o_sb + h * p.o_sh + orow * p.o_sr + c) = pack_bf16x2(a0, a1);
  }
}

// ------------------------------------------------------------- parts joined
// One CTA for each query row: m = max m_i, out = sum 2^(m_i - m) O_i /
// sum 2^(m_i - m) l_i over the row's parts, m_i the reference of a part.  Each warp takes every
// kJoinWarps-th part and the warps' sums are added in their order, so the
// result does not depend on timing.  A few microseconds of dependent loads:
// one thread per column over all parts in turn took 41 us at 200 parts.
template <int D, int kJoinWarps>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_state8_join_kernel(const __grid_constant__ State8Params p) {
  __shared__ float sm_red[4][kJoinWarps], sm_l[kJoinWarps], sm_o[kJoinWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pu = blockIdx.x / p.tile_rows, rr = blockIdx.x - pu * p.tile_rows;
  const int unit = p.n_full + pu;
  const int bh = unit / p.n_tiles, r = (unit - bh * p.n_tiles) * p.unit_rows + rr;
  const int b = bh / p.H, h = bh - b * p.H;
  int qi = -1;
  if (r < p.n_rows) qi = p.idx ? __ldg(p.idx + r) : r;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (qi < 0 || qi >= p.Nq) return;  // no row, or reported by the attention kernel
  const int n_rec = p.n_split << p.dual;
  const int64_t rec0 = int64_t(pu) * n_rec;
  RowRef ref;
  float lo = INFINITY, hi = -INFINITY;
  for (int s = threadIdx.x; s < n_rec; s += kJoinWarps * 32) {
    const PartView v = part_view(p, rec0 + s, D);
    const float4 ml = v.ml[rr];
    ref.take(ml.x, ml.z);
    lo = fminf(lo, v.range[0]), hi = fmaxf(hi, v.range[1]);
  }
#pragma unroll
  for (int e = 16; e; e >>= 1) {
    const float m = __shfl_xor_sync(0xffffffffu, ref.m, e), a = __shfl_xor_sync(0xffffffffu, ref.a, e);
    ref.take(m, a);
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, e));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, e));
  }
  if (lane == 0) sm_red[0][warp] = ref.m, sm_red[1][warp] = lo, sm_red[2][warp] = hi, sm_red[3][warp] = ref.a;
  __syncthreads();
  ref = RowRef();  // in the warps' order, so that all take the same
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    ref.take(sm_red[0][w], sm_red[3][w]);
    lo = fminf(lo, sm_red[1][w]), hi = fmaxf(hi, sm_red[2][w]);
  }
  float l = 0.f, acc[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int s = warp; s < n_rec; s += kJoinWarps) {
    const PartView v = part_view(p, rec0 + s, D);
    const float4 ml = v.ml[rr];
    float x[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) x[e] = v.o[rr * D + lane + 32 * e];
    const float w = ref.weight(ml.x, ml.z);
    l = fmaf(w, ml.y, l);
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] = fmaf(w, x[e], acc[e]);
  }
#pragma unroll
  for (int e = 0; e < D / 32; ++e) sm_o[warp][lane + 32 * e] = acc[e];
  if (lane == 0) sm_l[warp] = l;
  __syncthreads();
  if (threadIdx.x >= D) return;
  float sum = 0.f;
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) sum += sm_o[w][threadIdx.x], l += sm_l[w];
  if (threadIdx.x == 0) {
    if (hi - lo > kScaleSpread) set_status(p.status, SAFEDIT_ERR_INVALID_ARG);
    if (l == 0.f) set_status(p.status, SAFEDIT_ERR_MASKED_ROW);
  }
  sum = l == 0.f ? 0.f : sum / l;
  if (sum != sum) report_nan(p, b, h, qi, D);
  const int64_t orow = p.out_scattered ? int64_t(qi) : int64_t(r);
  p.out[b * p.o_sb + h * p.o_sh + orow * p.o_sr + threadIdx.x] = __float2bfloat16_rn(sum);
}

// ------------------------------------------------------------- plan
struct State8Plan {
  bool tc = false, dual = false, cluster = false;
  int unit_rows = 16, tile_rows = 16, n_tiles = 0, n_full = 0, n_split = 1;
  int64_t n_parts = 0, n_records = 0;  // units that run in parts, and their records
  size_t ws_bytes = 0;
};

static int state8_sms() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
    sms = 148;
  return sms;
}

// Rows of a slice up to which the warp-level kernel is taken.  Measured when the
// rule was made (both are some 7% slower since they look at the scales' range:
// 32 rows 113, 48 rows 128), us, warp-level / tensor-core kernel: 48 slices x 25600 keys of 96: 16 rows 64 /
// 120, 32 rows 108 / 118, 48 rows 148 / 122; x 4096 keys: 16 rows 23 / 33, 32
// rows 30 / 33, 48 rows 37 / 36; 32 slices x 16384 keys of 128: 32 rows 70 /
// 76, 48 rows 91 / 76; 4 slices x 4096 of 96: 32 rows 19 / 25.
constexpr int64_t kFewRows = 32;

static State8Plan plan_state8(int64_t n_rows, int64_t BH, int64_t Nk, int D, int sms) {
  State8Plan pl;
  pl.tc = n_rows > kFewRows;
  pl.unit_rows = pl.tc ? 256 : (n_rows <= 8 ? 8 : 16);
  pl.tile_rows = n_rows < pl.unit_rows ? int(n_rows) : pl.unit_rows;
  pl.n_tiles = int((n_rows + pl.unit_rows - 1) / pl.unit_rows);
  const int64_t units = pl.n_tiles * BH;
  if (units == 0) return pl;
  if (!pl.tc) {
    // One wave of what an SM holds.  Parts of three stages at least, joined by
    // a launch of their own (24 slices x 4999 keys, 13 rows: 9 parts 20.0 us, 24
    // parts 17.4 us), beyond 64 parts, which take their time to join, of eight
    // (one slice of 25600 keys: 200 parts were joined in 13 us).
    const int64_t wave = int64_t(sms) * (D == 64 ? RowsCfg<64>::CTAS : D == 96 ? RowsCfg<96>::CTAS : RowsCfg<128>::CTAS);
    const int64_t stages = (Nk + kStageKeys - 1) / kStageKeys;
    int64_t parts = stages < 16 ? 1 : stages / 3;
    if (parts > 64) parts = stages / 8 > 64 ? stages / 8 : 64;
    if (parts > wave / units) parts = wave / units;
    // Or as many CTAs of a cluster, which join their parts themselves: up to
    // the portable eight, from two stages each and eight stages on, and as many
    // as the GPU holds at once (clusters of two to eight fill 86.5% of its
    // places or more; nine for 48 slices left some for a second wave, 65 us
    // against 47).  The launch that this saves is worth twelve stages or so.
    // Measured in a captured graph when the rule was made, us, cluster / join: 24 slices x 4999 keys of
    // 64, 13 rows 14.0 / 15.0; 48 x 1000 of 96, 13 rows 10.5 / 13.1; 8 x 512 of
    // 96 5.9 / 7.5 (whole); 4 x 9000 of 128, 20 rows 21.8 / 15.5; launched one
    // by one, where a launch is the host's time: 48 x 25600 of 96, one row 46.6
    // / 49.0; 8 x 4096 of 96 18.6 / 23.6.
    int64_t c = stages < 8 ? 1 : int64_t(double(wave) * 0.865) / units;
    if (c > 8) c = 8;
    if (c > stages / 2) c = stages / 2;
    if (c > 1 && stages * (parts - c) <= 12 * c * parts) {
      pl.n_split = int(c);
      pl.cluster = true;
    } else if (parts > 1) {
      pl.n_split = int(parts);
      pl.n_parts = units;
    }
  } else {
    // The units that do not fill a wave of the SMs run as 2..16 parts over
    // the key tiles where that ends the call sooner.  Measured on B200: a CTA
    // costs about kFixedUs and, with both query tiles in use, 1.05 us + 6.8 ns
    // a column for each key tile of 128; the join kJoinUs and a pass over the
    // parts' records.  A predicted saving under 3% of the call did not show
    // (7680 rows x 25600 keys, 48 heads of 96: 3.63 ms whole, 3.72 ms with the
    // last 108 units in 4 parts; 4096 x 4096: 397 us whole, 369 us with 28
    // units in 4).
    constexpr double kFixedUs = 13.0, kJoinUs = 8.0;
    const int64_t nk = (Nk + 127) / 128;
    auto record_us = [&](int64_t records) { return double(records) * pl.tile_rows * D * 8 / 3.0e6; };
    if (n_rows <= 128) {
      // Both query tiles on the same rows, every unit in parts; or one tile
      // and no join, where there are few keys.
      constexpr double kDualTileUs = 1.2, kOneTileUs = 1.85;
      double best = double((units + sms - 1) / sms) * (kFixedUs + double(nk) * kOneTileUs);
      for (int s = 1; s <= 32 && s <= nk; ++s) {
        const double rounds = double((units * s + sms - 1) / sms);
        const double cost =
            rounds * (kFixedUs + double((nk + s - 1) / s) * kDualTileUs) + kJoinUs + record_us(units * s * 2);
        if (cost < best) best = cost, pl.n_split = s, pl.dual = true;
      }
      pl.n_parts = pl.dual ? units : 0;
    } else {
      const int64_t tail = units % sms;
      const double tile_us = 1.05 + 0.0068 * D;
      const double whole_us = kFixedUs + double(nk) * tile_us;
      double best = whole_us - 0.03 * whole_us * double((units + sms - 1) / sms);
      for (int s = 2; tail > 0 && s <= 16 && s <= nk; ++s) {
        const double rounds = double((tail * s + sms - 1) / sms);
        const double cost =
            rounds * (kFixedUs + double((nk + s - 1) / s) * tile_us) + kJoinUs + record_us(tail * s);
        if (cost < best) best = cost, pl.n_split = s;
      }
      pl.n_parts = pl.n_split > 1 ? tail : 0;
    }
  }
  pl.n_full = int(units - pl.n_parts);
  pl.n_records = (pl.n_parts * pl.n_split) << pl.dual;
  if (pl.n_parts) pl.ws_bytes = part_floats(pl.n_records, pl.tile_rows, D) * sizeof(float);
  return pl;
}

template <int D, int W>
static safedit_status launch_join(const State8Params& p, int64_t n_parts, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(n_parts * p.tile_rows));
  cfg.blockDim = dim3(W * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, attn_state8_join_kernel<D, W>, p) != cudaSuccess) return SAFEDIT_ERR_CUDA;
  return after_launch(1);
}

static safedit_status codes_map(CUtensorMap* m, const safedit_tensor* t) {
  const uint64_t dims[4] = {uint64_t(t->dims[3]), uint64_t(t->dims[2]), uint64_t(t->dims[1]), uint64_t(t->dims[0])};
  const uint64_t strides[3] = {uint64_t(t->strides[2]), uint64_t(t->strides[1]), uint64_t(t->strides[0])};
  const uint32_t box[4] = {uint32_t(t->dims[3]), uint32_t(kStageKeys), 1u, 1u};
  return encode_tmap(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, t->data, dims, strides, box,
                     t->dims[3] == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                     : t->dims[3] == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                        : CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <int D, bool PAD, bool E4M3>
static safedit_status launch_rows(const CUtensorMap& tmK, const CUtensorMap& tmV, const State8Params& p, int64_t BH,
                                  cudaStream_t s) {
  auto kern = p.unit_rows == 8 ? attn_state8_rows_kernel<D, 1, PAD, E4M3> : attn_state8_rows_kernel<D, 2, PAD, E4M3>;
  const safedit_status st = set_smem(reinterpret_cast<const void*>(kern), RowsCfg<D>::SMEM);
  if (st != SAFEDIT_OK) return st;
  const dim3 grid{unsigned(p.n_split), unsigned(p.n_tiles), unsigned(BH)};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kRowThreads8);
  cfg.dynamicSmemBytes = RowsCfg<D>::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(p.n_split);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kern, tmK, tmV, p) != cudaSuccess) return SAFEDIT_ERR_CUDA;
  return after_launch(1);
}

template <int D>
static safedit_status dispatch_state8(const safedit_tensor* k8, const safedit_tensor* v8, const State8Params& p,
                                      const State8Plan& pl, int64_t BH, cudaStream_t s) {
  safedit_status st;
  if (pl.tc) {
    st = launch_state8_tc(k8, v8, p, pl.n_full + pl.n_parts * pl.n_split, s);
  } else {
    CUtensorMap tmK, tmV;
    if ((st = codes_map(&tmK, k8)) != SAFEDIT_OK) return st;
    if ((st = codes_map(&tmV, v8)) != SAFEDIT_OK) return st;
    const bool e4m3 = k8->dtype == SAFEDIT_E4M3;
    if (p.pad)
      st = e4m3 ? launch_rows<D, true, true>(tmK, tmV, p, BH, s) : launch_rows<D, true, false>(tmK, tmV, p, BH, s);
    else
      st = e4m3 ? launch_rows<D, false, true>(tmK, tmV, p, BH, s) : launch_rows<D, false, false>(tmK, tmV, p, BH, s);
  }
  if (st != SAFEDIT_OK || pl.n_parts == 0) return st;
  // many parts of few rows, or few parts of many rows
  return pl.tc ? launch_join<D, 4>(p, pl.n_parts, s) : launch_join<D, 16>(p, pl.n_parts, s);
}

static safedit_status check_rows16(const safedit_tensor* t) {
  const safedit_status st = check_tensor(t, 4);
  if (st != SAFEDIT_OK) return st;
  if (t->dtype != SAFEDIT_BF16) return SAFEDIT_ERR_DTYPE;
  if (t->strides[3] != 1 || !aligned16(t->data)) return SAFEDIT_ERR_ALIGNMENT;
  for (int k = 0; k < 3; ++k)
    if (t->strides[k] % 8 != 0 || t->strides[k] < 0) return SAFEDIT_ERR_ALIGNMENT;
  return SAFEDIT_OK;
}

}  // namespace sd

using namespace sd;

extern "C" safedit_status safedit_attn_subset_state8(const safedit_tensor* q, const safedit_tensor* k8,
                                                     const safedit_tensor* k_scale, const safedit_tensor* v8,
                                                     const safedit_tensor* v_scale, int32_t block,
                                                     const int32_t* d_idx, int32_t n_idx,
                                                     const safedit_tensor* key_pad, float scale,
                                                     const safedit_tensor* out, int32_t out_scattered,
                                                     void* d_workspace, size_t workspace_bytes, void* stream) {
  safedit_status st;
  if ((st = check_rows16(q)) != SAFEDIT_OK) return st;
  if ((st = check_codes(k8)) != SAFEDIT_OK) return st;
  if ((st = check_codes(v8)) != SAFEDIT_OK) return st;
  if (!state8_block_ok(block)) return SAFEDIT_ERR_UNSUPPORTED;
  if ((st = check_scales(k_scale, k8, block)) != SAFEDIT_OK) return st;
  if ((st = check_scales(v_scale, v8, block)) != SAFEDIT_OK) return st;
  if ((st = check_rows16(out)) != SAFEDIT_OK) return st;
  if (k8->dtype != v8->dtype) return SAFEDIT_ERR_DTYPE;
  const int64_t B = q->dims[0], H = q->dims[1], Nq = q->dims[2], D = q->dims[3], Nk = k8->dims[2];
  for (const safedit_tensor* t : {k8, v8})
    if (t->dims[0] != B || t->dims[1] != H || t->dims[3] != D || t->dims[2] != Nk) return SAFEDIT_ERR_SHAPE;
  if (D != 64 && D != 96 && D != 128) return SAFEDIT_ERR_UNSUPPORTED;
  if (Nk < 1 || Nq > INT32_MAX || Nk > INT32_MAX - 256 || B * H > 65535) return SAFEDIT_ERR_SHAPE;
  if (out_scattered != 0 && out_scattered != 1) return SAFEDIT_ERR_INVALID_ARG;
  if (d_idx && n_idx < 0) return SAFEDIT_ERR_INVALID_ARG;
  const int64_t n_rows = d_idx ? n_idx : Nq;
  if (out->dims[0] != B || out->dims[1] != H || out->dims[3] != D) return SAFEDIT_ERR_SHAPE;
  if (out->dims[2] != (out_scattered ? Nq : n_rows)) return SAFEDIT_ERR_SHAPE;
  if ((n_rows + 255) / 256 * B * H * 16 > INT32_MAX) return SAFEDIT_ERR_SHAPE;  // parts counted in int
  State8Params p{};
  if (key_pad) {
    if ((st = check_tensor(key_pad, 2)) != SAFEDIT_OK) return st;
    if (key_pad->dtype != SAFEDIT_F32) return SAFEDIT_ERR_DTYPE;
    if (key_pad->dims[0] != B || key_pad->dims[1] != Nk) return SAFEDIT_ERR_SHAPE;
    if (key_pad->strides[1] != 1 || key_pad->strides[0] % 4 != 0 || key_pad->strides[0] < 0 ||
        !aligned16(key_pad->data))
      return SAFEDIT_ERR_ALIGNMENT;
    p.pad = static_cast<const float*>(key_pad->data);
    p.pad_sb = key_pad->strides[0];
  }
  const State8Plan pl = plan_state8(n_rows, B * H, Nk, int(D), state8_sms());
  if (pl.ws_bytes > 0) {
    if (!d_workspace || workspace_bytes < pl.ws_bytes) return SAFEDIT_ERR_INVALID_ARG;
    if (!aligned16(d_workspace)) return SAFEDIT_ERR_ALIGNMENT;
  }
  if (n_rows == 0 || B * H == 0) return SAFEDIT_OK;
  p.q = static_cast<const __nv_bfloat16*>(q->data);
  p.q_sb = q->strides[0], p.q_sh = q->strides[1], p.q_sr = q->strides[2];
  p.k = static_cast<const uint8_t*>(k8->data);
  p.k_sb = k8->strides[0], p.k_sh = k8->strides[1], p.k_sr = k8->strides[2];
  p.v = static_cast<const uint8_t*>(v8->data);
  p.v_sb = v8->strides[0], p.v_sh = v8->strides[1], p.v_sr = v8->strides[2];
  p.ks = static_cast<const float*>(k_scale->data);
  p.ks_sb = k_scale->strides[0], p.ks_sh = k_scale->strides[1];
  p.vs = static_cast<const float*>(v_scale->data);
  p.vs_sb = v_scale->strides[0], p.vs_sh = v_scale->strides[1];
  p.block_log2 = block == 16 ? 4 : block == 32 ? 5 : block == 64 ? 6 : 7;
  p.idx = d_idx;
  p.n_rows = int(n_rows);
  p.Nq = int(Nq);
  p.Nk = int(Nk);
  p.H = int(H);
  p.scale_log2 = ((scale > 0.f) ? scale : 1.0f / std::sqrt(float(D))) * kLog2eF;
  p.out = static_cast<__nv_bfloat16*>(out->data);
  p.o_sb = out->strides[0], p.o_sh = out->strides[1], p.o_sr = out->strides[2];
  p.out_scattered = out_scattered;
  p.wait_limit = wait_limit_ns();
  p.n_full = pl.n_full;
  p.n_split = pl.n_split;
  p.unit_rows = pl.unit_rows;
  p.tile_rows = pl.tile_rows;
  p.n_tiles = pl.n_tiles;
  p.n_records = pl.n_records;
  p.dual = pl.dual;
  p.cluster = pl.cluster;
  p.part = static_cast<float*>(d_workspace);
  p.status = status_ptr();
  if (!p.status) return SAFEDIT_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d_idx && out_scattered && index_check_enabled() &&
      (st = launch_index_check(d_idx, int32_t(n_rows), Nq, p.status, s)) != SAFEDIT_OK)
    return st;
  switch (D) {
    case 64: return dispatch_state8<64>(k8, v8, p, pl, B * H, s);
    case 96: return dispatch_state8<96>(k8, v8, p, pl, B * H, s);
    default: return dispatch_state8<128>(k8, v8, p, pl, B * H, s);
  }
}

extern "C" size_t safedit_attn_subset_state8_workspace_size(int64_t batch, int64_t heads, int64_t n_rows,
                                                            int64_t n_keys, int32_t head_dim) {
  if (batch <= 0 || heads <= 0 || n_rows <= 0 || n_keys <= 0) return 0;
  if (head_dim != 64 && head_dim != 96 && head_dim != 128) return 0;
  if (batch > 65535 || heads > 65535 || batch * heads > 65535 || n_keys > INT32_MAX - 256 ||
      n_rows > INT32_MAX || (n_rows + 255) / 256 * batch * heads * 16 > INT32_MAX)
    return 0;
  return plan_state8(n_rows, batch * heads, n_keys, head_dim, state8_sms()).ws_bytes;
}
