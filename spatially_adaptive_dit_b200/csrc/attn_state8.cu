// attn_state8.cu -- attention of gathered query rows over an 8-bit state.
#include <cmath>

#include "attn_state8.cuh"
#include "state8.cuh"

namespace sd {

// ------------------------------------------------------------- few rows
// One CTA: 16 query rows (one warp-level matrix tile) of a (b, h) slice and a
// range of the keys.  Bound by reading the state once: a producer warp keeps a
// ring of TMA copies of 64 keys' codes of K and V in flight, and four warps
// take 16 keys each of a stage.  Codes go from shared memory into the
// registers of the warp-level multiplication as they lie: the order of a
// row's elements inside the product is free as long as both operands agree,
// so each lane loads runs of consecutive bytes and hands them out as if they
// were the tile's scattered elements.
//   scores: lane (g = lane / 4, t = lane % 4) loads bytes [t D/4, (t+1) D/4) of
//     keys g and g + 8; step s multiplies bytes 4 s .. 4 s + 3.
//   values: it loads, of keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9 (whose weights it
//     holds), the elements of column group g, and interleaves them by bytes.
// The copies' 128-byte (d = 128) or 64-byte (d = 64) swizzle keeps those reads
// off each other's banks; rows of 96 bytes are so by themselves.
constexpr int kRowWarps = 4;                         // warps that multiply
constexpr int kRowThreads8 = kRowWarps * 32 + 32;    // and the producer
constexpr int kStageKeys = 16 * kRowWarps;
template <int D>
struct RowsCfg {
  static constexpr int TILE = kStageKeys * D;        // codes of K (or V) of a stage
  static constexpr int NST = D == 128 ? 6 : 8;       // stages
  static constexpr int CTAS = D == 128 ? 2 : (D == 96 ? 2 : 3);  // on an SM
  static constexpr int SMEM = 1024 + NST * 2 * TILE;
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

template <int D, bool PAD, bool E4M3>
__global__ void __launch_bounds__(kRowThreads8, RowsCfg<D>::CTAS)
    attn_state8_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                            const __grid_constant__ State8Params p) {
  using C = RowsCfg<D>;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int NT = D / 8;  // column tiles of the output
  extern __shared__ uint8_t rows_smem[];
  __shared__ uint64_t full[C::NST], empty[C::NST];
  __shared__ int abort_word;
  __shared__ float sm_m[kRowWarps][16], sm_l[kRowWarps][16], sm_range[kRowWarps][2];
  __shared__ float sm_o[16][D];
  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x, tile = blockIdx.y, bh = blockIdx.z;
  const int b = bh / p.H, h = bh - b * p.H;
  const int ns = (p.Nk + kStageKeys - 1) / kStageKeys;  // stages of the whole slice
  const int s_lo = int(int64_t(ns) * split / p.n_split), s_hi = int(int64_t(ns) * (split + 1) / p.n_split);
  const uint32_t ring = (smem_u32(rows_smem) + 1023u) & ~1023u;
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

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float lv_lo = INFINITY, lv_hi = -INFINITY;
  int my_q[2] = {-1, -1};
  bool ok = true;
  float o[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

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
    // ---- query rows g and g + 8 of the tile, f16, in the order of the key runs
    uint32_t aq[D / 16][4];
    float undo[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = tile * 16 + g + 8 * e;
      if (r < p.n_rows) {
        my_q[e] = p.idx ? __ldg(p.idx + r) : r;
        if (my_q[e] < 0 || my_q[e] >= p.Nq) {
          set_status(p.status, SAFEDIT_ERR_INDEX);
          my_q[e] = -1;
        }
      }
      uint32_t raw[D / 8];
#pragma unroll
      for (int c = 0; c < D / 8; ++c) raw[c] = 0u;
      if (my_q[e] >= 0) {
        const uint2* src = reinterpret_cast<const uint2*>(p.q + b * p.q_sb + h * p.q_sh + int64_t(my_q[e]) * p.q_sr +
                                                          t * (D / 4));
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
      const float f = query_factor(mb, p.scale_log2, undo[e]);
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        aq[s][e] = pack_f16x2(__uint_as_float(raw[2 * s] << 16) * f, __uint_as_float(raw[2 * s] & 0xFFFF0000u) * f);
        aq[s][e + 2] =
            pack_f16x2(__uint_as_float(raw[2 * s + 1] << 16) * f, __uint_as_float(raw[2 * s + 1] & 0xFFFF0000u) * f);
      }
    }
    const float* ksb = p.ks + b * p.ks_sb + h * p.ks_sh;
    const float* vsb = p.vs + b * p.vs_sb + h * p.vs_sh;
    const float* padb = PAD ? p.pad + b * p.pad_sb : nullptr;
    const int last_block = (p.Nk - 1) >> p.block_log2;
    bool bad = false;
    // scales and pads of the next stage are fetched a stage ahead
    float ks_n = 0.f, vs_n = 1.f, pad_n[4] = {0.f, 0.f, 0.f, 0.f};
    auto fetch = [&](int st) {
      const int key0 = st * kStageKeys + warp * 16;
      const int blk = min(key0 >> p.block_log2, last_block);
      ks_n = __ldg(ksb + blk);
      vs_n = __ldg(vsb + blk);
      if constexpr (PAD) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = key0 + 2 * t + (e & 1) + 8 * (e >> 1);
          pad_n[e] = key < p.Nk ? __ldg(padb + key) : -INFINITY;
        }
      }
    };
    if (s_lo < s_hi) fetch(s_lo);
    for (int st = s_lo, n = 0; st < s_hi; ++st, ++n) {
      const float ks = ks_n, vs = vs_n;
      float pad[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) pad[e] = pad_n[e];
      if (st + 1 < s_hi) fetch(st + 1);
      const int i = n % C::NST;
      if (!wait_warp(smem_u32(&full[i]), uint32_t((n / C::NST) & 1), ctl)) {
        ok = false;
        break;
      }
      const int key0 = st * kStageKeys + warp * 16;
      // a group past the end, or of masked keys alone (its scales may be anything)
      bool live = key0 < p.Nk;
      if constexpr (PAD)
        live = __any_sync(0xffffffffu, fmaxf(fmaxf(pad[0], pad[1]), fmaxf(pad[2], pad[3])) != -INFINITY);
      if (live) {
        const uint32_t kt = ring + uint32_t(i * 2 * C::TILE), vt = kt + uint32_t(C::TILE);
        const float lv = __log2f(vs);
        bad |= !(ks >= 0.f && ks < INFINITY && vs > 0.f && vs < INFINITY);
        lv_lo = fminf(lv_lo, lv);
        lv_hi = fmaxf(lv_hi, lv);
        float s[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t w[D / 16];
          const int r = warp * 16 + g + 8 * e;
          if constexpr (D == 96) {
#pragma unroll
            for (int c = 0; c < 3; ++c) lds_u64(kt + code_at<D>(r, t * 24 + c * 8), w[2 * c], w[2 * c + 1]);
          } else {
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              lds_u128(kt + code_at<D>(r, t * (D / 4) + c * 16), w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
          }
          s[e][0] = s[e][1] = s[e][2] = s[e][3] = 0.f;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint32_t x = bias_codes<E4M3>(w[c]);
            mma_16816(s[e], aq[c], widen_lo<E4M3>(x), widen_hi<E4M3>(x));
          }
        }
        // weights of rows g and g + 8, keys key0 + {2 t, 2 t + 1, 2 t + 8, 2 t + 9}
        float a[2][4];
        bool up = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float f = undo[r] * ks;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float raw = s[e >> 1][2 * r + (e & 1)];
            if constexpr (PAD) {
              a[r][e] = pad[e] == -INFINITY ? -INFINITY : fmaf(raw, f, pad_log2(pad[e]));
            } else {
              a[r][e] = raw * f;
              if (key0 + 16 > p.Nk && key0 + 2 * t + (e & 1) + 8 * (e >> 1) >= p.Nk) a[r][e] = -INFINITY;
            }
          }
          up |= fmaxf(fmaxf(a[r][0], a[r][1]), fmaxf(a[r][2], a[r][3])) + lv > m[r] + 8.f;
        }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float top = fmaxf(fmaxf(a[r][0], a[r][1]), fmaxf(a[r][2], a[r][3])) + lv;
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            if (top > m[r]) {
              const float al = ex2_approx(m[r] - top);  // 0 from m = -inf
              m[r] = top;
              l[r] *= al;
#pragma unroll
              for (int c = 0; c < NT; ++c) {
                o[c][2 * r] *= al;
                o[c][2 * r + 1] *= al;
              }
            }
          }
        }
        const float inv = ex2_approx(-lv);
        uint32_t ap[4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float mm = m[r] == -INFINITY ? 0.f : m[r];
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = ex2_approx((a[r][e] - mm) + lv);
          l[r] = fmaf((w[0] + w[1]) + (w[2] + w[3]), inv, l[r]);
          ap[r] = pack_f16x2(w[0], w[1]);
          ap[r + 2] = pack_f16x2(w[2], w[3]);
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
          if constexpr (PAD) {  // masked keys: zeros, whatever the codes (NaN) are
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
              if (pad[e] == -INFINITY) w[e][c] = 0u;
          }
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = bias_codes<E4M3>(w[e][c]);
          // bytes of keys (0, 1) and (2, 3) side by side, column by column
          const uint32_t a0 = __byte_perm(x[0], x[1], 0x5140), a1 = __byte_perm(x[0], x[1], 0x7362);
          const uint32_t b0 = __byte_perm(x[2], x[3], 0x5140), b1 = __byte_perm(x[2], x[3], 0x7362);
          mma_16816(o[4 * c], ap, widen_lo<E4M3>(a0), widen_lo<E4M3>(b0));
          mma_16816(o[4 * c + 1], ap, widen_hi<E4M3>(a0), widen_hi<E4M3>(b0));
          mma_16816(o[4 * c + 2], ap, widen_lo<E4M3>(a1), widen_lo<E4M3>(b1));
          mma_16816(o[4 * c + 3], ap, widen_hi<E4M3>(a1), widen_hi<E4M3>(b1));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&empty[i]));
    }
    if (bad) set_status(p.status, SAFEDIT_ERR_INVALID_ARG);
  }
  if (__syncthreads_or(!ok)) return;  // a wait ran out: reported, nothing is written

  // ---- the warps' results joined in shared memory
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    if (t == 0 && warp < kRowWarps) sm_m[warp][g + 8 * r] = m[r], sm_l[warp][g + 8 * r] = l[r];
  }
  if (lane == 0 && warp < kRowWarps) sm_range[warp][0] = lv_lo, sm_range[warp][1] = lv_hi;
  for (int e = threadIdx.x; e < 16 * D; e += kRowThreads8) (&sm_o[0][0])[e] = 0.f;
  __syncthreads();
  float mx[2], lx[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int rr = g + 8 * r;
    mx[r] = -INFINITY, lx[r] = 0.f;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) mx[r] = fmaxf(mx[r], sm_m[w][rr]);
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w)
      if (sm_m[w][rr] != -INFINITY) lx[r] = fmaf(ex2_approx(sm_m[w][rr] - mx[r]), sm_l[w][rr], lx[r]);
    m[r] = m[r] == -INFINITY ? 0.f : ex2_approx(m[r] - mx[r]);  // this warp's factor
  }
  for (int w = 0; w < kRowWarps; ++w) {  // one warp after another: the sum's order is fixed
    if (warp == w) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          sm_o[g + 8 * r][value_col<D>(2 * t, i)] += o[i][2 * r] * m[r];
          sm_o[g + 8 * r][value_col<D>(2 * t + 1, i)] += o[i][2 * r + 1] * m[r];
        }
    }
    __syncthreads();
  }
  for (int w = 0; w < kRowWarps; ++w) lv_lo = fminf(lv_lo, sm_range[w][0]), lv_hi = fmaxf(lv_hi, sm_range[w][1]);
  const int64_t rec = (int64_t(bh) * p.n_tiles + tile) * p.n_split + split;
  if (p.n_split > 1) {
    const PartView pv = part_view(p, rec, D);
    for (int e = threadIdx.x; e < p.tile_rows * D; e += kRowThreads8) pv.o[e] = (&sm_o[0][0])[e];
    if (warp == 0 && t == 0) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (g + 8 * r < p.tile_rows) pv.ml[(g + 8 * r) * 2] = mx[r], pv.ml[(g + 8 * r) * 2 + 1] = lx[r];
    }
    if (threadIdx.x == 0) pv.range[0] = lv_lo, pv.range[1] = lv_hi;
    return;
  }
  if (threadIdx.x == 0 && lv_hi - lv_lo > kScaleSpread) set_status(p.status, SAFEDIT_ERR_INVALID_ARG);
  if (warp == 0 && t == 0) {
#pragma unroll
    for (int r = 0; r < 2; ++r) sm_l[0][g + 8 * r] = lx[r], sm_m[0][g + 8 * r] = __int_as_float(my_q[r]);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 16 * D / 2; e += kRowThreads8) {
    const int rr = e / (D / 2), c = (e - rr * (D / 2)) * 2;
    const int qi = __float_as_int(sm_m[0][rr]);
    if (qi < 0) continue;
    const float ls = sm_l[0][rr];
    if (ls == 0.f && c == 0) set_status(p.status, SAFEDIT_ERR_MASKED_ROW);
    const float inv = ls == 0.f ? 0.f : 1.f / ls;
    const int64_t orow = p.out_scattered ? int64_t(qi) : int64_t(tile * 16 + rr);
    *reinterpret_cast<uint32_t*>(p.out + b * p.o_sb + h * p.o_sh + orow * p.o_sr + c) =
        pack_bf16x2(sm_o[rr][c] * inv, sm_o[rr][c + 1] * inv);
  }
}

// ------------------------------------------------------------- parts joined
// One CTA for each query row: m = max m_i, out = sum 2^(m_i - m) O_i /
// sum 2^(m_i - m) l_i over the row's parts, in their order.
template <int D>
__global__ void __launch_bounds__(D) attn_state8_join_kernel(const __grid_constant__ State8Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = threadIdx.x;
  const int pu = blockIdx.x / p.tile_rows, rr = blockIdx.x - pu * p.tile_rows;
  const int unit = p.n_full + pu;
  const int bh = unit / p.n_tiles, r = (unit - bh * p.n_tiles) * p.unit_rows + rr;
  if (r >= p.n_rows) return;
  const int b = bh / p.H, h = bh - b * p.H;
  const int qi = p.idx ? __ldg(p.idx + r) : r;
  if (qi < 0 || qi >= p.Nq) return;  // reported by the attention kernel
  const int64_t rec0 = int64_t(pu) * p.n_split;
  float m = -INFINITY, lv_lo = INFINITY, lv_hi = -INFINITY;
  for (int s = 0; s < p.n_split; ++s) {
    const PartView v = part_view(p, rec0 + s, D);
    m = fmaxf(m, v.ml[rr * 2]);
    lv_lo = fminf(lv_lo, v.range[0]), lv_hi = fmaxf(lv_hi, v.range[1]);
  }
  float l = 0.f, acc = 0.f;
#pragma unroll 4
  for (int s = 0; s < p.n_split; ++s) {
    const PartView v = part_view(p, rec0 + s, D);
    const float ms = v.ml[rr * 2];
    const float w = ms == -INFINITY ? 0.f : ex2_approx(ms - m);
    l = fmaf(w, v.ml[rr * 2 + 1], l);
    if (w != 0.f) acc = fmaf(w, v.o[rr * D + c], acc);
  }
  if (c == 0) {
    if (lv_hi - lv_lo > kScaleSpread) set_status(p.status, SAFEDIT_ERR_INVALID_ARG);
    if (l == 0.f) set_status(p.status, SAFEDIT_ERR_MASKED_ROW);
  }
  const int64_t orow = p.out_scattered ? int64_t(qi) : int64_t(r);
  p.out[b * p.o_sb + h * p.o_sh + orow * p.o_sr + c] = __float2bfloat16_rn(l == 0.f ? 0.f : acc / l);
}

// ------------------------------------------------------------- plan
struct State8Plan {
  bool tc = false;
  int unit_rows = 16, tile_rows = 16, n_tiles = 0, n_full = 0, n_split = 1;
  int64_t n_parts = 0;  // units that run in parts
  size_t ws_bytes = 0;
};

static int state8_sms() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
    sms = 148;
  return sms;
}

// Rows of a slice up to which the warp-level kernel is taken.
constexpr int64_t kFewRows = 16;

static State8Plan plan_state8(int64_t n_rows, int64_t BH, int64_t Nk, int D, int sms) {
  State8Plan pl;
  pl.tc = n_rows > kFewRows;
  pl.unit_rows = pl.tc ? 256 : 16;
  pl.tile_rows = n_rows < pl.unit_rows ? int(n_rows) : pl.unit_rows;
  pl.n_tiles = int((n_rows + pl.unit_rows - 1) / pl.unit_rows);
  const int64_t units = pl.n_tiles * BH;
  if (units == 0) return pl;
  if (!pl.tc) {
    // one wave of what an SM holds, each part two stages of keys at least
    int64_t split = int64_t(sms) * (D == 64 ? RowsCfg<64>::CTAS : RowsCfg<96>::CTAS) / units;
    const int64_t most = (Nk + 2 * kStageKeys - 1) / (2 * kStageKeys);
    if (split > most) split = most;
    pl.n_split = split > 1 ? int(split) : 1;
    pl.n_parts = split > 1 ? units : 0;
  } else {
    // The units that do not fill a wave of the SMs run as 2..16 parts over
    // the key tiles where that ends the call sooner: a CTA costs about
    // kFixedUs and kTileUs a key tile of 128, the join kJoinUs.
    constexpr double kFixedUs = 9.0, kTileUs = 1.9, kJoinUs = 5.0;
    const int64_t nk = (Nk + 127) / 128, tail = units % sms;
    const double tile_us = kTileUs * (D + 32) / 128.0;
    double best = kFixedUs + double(nk) * tile_us;
    for (int s = 2; tail > 0 && s <= 16 && s <= nk; ++s) {
      const double rounds = double((tail * s + sms - 1) / sms);
      const double cost = rounds * (kFixedUs + double((nk + s - 1) / s) * tile_us) + kJoinUs;
      if (cost < best) {
        best = cost;
        pl.n_split = s;
      }
    }
    pl.n_parts = pl.n_split > 1 ? tail : 0;
  }
  pl.n_full = int(units - pl.n_parts);
  if (pl.n_parts) pl.ws_bytes = part_floats(pl.n_parts * pl.n_split, pl.tile_rows, D) * sizeof(float);
  return pl;
}

template <int D>
static safedit_status launch_join(const State8Params& p, int64_t n_parts, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(n_parts * p.tile_rows));
  cfg.blockDim = dim3(D);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, attn_state8_join_kernel<D>, p) != cudaSuccess) return SAFEDIT_ERR_CUDA;
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
  auto kern = attn_state8_rows_kernel<D, PAD, E4M3>;
  const safedit_status st = set_smem(reinterpret_cast<const void*>(kern), RowsCfg<D>::SMEM);
  if (st != SAFEDIT_OK) return st;
  const dim3 grid{unsigned(p.n_split), unsigned(p.n_tiles), unsigned(BH)};
  kern<<<grid, kRowThreads8, RowsCfg<D>::SMEM, s>>>(tmK, tmV, p);
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
  return launch_join<D>(p, pl.n_parts, s);
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
  p.n_records = pl.n_parts * pl.n_split;
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
