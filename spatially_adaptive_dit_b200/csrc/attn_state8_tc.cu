// attn_state8_tc.cu -- attention of many query rows over an 8-bit state, on
// the fifth-generation tensor cores.
//
// One CTA per SM, 512 threads = 4 warpgroups, 256 query rows (two tiles of
// 128) of one (b, h) slice against a range of the keys:
//   * warpgroups 0 and 1: the softmax of one tile each, thread = query row =
//     TMEM lane.  They first gather their rows, scale them to f16 and lay them
//     out for the tensor core.
//   * warpgroup 2: warp 8 streams the codes of K and V by TMA (128 keys a
//     tile) into a ring; warp 9 issues tcgen05.mma.
//   * warpgroup 3 widens codes to f16 into the swizzled tiles that the tensor
//     core reads (the tensor core has no product of a 16-bit and an 8-bit
//     operand, and 8-bit queries or weights would lose what the state keeps),
//     and computes each tile's scale factors and pads.
//   * S_t = Q_t K_j^T into TMEM (fp32), weights back into TMEM as f16 in place
//     of S_t, O_t += W_t V_j; issue order per key tile W V_0(j), Q K_0(j+1),
//     W V_1(j), Q K_1(j+1), so one tile's softmax overlaps the other's MMAs.
//   * online softmax in base 2 with a lazy rescale (by more than 2^8), scales
//     of 16 keys at a time folded into the factor and offset of the exponent.
// Key tiles whose pads are all -inf are skipped by every role.  Every wait is
// bounded; an expired one raises the CTA's abort flag, drains what is in
// flight, frees TMEM and returns.
#include "attn_state8.cuh"

namespace sd {

template <int D>
struct TcCfg {
  static constexpr int BN = 128;                       // keys per tile
  static constexpr int CH = (D % 64 == 0) ? 64 : 32;   // f16 elements per swizzle chunk row
  static constexpr int NCH = D / CH;
  static constexpr int ROWB = CH * 2;
  static constexpr uint32_t LAYOUT = (CH == 64) ? 2u : 4u;  // 128B / 64B swizzle
  static constexpr int CHUNK_BYTES = 128 * ROWB;
  static constexpr int TILE_BYTES = NCH * CHUNK_BYTES;  // 128 rows of f16
  static constexpr int RAW_BYTES = 128 * D;             // 128 rows of codes
  static constexpr int NS = D == 128 ? 2 : 3;           // widened K (and V) tiles
  static constexpr int NR = 2;                          // raw tiles, K and V in turn
  static constexpr int NF = NS + 1;                     // slots of scale factors and pads, see below
  static constexpr int LIVE_WORDS = D == 128 ? 8 : 32;  // key tiles / 32 that can be skipped
  static constexpr int OFF_K = 2 * TILE_BYTES;
  static constexpr int OFF_V = OFF_K + NS * TILE_BYTES;
  static constexpr int OFF_RAW = OFF_V + NS * TILE_BYTES;
  static constexpr int OFF_BAR = OFF_RAW + NR * RAW_BYTES;
  static constexpr int N_BARS = 2 + 4 * NS + 2 * NR + 2 + 2 + 2;
  static constexpr int OFF_FACT = OFF_BAR + ((N_BARS * 8 + 8 + 15) / 16) * 16;
  static constexpr int OFF_PAD = OFF_FACT + ((NF * 8 * 12 + 15) / 16) * 16;
  static constexpr int OFF_LIVE = OFF_PAD + NF * 128 * 4;
  static constexpr int SMEM_PLAIN = 1024 + OFF_PAD;
  static constexpr int SMEM_PAD = 1024 + OFF_LIVE + LIVE_WORDS * 4;
  static_assert(SMEM_PAD <= 232448, "shared memory");
  static_assert(256 + 2 * D <= 512, "TMEM columns");
};

constexpr int kTcThreads = 512;
// 256 * 184 + 128 * 72 + 128 * 72 = 512 * 128
constexpr uint32_t kTcSoftmaxRegs = 184, kTcControlRegs = 72, kTcWidenRegs = 72;
static_assert(256 * kTcSoftmaxRegs + 128 * kTcControlRegs + 128 * kTcWidenRegs <= 512 * 128, "register split");
constexpr uint64_t kTcDrainNs = 1000000000ull;
// Pairs of columns (bit e of 16) whose exponentials go to the FMA pipe.
constexpr uint32_t kTcFmaPairs = 0x8888u;

__device__ __forceinline__ uint32_t tc_swizzle(uint32_t off, uint32_t layout) {
  return layout == 2u ? (off ^ (((off >> 7) & 7u) << 4)) : (off ^ (((off >> 7) & 3u) << 4));
}

__device__ __forceinline__ void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ float lds32(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ void sts32(uint32_t at, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

// Instruction descriptor of kind::f16 with f16 A and B, fp32 accumulate.
constexpr uint32_t idesc_f16_f32(int M, int N, int b_mn_major) {
  return (1u << 4) | (uint32_t(b_mn_major) << 16) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

// Waits for this warp's TMEM loads and names the registers of one of them, so
// that no use of it moves before the wait.
__device__ __forceinline__ void tmem_landed(float (&x)[32]) {
  tmem_wait_ld();
#pragma unroll
  for (int e = 0; e < 32; ++e) asm volatile("" : "+f"(x[e]));
}

template <int D, bool PAD, bool E4M3>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_state8_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ State8Params p) {
  using C = TcCfg<D>;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  auto BAR = [&](int i) { return sb + uint32_t(C::OFF_BAR) + 8u * uint32_t(i); };
  constexpr int Q_FULL = 0, K_FULL = 2, K_EMPTY = K_FULL + C::NS, V_FULL = K_EMPTY + C::NS, V_EMPTY = V_FULL + C::NS,
                RAW_FULL = V_EMPTY + C::NS, RAW_EMPTY = RAW_FULL + C::NR, S_FULL = RAW_EMPTY + C::NR,
                P_FULL = S_FULL + 2, O_FULL = P_FULL + 2, DRAIN = O_FULL + 1;
  static_assert(DRAIN + 1 == C::N_BARS, "barriers");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::N_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // CTAs below n_full take whole units; the others part (i % n_split) of unit
  // n_full + i / n_split
  const bool whole = int(blockIdx.x) < p.n_full;
  const int rest = int(blockIdx.x) - p.n_full;
  const int unit = whole ? int(blockIdx.x) : p.n_full + rest / p.n_split;
  const int part = whole ? 0 : rest % p.n_split;
  const int bh = unit / p.n_tiles;
  const int b = bh / p.H, h = bh - b * p.H;
  const int row0 = (unit - bh * p.n_tiles) * 256;
  const bool two = row0 + 128 < p.n_rows;  // the second tile has rows
  const int nk = (p.Nk + C::BN - 1) / C::BN;
  const int k_lo = whole ? 0 : int(int64_t(nk) * part / p.n_split);
  const int k_hi = whole ? nk : int(int64_t(nk) * (part + 1) / p.n_split);

  // live key tiles: one whose pads are all -inf carries no weight
  const uint32_t live_s = sb + uint32_t(C::OFF_LIVE);
  const bool skip_tiles = PAD && nk <= C::LIVE_WORDS * 32;
  if constexpr (PAD) {
    uint32_t* live_bits = reinterpret_cast<uint32_t*>(smem + C::OFF_LIVE);
    if (threadIdx.x < C::LIVE_WORDS) live_bits[threadIdx.x] = 0u;
    __syncthreads();
    if (skip_tiles) {
      const float* pr = p.pad + b * p.pad_sb;
      for (int j = k_lo + warp; j < k_hi; j += kTcThreads / 32) {
        bool live = false;
        for (int c = lane; c < C::BN && j * C::BN + c < p.Nk; c += 32)
          live |= !(__ldg(pr + j * C::BN + c) == -INFINITY);
        if (__any_sync(0xffffffffu, live) && lane == 0) atomicOr(live_bits + (j >> 5), 1u << (j & 31));
      }
    }
  }
  auto live_word = [&](int w) -> uint32_t { return __float_as_uint(lds32(live_s + uint32_t(w) * 4u)); };
  // first live tile at or after j (k_hi if none)
  auto next_live = [&](int j) -> int {
    if constexpr (PAD) {
      while (skip_tiles && j < k_hi) {
        const uint32_t w = live_word(j >> 5) >> (j & 31);
        if (w) return j + __ffs(w) - 1;
        j = (j | 31) + 1;
      }
    }
    return j;
  };
  auto live_count = [&]() -> int {  // bits are set inside [k_lo, k_hi) alone
    int n = k_hi - k_lo;
    if constexpr (PAD) {
      if (skip_tiles) {
        n = 0;
        for (int w = 0; w < C::LIVE_WORDS; ++w) n += __popc(live_word(w));
      }
    }
    return n;
  };

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(BAR(Q_FULL + t), 128);
      mbar_init(BAR(S_FULL + t), 1);
      mbar_init(BAR(P_FULL + t), 128);
    }
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(BAR(K_FULL + s), 128);
      mbar_init(BAR(K_EMPTY + s), 1);
      mbar_init(BAR(V_FULL + s), 128);
      mbar_init(BAR(V_EMPTY + s), 1);
    }
    for (int s = 0; s < C::NR; ++s) {
      mbar_init(BAR(RAW_FULL + s), 1);
      mbar_init(BAR(RAW_EMPTY + s), 128);
    }
    mbar_init(BAR(O_FULL), 1);
    mbar_init(BAR(DRAIN), 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == 9 && lane == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl ctl{abort_flag, p.status, p.wait_limit};

  if (warp < 8) {
    // ================================================== softmax warpgroups
    setmaxnreg_inc<kTcSoftmaxRegs>();
    const int t = warp >> 2;
    const int tid = threadIdx.x & 127;
    const int my_row = row0 + t * 128 + tid;
    if (t == 0 || two) {
      int my_q = -1;
      if (my_row < p.n_rows) {
        my_q = p.idx ? __ldg(p.idx + my_row) : my_row;
        if (my_q < 0 || my_q >= p.Nq) {
          set_status(p.status, SAFEDIT_ERR_INDEX);
          my_q = -1;
        }
      }
      // ---- this thread's query row: largest magnitude, factor to f16, the
      // swizzled K-major layout
      float undo;
      {
        uint32_t w[D / 2];
#pragma unroll
        for (int c = 0; c < D / 2; ++c) w[c] = 0u;
        if (my_q >= 0) {
          const uint4* src =
              reinterpret_cast<const uint4*>(p.q + b * p.q_sb + h * p.q_sh + int64_t(my_q) * p.q_sr);
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            const uint4 v = __ldg(src + c);
            w[4 * c] = v.x, w[4 * c + 1] = v.y, w[4 * c + 2] = v.z, w[4 * c + 3] = v.w;
          }
        }
        uint32_t m = 0u;
#pragma unroll
        for (int c = 0; c < D / 2; ++c) m = max(m, max((w[c] << 16) & 0x7FFF0000u, w[c] & 0x7FFF0000u));
        const float f = query_factor(m, p.scale_log2, undo);
        const uint32_t qs = sb + uint32_t(t * C::TILE_BYTES);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[e] = pack_f16x2(__uint_as_float(w[4 * c + e] << 16) * f, __uint_as_float(w[4 * c + e] & 0xFFFF0000u) * f);
          const uint32_t off = uint32_t((c * 8 / C::CH) * C::CHUNK_BYTES) +
                               tc_swizzle(uint32_t(tid * C::ROWB + (c * 8 % C::CH) * 2), C::LAYOUT);
          sts128(qs + off, o[0], o[1], o[2], o[3]);
        }
        fence_proxy_async_smem();
        mbar_arrive(BAR(Q_FULL + t));
      }

      const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
      const uint32_t tS = tmem + uint32_t(t * 128) + lane_base;
      const uint32_t tO = tmem + 256u + uint32_t(t * D) + lane_base;
      float m_run = -INFINITY, l_run = 0.f;
      bool ok = true;
      const int n_live = live_count();
      int j = next_live(k_lo), slot = 0;
      for (int it = 0; it < n_live; ++it) {
        if (!wait_warp(BAR(S_FULL + t), uint32_t(it & 1), ctl)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // factors of the tile's eight groups of 16 keys: ks, log2 vs, 1 / vs
        const uint32_t fact = sb + uint32_t(C::OFF_FACT + slot * 96);
        const uint32_t pads = sb + uint32_t(C::OFF_PAD + slot * 512);
        const int lim = p.Nk - j * C::BN;
        const bool ragged = !PAD && lim < C::BN;
        // columns 32 c .. 32 c + 31: with pads, or past the last key, the raw
        // scores become exponents undo ks x + pad here
        auto shape = [&](int c, float (&x)[32]) {
          if (PAD || ragged) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float kf = undo * lds32(fact + uint32_t(((32 * c + e) / 16) * 4));
              if constexpr (PAD) {
                const uint4 pd = lds128(pads + uint32_t((32 * c + e) * 4));
                x[e] = fmaf(x[e], kf, __uint_as_float(pd.x));
                x[e + 1] = fmaf(x[e + 1], kf, __uint_as_float(pd.y));
                x[e + 2] = fmaf(x[e + 2], kf, __uint_as_float(pd.z));
                x[e + 3] = fmaf(x[e + 3], kf, __uint_as_float(pd.w));
              } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) x[e + k] = 32 * c + e + k < lim ? x[e + k] * kf : -INFINITY;
              }
            }
          }
        };
        float mt = -INFINITY;
        auto take_max = [&](int c, const float (&x)[32]) {
#pragma unroll
          for (int gg = 0; gg < 2; ++gg) {
            const float* y = x + 16 * gg;
            const int g = 2 * c + gg;
            float m0 = max3(y[0], y[1], y[2]), m1 = max3(y[3], y[4], y[5]);
            m0 = max3(m0, y[6], y[7]), m1 = max3(m1, y[8], y[9]);
            m0 = max3(m0, y[10], y[11]), m1 = max3(m1, y[12], y[13]);
            m0 = max3(m0, y[14], y[15]);
            m0 = fmaxf(m0, m1);
            const float lv = lds32(fact + uint32_t(32 + g * 4));
            const float kf = PAD || ragged ? 1.f : undo * lds32(fact + uint32_t(g * 4));
            mt = fmaxf(mt, fmaf(m0, kf, lv));
          }
        };
        // The maximum needs all 128 columns before the first weight; half of
        // them stay in registers, the others are read from TMEM again.
        float x0[32], x1[32], x2[32];
        auto load = [&](int c, float (&x)[32]) {
          uint32_t r[32];
          tmem_ld32(tS + uint32_t(c * 32), r);
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(r[e]);
        };
        load(2, x0);
        load(3, x1);
        tmem_landed(x0);
        tmem_landed(x1);
        shape(2, x0);
        take_max(2, x0);
        shape(3, x1);
        take_max(3, x1);
        load(0, x0);
        load(1, x1);
        tmem_landed(x0);
        tmem_landed(x1);
        load(2, x2);
        shape(0, x0);
        take_max(0, x0);
        shape(1, x1);
        take_max(1, x1);
        bool need_o = false;
        float alpha = 1.f;
        if (mt > m_run + 8.f) {
          alpha = ex2_approx(m_run - mt);  // 0 from m = -inf
          l_run *= alpha;
          m_run = mt;
          need_o = it > 0;
        }
        if (__any_sync(0xffffffffu, need_o)) {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t r[16];
            tmem_ld16(tO + uint32_t(c * 16), r);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
            tmem_st16(tO + uint32_t(c * 16), r);
          }
        }
        const float neg_m = m_run == -INFINITY ? 0.f : -m_run;
        const uint64_t negm2 = f2_pack(neg_m, neg_m);
        auto emit = [&](int c, const float (&x)[32]) {
          uint32_t pk[16];
#pragma unroll
          for (int gg = 0; gg < 2; ++gg) {
            const int g = 2 * c + gg;
            const float lv = lds32(fact + uint32_t(32 + g * 4)), inv = lds32(fact + uint32_t(64 + g * 4));
            const float kf = PAD || ragged ? 1.f : undo * lds32(fact + uint32_t(g * 4));
            const float off = lv + neg_m;
            const uint64_t kf2 = f2_pack(kf, kf), off2 = f2_pack(off, off), lv2 = f2_pack(lv, lv);
            uint64_t s0 = f2_pack(0.f, 0.f), s1 = s0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint64_t xx = f2_pack(x[16 * gg + 2 * e], x[16 * gg + 2 * e + 1]);
              // with pads the difference to the maximum comes first: a pad of
              // the type's lowest value absorbs everything added to it
              const uint64_t a2 = PAD ? f2_add(f2_add(xx, negm2), lv2) : f2_fma(xx, kf2, off2);
              float a0, a1, p0, p1;
              f2_unpack(a2, a0, a1);
              if (!PAD && ((kTcFmaPairs >> (8 * gg + e)) & 1u)) {
                exp2_pair_fma(a0, a1, p0, p1);
              } else {
                p0 = ex2_approx(a0);
                p1 = ex2_approx(a1);
              }
              if (e & 1)
                s1 = f2_add(s1, f2_pack(p0, p1));
              else
                s0 = f2_add(s0, f2_pack(p0, p1));
              pk[8 * gg + e] = pack_f16x2(p0, p1);
            }
            float u0, u1;
            f2_unpack(f2_add(s0, s1), u0, u1);
            l_run = fmaf(u0 + u1, inv, l_run);
          }
          tmem_st16(tS + uint32_t(c * 16), pk);
        };
        // weights of columns 32 c.. land in columns 16 c.. : behind the reads
        emit(0, x0);
        load(3, x0);
        emit(1, x1);
        tmem_landed(x2);
        tmem_landed(x0);
        shape(2, x2);
        emit(2, x2);
        shape(3, x0);
        emit(3, x0);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(BAR(P_FULL + t));
        j = next_live(j + 1);
        slot = slot + 1 == C::NF ? 0 : slot + 1;
      }
      // ---- epilogue: O / l -> bf16 rows, or the part's record
      if (ok && wait_warp(BAR(O_FULL), 0u, ctl)) {
        tc_fence_after();
        const bool live = my_q >= 0;
        const bool empty = n_live == 0;  // O was never written
        if (live && whole && l_run == 0.f) set_status(p.status, SAFEDIT_ERR_MASKED_ROW);
        const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
        float* po = nullptr;
        __nv_bfloat16* orow = nullptr;
        if (whole) {
          const int64_t at = p.out_scattered ? int64_t(my_q) : int64_t(my_row);
          orow = p.out + b * p.o_sb + h * p.o_sh + at * p.o_sr;
        } else {
          const PartView pv = part_view(p, rest, D);
          const int rr = t * 128 + tid;
          po = pv.o + int64_t(rr) * D;
          if (live) {
            pv.ml[rr * 2] = m_run;
            pv.ml[rr * 2 + 1] = l_run;
          }
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t r[32];
          tmem_ld32(tO + uint32_t(c * 32), r);
          tmem_wait_ld();
          if (!live) continue;
          if (l_run == 0.f || empty) {
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = 0u;
          }
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(orow + c * 32);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t o[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                o[k] = pack_bf16x2(__uint_as_float(r[8 * e + 2 * k]) * inv, __uint_as_float(r[8 * e + 2 * k + 1]) * inv);
              dst[e] = make_uint4(o[0], o[1], o[2], o[3]);
            }
          } else {
            uint4* dst = reinterpret_cast<uint4*>(po + c * 32);
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[e] = make_uint4(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
          }
        }
      }
    }
  } else if (warp < 12) {
    setmaxnreg_dec<kTcControlRegs>();
    if (warp == 8) {
      // ================================================ TMA producer (codes)
      if (lane == 0) {
        int issued = 0;
        const int n_live = live_count();
        for (int it = 0, kt = next_live(k_lo); it < n_live; ++it, kt = next_live(kt + 1)) {
          bool ok = true;
          for (int kv = 0; kv < 2; ++kv) {
            const int s = issued % C::NR;
            if (!(ok = wait_bounded(BAR(RAW_EMPTY + s), uint32_t(((issued / C::NR) & 1) ^ 1), ctl))) break;
            mbar_arrive_expect_tx(BAR(RAW_FULL + s), C::RAW_BYTES);
            tma_load_4d(sb + uint32_t(C::OFF_RAW + s * C::RAW_BYTES), kv ? &tmV : &tmK, BAR(RAW_FULL + s), 0,
                        kt * C::BN, h, b);
            ++issued;
          }
          if (!ok) break;
        }
        // every copy has landed before the CTA leaves
        for (int i = issued > C::NR ? issued - C::NR : 0; i < issued; ++i)
          wait_drain(BAR(RAW_FULL + i % C::NR), uint32_t((i / C::NR) & 1), kTcDrainNs);
      }
    } else if (warp == 9) {
      // ================================================ MMA issuer
      if (lane == 0) {
        constexpr uint32_t idesc_qk = idesc_f16_f32(128, 128, 0), idesc_pv = idesc_f16_f32(128, D, 1);
        constexpr uint32_t SBO = 8u * C::ROWB;
        const uint64_t qd0 = smem_desc(sb, 16u, SBO, C::LAYOUT);
        const uint64_t kd0 = smem_desc(sb + C::OFF_K, 16u, SBO, C::LAYOUT);
        const uint64_t vd0 = smem_desc(sb + C::OFF_V, uint32_t(C::CHUNK_BYTES), SBO, C::LAYOUT);
        auto adv = [](uint64_t d, uint32_t bytes) {
          return (d & 0xFFFFFFFF00000000ull) | uint64_t(uint32_t(d) + (bytes >> 4));
        };
        auto issue_qk = [&](int t, int s) {
          const uint64_t qd = adv(qd0, uint32_t(t * C::TILE_BYTES)), kd = adv(kd0, uint32_t(s * C::TILE_BYTES));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = uint32_t(((kk * 16) / C::CH) * C::CHUNK_BYTES + ((kk * 16) % C::CH) * 2);
            mma_ss(tmem + uint32_t(t * 128), adv(qd, off), adv(kd, off), idesc_qk, kk > 0 ? 1u : 0u);
          }
          tc_commit(BAR(S_FULL + t));
        };
        auto issue_pv = [&](int t, int s, bool acc) {
          const uint64_t vd = adv(vd0, uint32_t(s * C::TILE_BYTES));
#pragma unroll
          for (int kk = 0; kk < C::BN / 16; ++kk)
            mma_ts(tmem + 256u + uint32_t(t * D), tmem + uint32_t(t * 128 + kk * 8), adv(vd, uint32_t(kk * 16 * C::ROWB)),
                   idesc_pv, (acc || kk > 0) ? 1u : 0u);
        };
        const int n_live = live_count();
        bool ok = wait_bounded(BAR(Q_FULL), 0u, ctl) && (!two || wait_bounded(BAR(Q_FULL + 1), 0u, ctl)) &&
                  (n_live == 0 || wait_bounded(BAR(K_FULL), 0u, ctl));
        if (ok && n_live > 0) {
          tc_fence_after();
          issue_qk(0, 0);
          if (two) issue_qk(1, 0);
          tc_commit(BAR(K_EMPTY));
        }
        for (int j = 0; ok && j < n_live; ++j) {
          const int s = j % C::NS, s1 = (j + 1) % C::NS;
          const bool more = j + 1 < n_live;
          if (!(ok = wait_bounded(BAR(V_FULL + s), uint32_t((j / C::NS) & 1), ctl))) break;
          if (!(ok = wait_bounded(BAR(P_FULL), uint32_t(j & 1), ctl))) break;
          tc_fence_after();
          issue_pv(0, s, j > 0);
          if (more) {
            if (!(ok = wait_bounded(BAR(K_FULL + s1), uint32_t(((j + 1) / C::NS) & 1), ctl))) break;
            tc_fence_after();
            issue_qk(0, s1);
          }
          if (two) {
            if (!(ok = wait_bounded(BAR(P_FULL + 1), uint32_t(j & 1), ctl))) break;
            tc_fence_after();
            issue_pv(1, s, j > 0);
          }
          tc_commit(BAR(V_EMPTY + s));
          if (more) {
            if (two) issue_qk(1, s1);
            tc_commit(BAR(K_EMPTY + s1));
          }
        }
        if (ok) tc_commit(BAR(O_FULL));
        // every MMA has completed before TMEM is freed, whoever aborted
        tc_commit(BAR(DRAIN));
        wait_drain(BAR(DRAIN), 0u, kTcDrainNs);
      }
    }
  } else {
    // ================================================ widening of the codes
    setmaxnreg_dec<kTcWidenRegs>();
    const int tid = threadIdx.x - 384;
    const float* padb = PAD ? p.pad + b * p.pad_sb : nullptr;
    const float* ksb = p.ks + b * p.ks_sb + h * p.ks_sh;
    const float* vsb = p.vs + b * p.vs_sb + h * p.vs_sh;
    constexpr int UPR = D / 16;  // 16-code units per row
    float lv_lo = INFINITY, lv_hi = -INFINITY;
    // raw tile -> f16 tile.  A unit becomes two 16-byte pieces; lanes of the
    // row's second chunk write theirs in the other order, which keeps eight
    // lanes on different banks.
    auto widen = [&](uint32_t raw, uint32_t to, int key0) {
#pragma unroll
      for (int i = 0; i < UPR; ++i) {
        const int u = tid + i * 128;
        const int r = u / UPR, c = u - r * UPR;
        uint4 v = lds128(raw + uint32_t(u * 16));
        if constexpr (PAD) {  // masked keys: zeros, whatever the codes (NaN) are
          const int key = key0 + r;
          if (key < p.Nk && __ldg(padb + key) == -INFINITY) v = make_uint4(0u, 0u, 0u, 0u);
        }
        uint32_t w[4] = {v.x, v.y, v.z, v.w}, o[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t x = bias_codes<E4M3>(w[e]);
          o[2 * e] = widen_lo<E4M3>(x);
          o[2 * e + 1] = widen_hi<E4M3>(x);
        }
        const int chunk = c * 16 / C::CH;
        const uint32_t row = uint32_t(r * C::ROWB + (c * 16 % C::CH) * 2);
        const uint32_t base = to + uint32_t(chunk * C::CHUNK_BYTES);
        const uint32_t a0 = base + tc_swizzle(row, C::LAYOUT), a1 = base + tc_swizzle(row + 16u, C::LAYOUT);
        if (chunk & 1) {
          sts128(a1, o[4], o[5], o[6], o[7]);
          sts128(a0, o[0], o[1], o[2], o[3]);
        } else {
          sts128(a0, o[0], o[1], o[2], o[3]);
          sts128(a1, o[4], o[5], o[6], o[7]);
        }
      }
    };
    const int n_live = live_count();
    int slot = 0;
    for (int it = 0, kt = next_live(k_lo); it < n_live; ++it, kt = next_live(kt + 1)) {
      const int s = it % C::NS;
      const uint32_t ph = uint32_t((it / C::NS) & 1) ^ 1u;
      const int key0 = kt * C::BN;
      int n = 2 * it;
      if (!wait_warp(BAR(RAW_FULL + n % C::NR), uint32_t((n / C::NR) & 1), ctl)) break;
      if (!wait_warp(BAR(K_EMPTY + s), ph, ctl)) break;
      // Scale factors and pads of the tile, NS + 1 slots: when the K tile
      // `it - NS` is free, its scores are done, which took the weights of
      // tile `it - NS - 1` from both query tiles, so nobody reads a slot
      // older than `it - NS`.
      if (tid < 8) {
        const int key = key0 + tid * 16;
        float ks = 0.f, lv = 0.f;
        if (key < p.Nk) {
          ks = __ldg(ksb + (key >> p.block_log2));
          const float vs = __ldg(vsb + (key >> p.block_log2));
          lv = __log2f(vs);
          bool used = true;  // a key of the group that is not masked
          if (!(ks >= 0.f && ks < INFINITY && vs > 0.f && vs < INFINITY)) {
            if constexpr (PAD) {
              used = false;
              for (int e = 0; e < 16 && key + e < p.Nk; ++e) used |= __ldg(padb + key + e) != -INFINITY;
            }
            if (used) set_status(p.status, SAFEDIT_ERR_INVALID_ARG);
            else ks = 0.f, lv = 0.f;
          } else {
            lv_lo = fminf(lv_lo, lv);
            lv_hi = fmaxf(lv_hi, lv);
          }
        }
        const uint32_t f = sb + uint32_t(C::OFF_FACT + slot * 96 + tid * 4);
        sts32(f, ks);
        sts32(f + 32u, lv);
        sts32(f + 64u, ex2_approx(-lv));
      }
      if constexpr (PAD)
        sts32(sb + uint32_t(C::OFF_PAD + slot * 512 + tid * 4),
              key0 + tid < p.Nk ? pad_log2(__ldg(padb + key0 + tid)) : -INFINITY);
      widen(sb + uint32_t(C::OFF_RAW + (n % C::NR) * C::RAW_BYTES), sb + uint32_t(C::OFF_K + s * C::TILE_BYTES), key0);
      mbar_arrive(BAR(RAW_EMPTY + n % C::NR));
      fence_proxy_async_smem();
      mbar_arrive(BAR(K_FULL + s));
      ++n;
      if (!wait_warp(BAR(RAW_FULL + n % C::NR), uint32_t((n / C::NR) & 1), ctl)) break;
      if (!wait_warp(BAR(V_EMPTY + s), ph, ctl)) break;
      widen(sb + uint32_t(C::OFF_RAW + (n % C::NR) * C::RAW_BYTES), sb + uint32_t(C::OFF_V + s * C::TILE_BYTES), key0);
      mbar_arrive(BAR(RAW_EMPTY + n % C::NR));
      fence_proxy_async_smem();
      mbar_arrive(BAR(V_FULL + s));
      slot = slot + 1 == C::NF ? 0 : slot + 1;
    }
    if (warp == 12) {
#pragma unroll
      for (int e = 1; e < 8; e <<= 1) {
        lv_lo = fminf(lv_lo, __shfl_xor_sync(0xffffffffu, lv_lo, e));
        lv_hi = fmaxf(lv_hi, __shfl_xor_sync(0xffffffffu, lv_hi, e));
      }
      if (lane == 0) {
        if (whole) {
          if (lv_hi - lv_lo > kScaleSpread) set_status(p.status, SAFEDIT_ERR_INVALID_ARG);
        } else {
          const PartView pv = part_view(p, rest, D);
          pv.range[0] = lv_lo;
          pv.range[1] = lv_hi;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool PAD, bool E4M3>
static safedit_status launch_tc(const CUtensorMap& tmK, const CUtensorMap& tmV, const State8Params& p, int64_t ctas,
                                cudaStream_t s) {
  auto kern = attn_state8_tc_kernel<D, PAD, E4M3>;
  constexpr int bytes = PAD ? TcCfg<D>::SMEM_PAD : TcCfg<D>::SMEM_PLAIN;
  const safedit_status st = set_smem(reinterpret_cast<const void*>(kern), bytes);
  if (st != SAFEDIT_OK) return st;
  kern<<<unsigned(ctas), kTcThreads, bytes, s>>>(tmK, tmV, p);
  return after_launch(1);
}

static safedit_status codes_map(CUtensorMap* m, const safedit_tensor* t) {
  const uint64_t dims[4] = {uint64_t(t->dims[3]), uint64_t(t->dims[2]), uint64_t(t->dims[1]), uint64_t(t->dims[0])};
  const uint64_t strides[3] = {uint64_t(t->strides[2]), uint64_t(t->strides[1]), uint64_t(t->strides[0])};
  const uint32_t box[4] = {uint32_t(t->dims[3]), 128u, 1u, 1u};
  return encode_tmap(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, t->data, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

safedit_status launch_state8_tc(const safedit_tensor* k8, const safedit_tensor* v8, const State8Params& p,
                                int64_t ctas, cudaStream_t s) {
  CUtensorMap tmK, tmV;
  safedit_status st;
  if ((st = codes_map(&tmK, k8)) != SAFEDIT_OK) return st;
  if ((st = codes_map(&tmV, v8)) != SAFEDIT_OK) return st;
  const bool e4m3 = k8->dtype == SAFEDIT_E4M3;
#define SD_TC(D)                                                                                        \
  if (p.pad)                                                                                            \
    return e4m3 ? launch_tc<D, true, true>(tmK, tmV, p, ctas, s) : launch_tc<D, true, false>(tmK, tmV, p, ctas, s); \
  return e4m3 ? launch_tc<D, false, true>(tmK, tmV, p, ctas, s) : launch_tc<D, false, false>(tmK, tmV, p, ctas, s);
  switch (k8->dims[3]) {
    case 64: SD_TC(64)
    case 96: SD_TC(96)
    default: SD_TC(128)
  }
#undef SD_TC
}

}  // namespace sd
