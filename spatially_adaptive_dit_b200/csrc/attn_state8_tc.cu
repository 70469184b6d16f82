// attn_state8_tc.cu -- attention of many query rows over an 8-bit state, on
// the fifth-generation tensor cores.
//
// One CTA per SM, 384 threads = 12 warps, 256 query rows (two tiles of 128)
// of one (b, h) slice against a range of the keys:
//   * warpgroups 0 and 1: the softmax of one tile each, thread = query row =
//     TMEM lane.  They first gather their rows, scale them to f16 and lay them
//     out for the tensor core.
//   * warp 11 issues tcgen05.mma.
//   * warps 8 to 10 stream the codes of K and V by TMA (128 keys a tile) into a
//     ring and widen them to f16 into the swizzled tiles that the tensor
//     core reads (the tensor core has no product of a 16-bit and an 8-bit
//     operand, and 8-bit queries or weights would lose what the state keeps),
//     and compute each tile's scale factors and pads.
//   * S_t = Q_t K_j^T into TMEM (fp32), weights back into TMEM as f16 in place
//     of S_t, O_t += W_t V_j, each half of the keys as soon as its weights are
//     there; issue order per key tile W V_0(j), Q K_0(j+1), W V_1(j),
//     Q K_1(j+1), so one tile's softmax overlaps the other's MMAs.
//   * online softmax in base 2 with a lazy rescale (by more than 2^8), scales
//     of 16 keys at a time folded into the factor and offset of the exponent.
//   * a tile with a wide key (see attn_state8.cuh) has pairs of bf16 weights and
//     V as bf16, with a path of its own in each role.
// With at most 128 query rows both tiles hold the same rows and take the key
// tiles in turn, each with its own sums, which are joined like parts.
//
// Bound, at d = 96, by the chain softmax -> products -> softmax of a tile
// (3300 cycles for 128 keys: 1000 waiting for scores, 300 reading them, 2000
// for maximum and weights, of which the special function unit needs 1024, or
// 2048 where the two tiles meet) against 1536 of tensor time; at d = 128 the
// tensor time is 2048 and the widening of int8 codes (two instructions a pair
// and an exclusive or, against one conversion of e4m3) shows too.  One wave of
// 148 CTAs over 8192 keys, us (TFLOP/s), e4m3 / int8: d = 64 120 / 126 (660 /
// 630), d = 96 130 / 136 (915 / 875), d = 128 147 / 162 (1080 / 980), with pads
// 161 / 163, 170 / 178, 183 / 206; the same shapes over a bf16 state take 125 at
// d = 96.  The paths for wide tiles and large scores, not taken there, cost 5% of
// this (123 / 129 and 140 / 151 without them): registers and code beside the
// usual tile's.  Taken, they take 2.3 times as long.  Measured, before them, and
// not kept: two warpgroups to a tile (24 warps, 80 registers; 154 against 127),
// halves of the keys with their own score products (N = 64 products read the
// query tile twice and run at 48 cycles instead of 32; 169 against 139 at d =
// 128), 1/8 or 1/4 of the exponentials as a polynomial (126 to 131 against 127).
// Key tiles whose pads are all -inf are skipped by every role.  Every wait is
// bounded; an expired one raises the CTA's abort flag, drains what is in
// flight, frees TMEM and returns.
#include <type_traits>

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
  static constexpr int N_BARS = 1 + 4 * NS + NR + 2 + 4 + 2;
  static constexpr int OFF_FACT = OFF_BAR + ((N_BARS * 8 + 8 + 15) / 16) * 16;
  static constexpr int OFF_BASE = OFF_FACT + NF * 8 * 12;  // of the V scales
  static constexpr int OFF_FLAGS = OFF_BASE + 4;  // for each slot its largest ks; sign: wide, lowest bit: a masked key
  static constexpr int OFF_PAD = OFF_BASE + ((4 + NF * 4 + 15) / 16) * 16;
  static constexpr int OFF_LIVE = OFF_PAD + NF * 128 * 4;
  static constexpr int OFF_TOP = OFF_LIVE + LIVE_WORDS * 4;  // the largest pad
  static constexpr int SMEM_PLAIN = 1024 + OFF_PAD;
  static constexpr int SMEM_PAD = 1024 + OFF_TOP + 4;
  static_assert(SMEM_PAD <= 232448, "shared memory");
  static_assert(8 * 32 * (2 * D + 16) <= OFF_RAW, "rows on their way out");
  static_assert(256 + 2 * D <= 512, "TMEM columns");
};

constexpr int kTcThreads = 384;
constexpr int kTcWidenThreads = 96;
// 256 * 208 + 128 * 88 = 256 * 192 + 128 * 120 = 384 * 168.  The second split
// is the pads' (8192 keys of 96, e4m3, when it was chosen: 160 us against 183
// with the first, which spills there; without pads 130 against 127).
template <bool PAD>
struct TcRegs {
  static constexpr uint32_t SOFTMAX = PAD ? 192 : 208, OTHER = PAD ? 120 : 88;
  static_assert(256 * SOFTMAX + 128 * OTHER <= 384 * 168, "register split");
};
constexpr uint64_t kTcDrainNs = 1000000000ull;
// A batch whose largest pad is within this (in log2 units) has lv added to
// its pads: a sum that matters is off by 2^-13 at most, within the weights' f16
// rounding (keys 2^13 below the largest have no weight either way).  Beyond
// it, where the pad absorbs lv and the score itself, as it does in the
// plain sum, the largest pad comes off first.
constexpr float kFarPad = 4096.f;
// A row's factor of the products from which on scores may reach 2^22: products are
// sums of at most 128 of a query of 2^13 and a code of 448.
constexpr float kLargeFactor = 4194304.f / (8192.f * 448.f * 128.f);

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
// Asynchronous 16-byte copy, zeros past `bytes` (0 or 16).
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ float lds32(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ float2 lds64(uint32_t at) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at));
  return v;
}
__device__ __forceinline__ void sts32(uint32_t at, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

// The warp's largest.
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// Two weights -> f16x2; what rounding of a huge exponent takes past 65504 stays there.
__device__ __forceinline__ uint32_t pack_f16x2_sat(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The larger ones of two pairs of bf16, NaN where one is.
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ bool nan_bf16x2(uint32_t v) {
  return (v & 0x7FFFu) > 0x7F80u || (v & 0x7FFF0000u) > 0x7F800000u;
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0u;
}

// One arrival for the whole warp: 32 of them on one barrier serialise (at 256
// for each query tile and 512 for the widening they were most of the time
// between the last weight and the next product).
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// Barrier of `threads` threads that also tells all of them whether any has v.
__device__ __forceinline__ bool bar_any(int id, int threads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred.aligned q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(uint32_t(v))
      : "memory");
  return r != 0u;
}

// Instruction descriptor of kind::f16 with f16 A and B, fp32 accumulate.
constexpr uint32_t idesc_f16_f32(int M, int N, int b_mn_major) {
  return (1u << 4) | (uint32_t(b_mn_major) << 16) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
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
  constexpr int Q_FULL = 0, K_FULL = 1, K_EMPTY = K_FULL + C::NS, V_FULL = K_EMPTY + C::NS, V_EMPTY = V_FULL + C::NS,
                RAW_FULL = V_EMPTY + C::NS, S_FULL = RAW_FULL + C::NR,
                P_FULL = S_FULL + 2, O_FULL = P_FULL + 4, DRAIN = O_FULL + 1;
  static_assert(DRAIN + 1 == C::N_BARS, "barriers");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::N_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  // uniform, so that what depends on the role alone stays in uniform registers
  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  // CTAs below n_full take whole units; the others part (i % n_split) of unit
  // n_full + i / n_split
  const bool whole = int(blockIdx.x) < p.n_full;
  const int rest = int(blockIdx.x) - p.n_full;
  const int unit = whole ? int(blockIdx.x) : p.n_full + rest / p.n_split;
  const int part = whole ? 0 : rest % p.n_split;
  const int bh = unit / p.n_tiles;
  const int b = bh / p.H, h = bh - b * p.H;
  const int row0 = (unit - bh * p.n_tiles) * 256;
  const bool dual = p.dual;  // both tiles hold the same rows and take the key tiles in turn
  const bool two = row0 + 128 < p.n_rows;  // the second tile has rows of its own
  const int nk = (p.Nk + C::BN - 1) / C::BN;
  int k_lo = whole ? 0 : int(int64_t(nk) * part / p.n_split);
  int k_hi = whole ? nk : int(int64_t(nk) * (part + 1) / p.n_split);

  // live key tiles: one whose pads are all -inf carries no weight; and the
  // batch's largest pad (over all keys, so that every part refers to the same)
  const uint32_t live_s = sb + uint32_t(C::OFF_LIVE);
  bool skip_tiles = PAD && nk <= C::LIVE_WORDS * 32;
  float far_pad = 0.f;  // what comes off the exponents first (0 unless it is far)
  if constexpr (PAD) {
    uint32_t* live_bits = reinterpret_cast<uint32_t*>(smem + C::OFF_LIVE);
    int* const top_bits = reinterpret_cast<int*>(smem + C::OFF_TOP);
    // fp32 as an integer of the same order
    auto ordered = [](float v) { const int i = __float_as_int(v); return i >= 0 ? i : i ^ 0x7FFFFFFF; };
    if (threadIdx.x < C::LIVE_WORDS) live_bits[threadIdx.x] = 0u;
    if (threadIdx.x == 0) *top_bits = ordered(-INFINITY);
    __syncthreads();
    const float* pr = p.pad + b * p.pad_sb;
    float top = -INFINITY;
    // four tiles at a time in flight, four pads a lane
    for (int j0 = warp; j0 < nk; j0 += 4 * (kTcThreads / 32)) {
      float most[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = j0 + e * (kTcThreads / 32), k = j * C::BN + 4 * lane;
        float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (j < nk && k + 4 <= p.Nk) {
          v = __ldg(reinterpret_cast<const float4*>(pr + k));
        } else if (j < nk) {
          if (k < p.Nk) v.x = __ldg(pr + k);
          if (k + 1 < p.Nk) v.y = __ldg(pr + k + 1);
          if (k + 2 < p.Nk) v.z = __ldg(pr + k + 2);
        }
        most[e] = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
        if (v.x != v.x || v.y != v.y || v.z != v.z || v.w != v.w) most[e] = INFINITY;  // a NaN is no mask
        top = fmaxf(top, most[e]);
      }
      if (skip_tiles) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = j0 + e * (kTcThreads / 32);
          if (__any_sync(0xffffffffu, most[e] != -INFINITY) && lane == 0 && j >= k_lo && j < k_hi)
            atomicOr(live_bits + (j >> 5), 1u << (j & 31));
        }
      }
    }
    atomicMax(top_bits, ordered(top));
    __syncthreads();
    const int t = *top_bits;
    top = pad_log2(__int_as_float(t >= 0 ? t : t ^ 0x7FFFFFFF));
    if (fabsf(top) > kFarPad && fabsf(top) < INFINITY) far_pad = top;
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

  if constexpr (PAD) {  // live tiles that lie together (padding at an end): a shorter range, nothing to skip
    if (skip_tiles) {
      const int n = live_count(), first = next_live(k_lo);
      int j = first;
      while (j < k_hi && next_live(j) == j) ++j;
      if (n == 0 || j - first == n) {
        k_lo = n ? first : k_lo;
        k_hi = k_lo + n;
        skip_tiles = false;
      }
    }
  }

  if (threadIdx.x == 0) {
    mbar_init(BAR(Q_FULL), two || dual ? 8 : 4);
    for (int t = 0; t < 2; ++t) {
      mbar_init(BAR(S_FULL + t), 1);
      for (int hf = 0; hf < 2; ++hf) mbar_init(BAR(P_FULL + 2 * t + hf), 4);  // halves of the keys
    }
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(BAR(K_FULL + s), kTcWidenThreads / 32);
      mbar_init(BAR(K_EMPTY + s), 1);
      mbar_init(BAR(V_FULL + s), kTcWidenThreads / 32);
      mbar_init(BAR(V_EMPTY + s), 1);
    }
    for (int s = 0; s < C::NR; ++s) {
      mbar_init(BAR(RAW_FULL + s), 1);
    }
    mbar_init(BAR(O_FULL), 1);
    mbar_init(BAR(DRAIN), 1);
    *abort_flag = 0;
    sts32(sb + uint32_t(C::OFF_BASE), 0.f);
    mbar_fence_init();
  }
  if (warp == 11) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl ctl{abort_flag, p.status, p.wait_limit};
  auto flags_of = [&](int slot) { return __float_as_uint(lds32(sb + uint32_t(C::OFF_FLAGS + slot * 4))); };

  if (warp < 8) {
    // ================================================== softmax warpgroups
    setmaxnreg_inc<TcRegs<PAD>::SOFTMAX>();
    const int t = warp >> 2;  // query tile
    const int rr = dual ? threadIdx.x & 127 : threadIdx.x;  // row of the unit
    const int my_row = row0 + rr;
    if (t == 0 || two || dual) {
      int my_q = -1;
      if (my_row < p.n_rows) {
        my_q = p.idx ? __ldg(p.idx + my_row) : my_row;
        if (my_q < 0 || my_q >= p.Nq) {
          set_status(p.status, SAFEDIT_ERR_INDEX);
          my_q = -1;
        }
      }
      // ---- the warp's 32 query rows: copied piece by piece (16 bytes a lane,
      // neighbouring lanes on neighbouring pieces) into the swizzled K-major
      // layout; then each thread takes its own row's largest magnitude and
      // turns it into f16 in place.  A row to a thread straight from global
      // memory took 3.5 us, 32 cache lines a load.
      float undo;
      {
        constexpr int UNITS = D / 8;
        const uint32_t qs = sb + uint32_t(t * C::TILE_BYTES);
        auto piece = [&](int row, int c) {  // row of the tile, 16-byte piece
          return qs + uint32_t((c * 8 / C::CH) * C::CHUNK_BYTES) +
                 tc_swizzle(uint32_t(row * C::ROWB + (c * 8 % C::CH) * 2), C::LAYOUT);
        };
        const __nv_bfloat16* const qb = p.q + b * p.q_sb + h * p.q_sh;
        const int wrow = rr & 96;  // first row of the warp in the tile
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
          const int u = lane + 32 * i, row = u / UNITS, c = u - row * UNITS;
          const int qi = __shfl_sync(0xffffffffu, my_q, row);
          cp_async16_zfill(piece(wrow + row, c), qb + (qi < 0 ? 0 : int64_t(qi) * p.q_sr + c * 8), qi < 0 ? 0u : 16u);
        }
        asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
        __syncwarp();
        uint32_t m = 0u;
#pragma unroll
        for (int c = 0; c < UNITS; ++c) {
          const uint4 v = lds128(piece(rr & 127, c));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) m = max(m, max((w[e] << 16) & 0x7FFF0000u, w[e] & 0x7FFF0000u));
        }
        const float f = query_factor(m, p.scale_log2, undo);
#pragma unroll
        for (int c = 0; c < UNITS; ++c) {
          const uint32_t at = piece(rr & 127, c);
          const uint4 v = lds128(at);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[e] = pack_f16x2(__uint_as_float(w[e] << 16) * f, __uint_as_float(w[e] & 0xFFFF0000u) * f);
          sts128(at, o[0], o[1], o[2], o[3]);
        }
        fence_proxy_async_smem();
        warp_arrive(BAR(Q_FULL), lane);
      }

      const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
      const uint32_t tS = tmem + uint32_t(t * 128) + lane_base;
      const uint32_t tO = tmem + 256u + uint32_t(t * D) + lane_base;
      float m_run = -INFINITY, l_run = 0.f;
      bool ok = true;
      // this tile's key tiles: all of them, or every other one
      const int step = dual ? 2 : 1, begin = dual ? t : 0;
      const int n_mine = (live_count() - begin + step - 1) / step;
      int j = next_live(k_lo), slot = begin;
      if (begin && n_mine > 0) j = next_live(j + 1);
      // The reference of the row's weights brought to a new maximum, with what was summed.
      auto follow = [&](float mt, bool sums) {
        float alpha = 1.f;
        bool need_o = false;
        if (mt > m_run + kLazyTop) {
          const float to = mt - kHeadroom;
          alpha = ex2_approx(m_run - to);  // 0 from m = -inf
          l_run *= alpha;
          m_run = to;
          need_o = sums;
        }
        if (__any_sync(0xffffffffu, need_o)) {
#pragma unroll 1
          for (int e0 = 0; e0 < D; e0 += 16) {
            uint32_t r[16];
            tmem_ld16(tO + uint32_t(e0), r);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
            tmem_st16(tO + uint32_t(e0), r);
          }
        }
      };
      // A tile out of the ordinary: scores are read 32 at a time and twice (few
      // registers, so that the usual tile keeps its).  `pair`: a wide one, pairs of
      // bf16, 32 keys' in the columns of their scores.  Else one whose scores may be
      // large: each exponent is rounded before the reference comes off, so that the
      // largest one's does not depend on its size.  (The usual path takes a fused
      // product, which at scores of 2^31 left the reference by 2^7.)
      auto other_tile = [&](uint32_t fact, uint32_t pads, int lim, bool sums, bool pair) {
        auto exponents = [&](int c, float (&a)[32]) {  // of 32 keys, without the reference
          uint32_t r[32];
          tmem_ld32(tS + uint32_t(c * 32), r);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const uint32_t at = fact + uint32_t((2 * c + e / 16) * 4);
            const float k = undo * lds32(at), v = lds32(at + 32u), y = __uint_as_float(r[e]);
            if constexpr (PAD) {
              a[e] = fmaf(y, k, lds32(pads + uint32_t((32 * c + e) * 4)));
              if (far_pad != 0.f) a[e] = (a[e] - far_pad) + v;
            } else {
              a[e] = 32 * c + e < lim ? fmaf(y, k, v) : -INFINITY;
            }
          }
        };
        float mt = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float a[32];
          exponents(c, a);
#pragma unroll
          for (int e = 0; e < 32; ++e) mt = fmaxf(mt, a[e]);
        }
        follow(mt, sums);
        const float neg_m = m_run == -INFINITY ? 0.f : -m_run;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float a[32];
          exponents(c, a);
          uint32_t w[16];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float sum = 0.f;
#pragma unroll
            for (int e = 16 * g; e < 16 * g + 16; ++e) {
              a[e] = ex2_approx(a[e] + neg_m);
              sum += a[e];
            }
            l_run = fmaf(sum, lds32(fact + uint32_t(64 + (2 * c + g) * 4)), l_run);
          }
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] = pair ? take_bf16x2(a[2 * e], a[2 * e + 1]) : pack_f16x2_sat(a[2 * e], a[2 * e + 1]);
          tmem_st16(tS + uint32_t(c * (pair ? 32 : 16)), w);
          if (pair) {
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(a[2 * e], a[2 * e + 1]);
            tmem_st16(tS + uint32_t(c * 32 + 16), w);
          }
          if (c & 1) {
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(BAR(P_FULL + 2 * t + c / 2), lane);
          }
        }
      };
      for (int it = 0; it < n_mine; ++it) {
        if (!wait_warp(BAR(S_FULL + t), uint32_t(it & 1), ctl)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // factors of the tile's eight groups of 16 keys: ks, lv, 2^-lv
        const uint32_t fact = sb + uint32_t(C::OFF_FACT + slot * 96);
        const uint32_t pads = sb + uint32_t(C::OFF_PAD + slot * 512);
        const int lim = p.Nk - j * C::BN;
        const uint32_t flags = flags_of(slot);
        const bool other = flags >= 0x80000000u || !(__uint_as_float(flags) * undo < kLargeFactor);
        if (__builtin_expect(__any_sync(0xffffffffu, other), 0)) {
          other_tile(fact, pads, lim, it > 0, flags >> 31);
        } else {
          float x[128];
          {
            uint32_t r[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(tS + uint32_t(c * 32), r[c]);
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e) x[c * 32 + e] = __uint_as_float(r[c][e]);
          }
          const bool ragged = !PAD && lim < C::BN;
          float kf[8], lv[8];
#pragma unroll
          for (int g = 0; g < 8; g += 4) {
            const uint4 k4 = lds128(fact + uint32_t(g * 4)), l4 = lds128(fact + uint32_t(32 + g * 4));
            kf[g] = undo * __uint_as_float(k4.x), kf[g + 1] = undo * __uint_as_float(k4.y);
            kf[g + 2] = undo * __uint_as_float(k4.z), kf[g + 3] = undo * __uint_as_float(k4.w);
            lv[g] = __uint_as_float(l4.x), lv[g + 1] = __uint_as_float(l4.y);
            lv[g + 2] = __uint_as_float(l4.z), lv[g + 3] = __uint_as_float(l4.w);
          }
          tmem_wait_ld();
          if constexpr (PAD) {  // exponents undo ks x + pad + lv; kf and lv have done their part
            // (the pads of 16 keys are read together: one read at a time, each
            // waited for, cost a third of the tile)
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              uint4 pd[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) pd[e] = lds128(pads + uint32_t(g * 64 + e * 16));
              const uint64_t kf2 = f2_pack(kf[g], kf[g]);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float* y = x + 16 * g + 4 * e;
                f2_unpack(f2_fma(f2_pack(y[0], y[1]), kf2, f2_pack(__uint_as_float(pd[e].x), __uint_as_float(pd[e].y))),
                          y[0], y[1]);
                f2_unpack(f2_fma(f2_pack(y[2], y[3]), kf2, f2_pack(__uint_as_float(pd[e].z), __uint_as_float(pd[e].w))),
                          y[2], y[3]);
              }
            }
            if (far_pad != 0.f) {  // the pads here lack lv
              const uint64_t off = f2_pack(-far_pad, -far_pad);
#pragma unroll
              for (int c = 0; c < 128; c += 2) {
                const float v = lv[c / 16];
                f2_unpack(f2_add(f2_add(f2_pack(x[c], x[c + 1]), off), f2_pack(v, v)), x[c], x[c + 1]);
              }
            }
#pragma unroll
            for (int g = 0; g < 8; ++g) kf[g] = 1.f, lv[g] = 0.f;
          } else if (ragged) {
#pragma unroll
            for (int c = 0; c < 128; ++c) x[c] = c < lim ? x[c] * kf[c / 16] : -INFINITY;
#pragma unroll
            for (int g = 0; g < 8; ++g) kf[g] = 1.f;
          }
          // The row's reference m follows the maximum lazily, by more than 2^8
          // at a time.  (Taking the weights first and again where their sum says
          // that m was too low saves the maximum, but keeps all 128 scores alive
          // to the end: slower, for want of registers.)
          float mt = -INFINITY;
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            const float* y = x + 16 * g;
            float m0 = max3(y[0], y[1], y[2]), m1 = max3(y[3], y[4], y[5]);
            m0 = max3(m0, y[6], y[7]), m1 = max3(m1, y[8], y[9]);
            m0 = max3(m0, y[10], y[11]), m1 = max3(m1, y[12], y[13]);
            m0 = max3(m0, y[14], y[15]);
            mt = fmaxf(mt, fmaf(fmaxf(m0, m1), kf[g], lv[g]));
          }
          follow(mt, it > 0);
          const float neg_m = m_run == -INFINITY ? 0.f : -m_run;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float2 inv = lds64(fact + uint32_t(64 + c * 8));
            uint32_t pk[16];
#pragma unroll
            for (int gg = 0; gg < 2; ++gg) {
              const int g = 2 * c + gg;
              const float off = lv[g] + neg_m;
              const uint64_t kf2 = f2_pack(kf[g], kf[g]), off2 = f2_pack(off, off);
              uint64_t s0 = f2_pack(0.f, 0.f), s1 = s0;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint64_t xx = f2_pack(x[16 * g + 2 * e], x[16 * g + 2 * e + 1]);
                float a0, a1;
                f2_unpack(PAD ? f2_add(xx, off2) : f2_fma(xx, kf2, off2), a0, a1);
                const float p0 = ex2_approx(a0), p1 = ex2_approx(a1);
                if (e & 1)
                  s1 = f2_add(s1, f2_pack(p0, p1));
                else
                  s0 = f2_add(s0, f2_pack(p0, p1));
                pk[8 * gg + e] = pack_f16x2(p0, p1);
              }
              float u0, u1;
              f2_unpack(f2_add(s0, s1), u0, u1);
              l_run = fmaf(u0 + u1, gg ? inv.y : inv.x, l_run);
            }
            tmem_st16(tS + uint32_t(c * 16), pk);
            if (c & 1) {  // half of the keys: their products start
              tmem_wait_st();
              tc_fence_before();
              warp_arrive(BAR(P_FULL + 2 * t + c / 2), lane);
            }
          }
        }
        j = next_live(j + 1);
        if (dual) j = next_live(j + 1);
        slot += step;
        if (slot >= C::NF) slot -= C::NF;
      }
      // ---- epilogue: O / l -> bf16 rows, or the part's record
      if (ok && wait_warp(BAR(O_FULL), 0u, ctl)) {
        tc_fence_after();
        const bool live = my_q >= 0;
        const bool empty = l_run == 0.f;  // O may never have been written
        const float base = lds32(sb + uint32_t(C::OFF_BASE));
        if (live && whole && empty) set_status(p.status, SAFEDIT_ERR_MASKED_ROW);
        const float inv = empty ? 0.f : pow2(base) / l_run;
        // Rows leave through shared memory (the query tiles', free by now), so
        // that a warp's stores run along rows: bf16 rows at once, a part's
        // fp32 rows half a row at a time.  Rows are 16 bytes apart from a
        // multiple of 128, which keeps eight lanes on different banks.
        constexpr int PITCH = 2 * D + 16, UNITS = D / 8;
        const uint32_t stage = sb + uint32_t(warp * 32 * PITCH);
        const uint32_t mine = stage + uint32_t(lane * PITCH);
        if (whole) {
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            uint32_t r[32];
            tmem_ld32(tO + uint32_t(c), r);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t o[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                o[k] = empty ? 0u
                             : pack_bf16x2(__uint_as_float(r[8 * e + 2 * k]) * inv,
                                           __uint_as_float(r[8 * e + 2 * k + 1]) * inv);
              sts128(mine + uint32_t(c * 2 + e * 16), o[0], o[1], o[2], o[3]);
            }
          }
          __syncwarp();
          __nv_bfloat16* const ob = p.out + b * p.o_sb + h * p.o_sh;
          uint32_t top[2] = {0u, 0u};  // NaN where the lane sees one on its way
#pragma unroll
          for (int i = 0; i < UNITS; ++i) {
            const int u = lane + 32 * i, row = u / UNITS, c = u - row * UNITS;
            const int qi = __shfl_sync(0xffffffffu, my_q, row);
            const int64_t at = p.out_scattered ? int64_t(qi) : int64_t(row0 + (rr & ~31) + row);
            const uint4 v = lds128(stage + uint32_t(row * PITCH + c * 16));
            if constexpr (E4M3) {
              top[0] = max_nan_bf16x2(max_nan_bf16x2(top[0], v.x), v.y);
              top[1] = max_nan_bf16x2(max_nan_bf16x2(top[1], v.z), v.w);
            }
            if (qi >= 0) *reinterpret_cast<uint4*>(ob + at * p.o_sr + c * 8) = v;
          }
          bool nan = inv != inv;  // of scores; a NaN code of V leaves the sum alone (int8 has none)
          if constexpr (E4M3) {
            if (__any_sync(0xffffffffu, nan_bf16x2(top[0]) || nan_bf16x2(top[1]))) {  // each lane its own row
#pragma unroll 1
              for (int c = 0; c < D / 2; ++c) nan |= nan_bf16x2(__float_as_uint(lds32(mine + uint32_t(c * 4))));
            }
          }
          if (nan && live) report_nan(p, b, h, my_q, D);
        } else {
          const PartView pv = part_view(p, dual ? 2 * rest + t : rest, D);
          float up;
          const float base_a = leave_base(base, l_run, up);
          if (live) pv.ml[rr] = make_float4(m_run, l_run, base_a, 0.f);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int c = 0; c < D / 2; c += 16) {
              uint32_t r[16];
              tmem_ld16(tO + uint32_t(half * (D / 2) + c), r);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 4; ++e)
              {
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k] = empty ? 0u : __float_as_uint(__uint_as_float(r[4 * e + k]) * up);
                sts128(mine + uint32_t(c * 4 + e * 16), o[0], o[1], o[2], o[3]);
              }
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
              const int u = lane + 32 * i, row = u / UNITS, c = u - row * UNITS;
              const int qi = __shfl_sync(0xffffffffu, my_q, row);
              if (qi >= 0)
                *reinterpret_cast<uint4*>(pv.o + int64_t((rr & ~31) + row) * D + half * (D / 2) + c * 4) =
                    lds128(stage + uint32_t(row * PITCH + c * 16));
            }
            __syncwarp();
          }
        }
      }
    }
  } else {
    setmaxnreg_dec<TcRegs<PAD>::OTHER>();
    if (warp == 11) {
      // ================================================ MMA issuer
      // The whole warp walks the loop and one elected lane issues, with the
      // descriptors in uniform registers: with a single lane in the loop each
      // of the 28 products of a tile took some 90 cycles to issue, which was
      // two thirds of the tile's time.
      constexpr uint32_t idesc_qk = idesc_f16_f32(128, 128, 0), idesc_pv = idesc_f16_f32(128, D, 1),
                         idesc_pv_bf16 = idesc_bf16_f32(128, D, 0, 1);
      constexpr uint32_t SBO = 8u * C::ROWB;
      const uint64_t qd0 = smem_desc(sb, 16u, SBO, C::LAYOUT);
      const uint64_t kd0 = smem_desc(sb + C::OFF_K, 16u, SBO, C::LAYOUT);
      const uint64_t vd0 = smem_desc(sb + C::OFF_V, uint32_t(C::CHUNK_BYTES), SBO, C::LAYOUT);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      // the address field of a descriptor advances in units of 16 bytes and
      // stays below 2^14, so a 64-bit add does not carry out of it
      auto issue_qk = [&](int t, int s) {
        const uint64_t qd = qd0 + uint64_t(uint32_t(t * C::TILE_BYTES) >> 4), kd = kd0 + uint64_t(uint32_t(s * C::TILE_BYTES) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = uint32_t(((kk * 16) / C::CH) * C::CHUNK_BYTES + ((kk * 16) % C::CH) * 2) >> 4;
            mma_ss(tm + uint32_t(t * 128), qd + off, kd + off, idesc_qk, kk > 0 ? 1u : 0u);
          }
          tc_commit(BAR(S_FULL + t));
        }
      };
      auto issue_pv = [&](int t, int hf, int s, bool acc, bool wide) {  // half of the keys
        const uint64_t vd = vd0 + uint64_t(uint32_t(s * C::TILE_BYTES + hf * 64 * C::ROWB) >> 4);
        const uint32_t to = tm + 256u + uint32_t(t * D), from = tm + uint32_t(t * 128);
        if (__builtin_expect(wide, 0)) {  // a pair of bf16 each, where the scores were
          if (elect_one()) {
#pragma unroll 1
            for (int kk = 0; kk < C::BN / 32; ++kk) {
              const uint32_t pair = from + uint32_t((hf * 2 + kk / 2) * 32 + (kk & 1) * 8);
              const uint64_t at = vd + (uint32_t(kk * 16 * C::ROWB) >> 4);
              mma_ts(to, pair, at, idesc_pv_bf16, (acc || kk > 0) ? 1u : 0u);
              mma_ts(to, pair + 16u, at, idesc_pv_bf16, 1u);
            }
          }
        } else if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < C::BN / 32; ++kk)
            mma_ts(to, from + uint32_t(hf * 32 + kk * 8), vd + (uint32_t(kk * 16 * C::ROWB) >> 4), idesc_pv,
                   (acc || kk > 0) ? 1u : 0u);
        }
      };
      auto commit = [&](int bar) {
        if (elect_one()) tc_commit(BAR(bar));
      };
      const int n_live = live_count();
      // both halves of tile t's weights for its i-th key tile, as they come
      auto weigh = [&](int t, int s, int i, bool wide) {
        for (int hf = 0; hf < 2; ++hf) {
          if (!wait_warp(BAR(P_FULL + 2 * t + hf), uint32_t(i & 1), ctl)) return false;
          tc_fence_after();
          issue_pv(t, hf, s, i > 0 || hf > 0, wide);
        }
        return true;
      };
      auto keys_there = [&](int j) {
        if (!wait_warp(BAR(K_FULL + j % C::NS), uint32_t((j / C::NS) & 1), ctl)) return false;
        tc_fence_after();
        return true;
      };
      bool ok = wait_warp(BAR(Q_FULL), 0u, ctl);
      for (int j = 0; ok && j < (dual ? 2 : 1) && j < n_live; ++j) {
        if (!(ok = keys_there(j))) break;
        issue_qk(dual ? j : 0, j);
        if (two) issue_qk(1, j);
        commit(K_EMPTY + j);
      }
      for (int j = 0; ok && j < n_live; ++j) {
        const int s = j % C::NS;
        if (!(ok = wait_warp(BAR(V_FULL + s), uint32_t((j / C::NS) & 1), ctl))) break;
        const int ahead = dual ? 2 : 1, s1 = (j + ahead) % C::NS;
        const bool more = j + ahead < n_live;
        const int t = dual ? j & 1 : 0;
        const bool wide = __shfl_sync(0xffffffffu, flags_of(j % C::NF), 0) >> 31;
        if (!(ok = weigh(t, s, dual ? j >> 1 : j, wide))) break;
        if (dual) commit(V_EMPTY + s);
        if (more) {
          if (!(ok = keys_there(j + ahead))) break;
          issue_qk(t, s1);
        }
        if (!dual) {
          if (two && !(ok = weigh(1, s, j, wide))) break;
          commit(V_EMPTY + s);
          if (more && two) issue_qk(1, s1);
        }
        if (more) commit(K_EMPTY + s1);
      }
      if (ok) commit(O_FULL);
      // every MMA has completed before TMEM is freed, whoever aborted
      commit(DRAIN);
      wait_drain(BAR(DRAIN), 0u, kTcDrainNs);
      __syncwarp();
    } else {
    // ================================================ widening of the codes
    const int tid = threadIdx.x - 256;
    const float* padb = PAD ? p.pad + b * p.pad_sb : nullptr;
    const float* ksb = p.ks + b * p.ks_sb + h * p.ks_sh;
    const float* vsb = p.vs + b * p.vs_sb + h * p.vs_sh;
    constexpr int UPR = D / 16;  // 16-code units per row
    float lv_lo = INFINITY, lv_hi = -INFINITY;
    // raw tile -> f16 tile, in units of 16 codes, each two 16-byte pieces of
    // the f16 row, by 96 threads at offsets fixed for the kernel.
    //   d = 96: thread r takes row r (stores of eight lanes fall on different
    //     banks, loads two by two on the same); the last 32 rows go two units
    //     to a thread.
    //   d = 64, 128: units tid, tid + 96, ..: rows 24 or 12 apart, so the
    //     swizzle is the first's or, every other time at d = 128, has its
    //     third bit flipped.  Lanes of a row's second chunk write their pieces
    //     in the other order, which keeps eight lanes on different banks.
    auto place = [&](uint4 v, uint32_t a0, uint32_t a1) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t o[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t x = bias_codes<E4M3>(w[e]);
        o[2 * e] = widen_lo<E4M3>(x);
        o[2 * e + 1] = widen_hi<E4M3>(x);
      }
      sts128(a0, o[0], o[1], o[2], o[3]);
      sts128(a1, o[4], o[5], o[6], o[7]);
    };
    // What a tile rarely needs after its widening, row by row.  `clear`: rows of
    // masked keys back to zero, whatever their codes (NaN) became.  (int8 has no
    // NaN: what it holds, a weight of 0 takes out.)  `wide`: f16 -> bf16.
    auto mend = [&](uint32_t to, uint32_t pads, bool clear, bool wide) {
#pragma unroll 1
      for (int r = tid; r < C::BN; r += kTcWidenThreads) {
        bool zero = false;
        if constexpr (PAD) zero = clear && lds32(pads + uint32_t(r * 4)) == -INFINITY;
        if (!zero && !wide) continue;
#pragma unroll 1
        for (int c = 0; c < D / 8; ++c) {
          const uint32_t at = to + uint32_t((c * 8 / C::CH) * C::CHUNK_BYTES) +
                              tc_swizzle(uint32_t(r * C::ROWB + (c * 8 % C::CH) * 2), C::LAYOUT);
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (!zero) {
            v = lds128(at);
            v = make_uint4(f16x2_to_bf16x2(v.x), f16x2_to_bf16x2(v.y), f16x2_to_bf16x2(v.z), f16x2_to_bf16x2(v.w));
          }
          sts128(at, v.x, v.y, v.z, v.w);
        }
      }
    };
    constexpr int RPP = kTcWidenThreads / UPR;  // d = 64, 128: rows a pass
    const int u_row = tid / UPR, u_col = tid % UPR;
    const bool swap = D != 96 && ((u_col * 16 / C::CH) & 1);
    const uint32_t in_row = uint32_t(u_row * C::ROWB + (u_col * 16 % C::CH) * 2);
    const uint32_t chunk0 = uint32_t((u_col * 16 / C::CH) * C::CHUNK_BYTES);
    const uint32_t p0 = chunk0 + tc_swizzle(in_row + (swap ? 16u : 0u), C::LAYOUT);
    const uint32_t p1 = chunk0 + tc_swizzle(in_row + (swap ? 0u : 16u), C::LAYOUT);
    // the loads of four units go out before the first is widened
    auto widen = [&](uint32_t raw, uint32_t to) {
      if constexpr (D == 96) {
#pragma unroll
        for (int i0 = 0; i0 < 8; i0 += 4) {
          uint4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = i0 + i < 6 ? tid : 96 + lane, c = i0 + i < 6 ? i0 + i : (tid >> 5) * 2 + i0 + i - 6;
            v[i] = lds128(raw + uint32_t(r * D + c * 16));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = i0 + i < 6 ? tid : 96 + lane, c = i0 + i < 6 ? i0 + i : (tid >> 5) * 2 + i0 + i - 6;
            const uint32_t in = uint32_t(r * C::ROWB + (c & 1) * 32), base = to + uint32_t((c / 2) * C::CHUNK_BYTES);
            place(v[i], base + tc_swizzle(in, C::LAYOUT), base + tc_swizzle(in + 16u, C::LAYOUT));
          }
        }
      } else {
        constexpr int PASSES = (128 + RPP - 1) / RPP;
#pragma unroll
        for (int i0 = 0; i0 < PASSES; i0 += 4) {
          uint4 v[4];
#pragma unroll
          for (int i = i0; i < i0 + 4 && i < PASSES; ++i) {
            if (i + 1 < PASSES || u_row + i * RPP < 128) {
              v[i - i0] = lds128(raw + uint32_t(tid * 16 + i * RPP * D));
            }
          }
#pragma unroll
          for (int i = i0; i < i0 + 4 && i < PASSES; ++i) {
            if (i + 1 < PASSES || u_row + i * RPP < 128) {
              const uint4 x = v[i - i0];
              const uint32_t flip = (RPP * i) & 4 ? 64u : 0u, at = to + uint32_t(i * RPP * C::ROWB);
              place(swap ? make_uint4(x.z, x.w, x.x, x.y) : x, at + (p0 ^ flip), at + (p1 ^ flip));
            }
          }
        }
      }
    };
    // Raw tiles come by TMA into a ring, K and V of a key tile in turn: tile n
    // of them goes to slot n % NR.  Thread 0 issues, tile n + NR once the
    // group's barrier says that tile n has been read.
    const int n_live = live_count();
    int issued = 0, kt_load = next_live(k_lo);
    auto load_next = [&]() {  // thread 0
      if (issued >= 2 * n_live) return;
      const int s = issued % C::NR;
      mbar_arrive_expect_tx(BAR(RAW_FULL + s), C::RAW_BYTES);
      tma_load_4d(sb + uint32_t(C::OFF_RAW + s * C::RAW_BYTES), issued & 1 ? &tmV : &tmK, BAR(RAW_FULL + s), 0,
                  kt_load * C::BN, h, b);
      if (issued & 1) kt_load = next_live(kt_load + 1);
      ++issued;
    };
    if (tid == 0)
      for (int n = 0; n < C::NR; ++n) load_next();
    // Scale factors and pads of a key tile, in NS + 1 slots, published a tile
    // ahead: with the V tile of tile `it`, when V tile `it - NS` is free.  Its
    // products took the weights of tile `it - NS` from both query tiles, so
    // nobody reads that slot any more, and tile `it + 1` takes it.  Their loads
    // go out a step before.
    // Warp 8 does it: a lane holds the scales of group lane % 8 and the pads of
    // keys 4 lane .. 4 lane + 3, so it knows each group's live keys; scales of a
    // group without one count for nothing, whatever they are.
    float next_ks = 0.f, next_vs = 1.f;
    float4 next_pad = make_float4(0.f, 0.f, 0.f, 0.f);
    float base = NAN, lv_top = -INFINITY;  // of the V scales (base: NaN before the first in use)
    auto fetch = [&](int kt) {
      const int key = kt * C::BN + (lane & 7) * 16;
      if (key < p.Nk) {
        next_ks = __ldg(ksb + (key >> p.block_log2));
        next_vs = __ldg(vsb + (key >> p.block_log2));
      }
      if constexpr (PAD) {
        const int k = kt * C::BN + 4 * lane;
        next_pad = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (k + 4 <= p.Nk) {
          next_pad = __ldg(reinterpret_cast<const float4*>(padb + k));
        } else {
          if (k < p.Nk) next_pad.x = __ldg(padb + k);
          if (k + 1 < p.Nk) next_pad.y = __ldg(padb + k + 1);
          if (k + 2 < p.Nk) next_pad.z = __ldg(padb + k + 2);
        }
      }
    };
    auto publish = [&](int kt, int slot) {
      bool used = kt * C::BN + (lane & 7) * 16 < p.Nk;
      if constexpr (PAD) {
        const uint32_t live = __ballot_sync(0xffffffffu, next_pad.x != -INFINITY || next_pad.y != -INFINITY ||
                                                             next_pad.z != -INFINITY || next_pad.w != -INFINITY);
        used = (live >> (4 * (lane & 7)) & 15u) != 0u;
      }
      float ks = 0.f, lv = 0.f;
      if (used) {
        ks = next_ks;
        lv = __log2f(next_vs);
        if (!(ks >= 0.f && ks < INFINITY && next_vs > 0.f && next_vs < INFINITY)) {
          set_status(p.status, SAFEDIT_ERR_INVALID_ARG);
        } else {
          scale_range(next_vs, lv, lv_lo, lv_hi);
        }
      }
      const uint32_t in_use = __ballot_sync(0xffffffffu, used) & 255u;
      if (base != base && in_use != 0u) {
        base = scale_base(__shfl_sync(0xffffffffu, lv, __ffs(in_use) - 1));
        if (lane == 0) sts32(sb + uint32_t(C::OFF_BASE), base);
      }
      if (used) lv -= base;
      lv_top = fmaxf(lv_top, warp_max(used ? lv : -INFINITY));
      uint32_t flags = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(ks, 0.f))) & 0x7FFFFFFEu;
      if (__any_sync(0xffffffffu, used && lv < lv_top - kHalfSpread)) flags |= 0x80000000u;
      if (lane < 8) {
        const uint32_t f = sb + uint32_t(C::OFF_FACT + slot * 96 + lane * 4);
        sts32(f, ks);
        sts32(f + 32u, lv);
        sts32(f + 64u, ex2_approx(-lv));
      }
      if constexpr (PAD) {
        float pd[4] = {next_pad.x, next_pad.y, next_pad.z, next_pad.w};
        const float lk = far_pad != 0.f ? 0.f : __shfl_sync(0xffffffffu, lv, lane >> 2);
        bool dead = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pd[e] = pad_log2(pd[e]);
          dead |= pd[e] == -INFINITY;
          if (pd[e] != -INFINITY) pd[e] += lk;
        }
        sts128(sb + uint32_t(C::OFF_PAD + slot * 512 + lane * 16), __float_as_uint(pd[0]), __float_as_uint(pd[1]),
               __float_as_uint(pd[2]), __float_as_uint(pd[3]));
        if (E4M3 && __any_sync(0xffffffffu, dead)) flags |= 1u;
      }
      if (lane == 0) sts32(sb + uint32_t(C::OFF_FLAGS + slot * 4), __uint_as_float(flags));
    };
    bool ok = true;
    int slot = 0, kt = next_live(k_lo);
    if (warp == 8 && n_live > 0) {
      fetch(kt);
      publish(kt, 0);
    }
    bar_any(1, kTcWidenThreads, false);
    for (int it = 0; ok && it < n_live; ++it) {
      const int s = it % C::NS;
      const uint32_t ph = uint32_t((it / C::NS) & 1) ^ 1u;
      const int kt1 = next_live(kt + 1), slot1 = slot + 1 == C::NF ? 0 : slot + 1;
      const bool more = it + 1 < n_live;
      if (warp == 8 && more) fetch(kt1);
      const uint32_t flags = flags_of(slot);
      const bool wide = flags >> 31, dead = PAD && E4M3 && (flags & 1u);
      for (int kv = 0; ok && kv < 2; ++kv) {
        const int n = 2 * it + kv, raw = n % C::NR;
        ok = wait_warp(BAR(RAW_FULL + raw), uint32_t((n / C::NR) & 1), ctl) &&
             wait_warp(BAR((kv ? V_EMPTY : K_EMPTY) + s), ph, ctl);
        const uint32_t to = sb + uint32_t((kv ? C::OFF_V : C::OFF_K) + s * C::TILE_BYTES);
        if (ok) {
          widen(sb + uint32_t(C::OFF_RAW + raw * C::RAW_BYTES), to);
        }
        if (__builtin_expect(dead || (kv && wide), 0)) {  // all three warps see the same, and come here whether or not a wait ran out
          ok = !bar_any(2, kTcWidenThreads, !ok);
          if (ok) mend(to, sb + uint32_t(C::OFF_PAD + slot * 512), dead, kv && wide);
        }
        if (ok) {
          fence_proxy_async_smem();
          warp_arrive(BAR((kv ? V_FULL : K_FULL) + s), lane);
          if (warp == 8 && kv && more) publish(kt1, slot1);
        }
        ok = !bar_any(1, kTcWidenThreads, !ok);  // read by all three warps, or given up by all
        if (ok && tid == 0) load_next();
      }
      kt = kt1;
      slot = slot1;
    }
    // every copy has landed before the CTA leaves
    if (tid == 0)
      for (int i = issued > C::NR ? issued - C::NR : 0; i < issued; ++i)
        wait_drain(BAR(RAW_FULL + i % C::NR), uint32_t((i / C::NR) & 1), kTcDrainNs);
    __syncwarp();
    if (warp == 8) {
#pragma unroll
      for (int e = 1; e < 8; e <<= 1) {
        lv_lo = fminf(lv_lo, __shfl_xor_sync(0xffffffffu, lv_lo, e));
        lv_hi = fmaxf(lv_hi, __shfl_xor_sync(0xffffffffu, lv_hi, e));
      }
      if (lane == 0) {
        if (whole) {
          if (lv_hi - lv_lo > kScaleSpread) set_status(p.status, SAFEDIT_ERR_INVALID_ARG);
        } else {
          for (int e = 0; e < (dual ? 2 : 1); ++e) {
            const PartView pv = part_view(p, dual ? 2 * rest + e : rest, D);
            pv.range[0] = lv_lo;
            pv.range[1] = lv_hi;
          }
        }
      }
    }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 11) {
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
