// state8.cu -- rows written into the 8-bit state.
//
//   scale = max |x| / qmax over the block's rows and the head's width,
//   code  = x qmax / max |x|, rounded once to the nearest code (ties to even),
//
// with the rows rotated in fp32 first where the tensor asks for it (K before
// its rounding to 8 bits, so no 16-bit rounding comes between).  Bound by
// memory: 3 bytes for each 16-bit element.  One CTA holds one block of tokens
// in registers, reads it once, and walks the heads of its group with the
// angles of its tokens kept, the next heads' loads in flight while this one
// is reduced (one barrier for each head).  K and V of 25600 tokens x 48 heads
// of 96 (708 MB): 140 to 150 us with K rotated, 128 us without (blocks of 64);
// d = 128: 170 and 156 us, 5.5 and 6.0 TB/s.
//
// The arithmetic is fp32's: an f32 or a rotated element within 2^-22 of the
// border between two codes may take either one, a 16-bit one that is not rotated
// meets every border as it is.
#include <type_traits>

#include <cuda_fp16.h>

#include "rope.cuh"
#include "state8.cuh"

namespace sd {

constexpr int kMaxStoreTensors = 4;
// a block whose magnitudes all lie below this is scaled as if its largest were this
constexpr float kLeastMax = 7.888609052210118e-31f;  // 2^-100

struct StoreParams {
  RopeTable tab;
  RopePos pos;
  const void* src[kMaxStoreTensors];
  uint8_t* code[kMaxStoreTensors];
  float* scale[kMaxStoreTensors];
  int64_t s_sb[kMaxStoreTensors], s_sh[kMaxStoreTensors], s_sr[kMaxStoreTensors];
  int64_t c_sb[kMaxStoreTensors], c_sh[kMaxStoreTensors], c_sr[kMaxStoreTensors];
  int64_t f_sb[kMaxStoreTensors], f_sh[kMaxStoreTensors];
  int rotate[kMaxStoreTensors];
  int heads[kMaxStoreTensors], group_end[kMaxStoreTensors];  // head groups of tensors 0..t together
  int heads_per_group, groups, any_rotate, slots, e4m3;
  int n_rows, row0, state_rows;
  int64_t limit;
  const int* idx;
  int src_indexed;
  int* status;
};

// Four fp32 values already scaled into the code's range -> four codes.
template <bool E4M3>
__device__ __forceinline__ uint32_t pack_codes(float a, float b, float c, float d) {
  if constexpr (E4M3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return uint32_t(lo) | uint32_t(hi) << 16;
  } else {
    // adding 1.5 * 2^23 rounds to an integer (ties to even) in the low bits
    constexpr float kMagic = 12582912.f;
    const uint32_t w0 = __float_as_uint(a + kMagic), w1 = __float_as_uint(b + kMagic);
    const uint32_t w2 = __float_as_uint(c + kMagic), w3 = __float_as_uint(d + kMagic);
    return __byte_perm(__byte_perm(w0, w1, 0x0040), __byte_perm(w2, w3, 0x0040), 0x5410);
  }
}

// BLOCK tokens, RP rows side by side (thread = slot of a row, d / 8 slots),
// R = BLOCK / RP rows of each thread.
template <int BLOCK>
struct StoreCfg {
  static constexpr int RP = BLOCK <= 64 ? 16 : 32;
  static constexpr int R = BLOCK / RP;
  static constexpr int MAX_THREADS = RP * 16;
  // 64, 80 and 128 registers a thread for one, two and four rows
  static constexpr int MIN_CTAS = (R == 1 ? 1024 : R == 2 ? 768 : 512) / MAX_THREADS;
};

template <typename T>
constexpr int kStoreDepth = sizeof(T) == 4 ? 3 : 4;  // heads of a block in shared memory

// A slot's two runs of 4 elements -> this thread's place, zeros where there is
// no row; and back.
template <typename T, bool HALVES>
__device__ __forceinline__ void slot_async(uint32_t dst, const T* row, int lo, int hi, bool there) {
  if constexpr (sizeof(T) == 2 && HALVES) {
    const uint32_t bytes = there ? 8u : 0u;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(row + lo), "r"(bytes) : "memory");
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst + 8u), "l"(row + hi), "r"(bytes) : "memory");
  } else {
    const uint32_t bytes = there ? 16u : 0u;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(row + lo), "r"(bytes) : "memory");
    if constexpr (sizeof(T) == 4)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 16u), "l"(row + hi), "r"(bytes) : "memory");
  }
}
template <typename T>
__device__ __forceinline__ void slot_read(uint32_t (&w)[SlotWords<T>::N], uint32_t at) {
#pragma unroll
  for (int e = 0; e < SlotWords<T>::N; e += 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[e]), "=r"(w[e + 1]), "=r"(w[e + 2]), "=r"(w[e + 3])
                 : "r"(at + uint32_t(e * 4)));
}

// max(m, |a|, |b|), NaN if one is.
__device__ __forceinline__ float max_abs3(float m, float a, float b) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
  return r;
}

template <typename T, int BLOCK, bool HALVES>
__global__ void __launch_bounds__(StoreCfg<BLOCK>::MAX_THREADS, StoreCfg<BLOCK>::MIN_CTAS)
    state8_store_kernel(const __grid_constant__ StoreParams p) {
  using C = StoreCfg<BLOCK>;
  constexpr int NW = SlotWords<T>::N;
  const float qmax = p.e4m3 ? 448.f : 127.f;
  __shared__ uint32_t part[2][C::MAX_THREADS / 32];
  const int rr = threadIdx.x / p.slots, slot = threadIdx.x - rr * p.slots;
  const int lane = threadIdx.x & 31, warps = int(blockDim.x) >> 5;
  const int b = blockIdx.z;
  // the head groups of a block of tokens follow one another, so rotated and
  // plain tensors (one bound by arithmetic, one by memory) run side by side
  const int blk = int(blockIdx.x) / p.groups;
  int group = int(blockIdx.x) - blk * p.groups;
  const int r0 = blk * BLOCK;
  int t = 0;
  while (group >= p.group_end[t]) ++t;
  if (t) group -= p.group_end[t - 1];
  const int h_begin = group * p.heads_per_group, h_end = min(p.heads[t], h_begin + p.heads_per_group);
  const bool rotate = p.rotate[t];
  int lo = slot * 8, hi = slot * 8 + 4;
  if (HALVES && p.any_rotate) {
    const uint32_t runs = p.tab.slot[slot].runs;
    lo = RopeSlot::lo(runs), hi = RopeSlot::hi(runs);
  }
  const T* from[C::R];  // source row of head h, null: none (its codes are zero)
  int token[C::R];
  const T* base = static_cast<const T*>(p.src[t]) + b * p.s_sb[t] + h_begin * p.s_sh[t];
#pragma unroll
  for (int k = 0; k < C::R; ++k) {
    const int r = r0 + rr + k * C::RP;
    from[k] = nullptr;
    token[k] = -1;
    if (r < p.n_rows) {
      const int i = p.idx ? __ldg(p.idx + r) : r;
      if (p.idx && (i < 0 || i >= p.limit)) {
        set_status(p.status, SAFEDIT_ERR_INDEX);
      } else {
        from[k] = base + int64_t(p.src_indexed ? i : r) * p.s_sr[t];
        token[k] = i;
      }
    }
  }
  // The next heads' elements are on their way into this thread's own places in
  // shared memory (so no barrier is needed for them), kStoreDepth<T> heads
  // deep: registers for one head ahead kept 24 KB in flight on an SM, which
  // bounds the rate at 4.4 TB/s by the memory's latency alone.
  constexpr int DEPTH = kStoreDepth<T>;
  extern __shared__ __align__(16) uint8_t store_ring[];
  const uint32_t ring = smem_u32(store_ring) + threadIdx.x * uint32_t(NW * 4);
  const uint32_t pitch = uint32_t(blockDim.x) * uint32_t(NW * 4);  // between a thread's rows and heads
  const uint32_t ring_end = ring + uint32_t(DEPTH * C::R) * pitch;
  // this tensor's strides, out of the parameter arrays once
  const int64_t s_sh = p.s_sh[t], c_sh = p.c_sh[t], c_rows = C::RP * p.c_sr[t];
  uint32_t put = ring, get = ring;  // where the next head goes, where this one is
  auto load = [&]() {
#pragma unroll
    for (int k = 0; k < C::R; ++k) {
      slot_async<T, HALVES>(put, from[k] ? from[k] : base, lo, hi, from[k] != nullptr);
      put += pitch;
      if (from[k]) from[k] += s_sh;
    }
    if (put == ring_end) put = ring;
  };
  const int first = p.row0 + r0 + rr;  // state row of the thread's first row
  uint8_t* to = p.code[t] + b * p.c_sb[t] + h_begin * p.c_sh[t] + int64_t(first) * p.c_sr[t];
  float* to_scale = p.scale[t] + b * p.f_sb[t] + h_begin * p.f_sh[t] + p.row0 / BLOCK + blk;
#pragma unroll
  for (int i = 0; i < DEPTH - 1; ++i) {
    if (h_begin + i < h_end) load();
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  float c[C::R][4], s[C::R][4];
#pragma unroll
  for (int k = 0; k < C::R; ++k) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c[k][j] = 1.f, s[k][j] = 0.f;
    if (rotate && token[k] >= 0) rope_angles(p.tab.slot[slot], p.pos, b, token[k], 1.f, c[k], s[k]);
  }
  for (int h = h_begin; h < h_end; ++h) {
    float x[C::R][8];
    asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 2) : "memory");
#pragma unroll
    for (int k = 0; k < C::R; ++k) {
      uint32_t w[NW];
      slot_read<T>(w, get);
      get += pitch;
      slot_widen<T>(w, x[k]);
    }
    if (get == ring_end) get = ring;
    if (h + DEPTH - 1 < h_end) load();
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (rotate) {
#pragma unroll
      for (int k = 0; k < C::R; ++k) rope_turn<HALVES>(x[k], c[k], s[k]);
    }
    // largest magnitude of the block: the bits of |x| order as integers, and
    // infinities and NaN come out on top
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < C::R; ++k)
#pragma unroll
      for (int e = 0; e < 8; e += 2) m = max_abs3(m, x[k][e], x[k][e + 1]);
    const int buf = (h - h_begin) & 1;
    auto over_block = [&](uint32_t bits) {
      bits = __reduce_max_sync(0xffffffffu, bits);
      if (lane == 0) part[buf][threadIdx.x >> 5] = bits;
      __syncthreads();
      return __reduce_max_sync(0xffffffffu, lane < warps ? part[buf][lane] : 0u);
    };
    uint32_t top = over_block(__float_as_uint(m) & 0x7FFFFFFFu);
    if (__builtin_expect(top >= 0x7F800000u, 0)) {  // infinities saturate, NaN becomes 0; reported
      if (rotate) {
        // this head's place in the ring is written again by the next head's load
        uint32_t at = (get == ring ? ring_end : get) - uint32_t(C::R) * pitch;
        const uint32_t turning = RopeSlot::turning(p.tab.slot[slot].runs);
#pragma unroll
        for (int k = 0; k < C::R; ++k, at += pitch) {
          uint32_t w[NW];
          float x0[8];
          slot_read<T>(w, at);
          slot_widen<T>(w, x0);
          rope_keep<HALVES>(x[k], x0, turning);
        }
      }
      uint32_t f = 0u;
#pragma unroll
      for (int k = 0; k < C::R; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t a = __float_as_uint(x[k][e]) & 0x7FFFFFFFu;
          f = max(f, a >= 0x7F800000u ? 0u : a);
        }
      __syncthreads();
      top = over_block(f);
      if (threadIdx.x == 0) set_status(p.status, SAFEDIT_ERR_INVALID_ARG);
      const float big = top ? __uint_as_float(top) : qmax;
#pragma unroll
      for (int k = 0; k < C::R; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = x[k][e];
          if (v != v)
            x[k][e] = 0.f;
          else if (fabsf(v) > big)
            x[k][e] = copysignf(big, v);
        }
    }
    const float most = top ? fmaxf(__uint_as_float(top), kLeastMax) : qmax;
    if (threadIdx.x == 0) *to_scale = most / qmax;
    // x qmax / most with one rounding: both sides by the power of two that
    // brings `most` into [1, 2) (exact), then Markstein's correction of
    // x * RN(1 / most).  With 16-bit rows the product x qmax is exact, so a
    // tie between two codes is met as one; x * (qmax / most) missed ties and
    // gave the neighbour.
    const uint32_t bits = __float_as_uint(most);
    const float m1 = __uint_as_float((bits & 0x007FFFFFu) | 0x3F800000u);
    // qmax 2^-exponent, exact
    const float up = __uint_as_float((uint32_t(127 + 6 + 127) << 23) - (bits & 0x7F800000u)) * (qmax / 64.f);
    const float inv = 1.f / m1;
    const uint64_t up2 = f2_pack(up, up), inv2 = f2_pack(inv, inv), neg2 = f2_pack(-m1, -m1);
#pragma unroll
    for (int k = 0; k < C::R; ++k) {
      if (first + k * C::RP >= p.state_rows) continue;
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const uint64_t a = f2_mul(f2_pack(x[k][e], x[k][e + 1]), up2);
        const uint64_t q = f2_mul(a, inv2);
        f2_unpack(f2_fma(f2_fma(q, neg2, a), inv2, q), y[e], y[e + 1]);
      }
      uint32_t o0, o1;
      if (p.e4m3) {
        o0 = pack_codes<true>(y[0], y[1], y[2], y[3]);
        o1 = pack_codes<true>(y[4], y[5], y[6], y[7]);
      } else {
        o0 = pack_codes<false>(y[0], y[1], y[2], y[3]);
        o1 = pack_codes<false>(y[4], y[5], y[6], y[7]);
      }
      uint8_t* row = to + k * c_rows;
      if constexpr (HALVES) {
        *reinterpret_cast<uint32_t*>(row + lo) = o0;
        *reinterpret_cast<uint32_t*>(row + hi) = o1;
      } else {
        *reinterpret_cast<uint2*>(row + lo) = make_uint2(o0, o1);
      }
    }
    to += c_sh;
    to_scale += p.f_sh[t];
  }
}

template <typename T, int BLOCK, bool HALVES>
static safedit_status launch_store(StoreParams& p, int64_t B, int64_t n_heads, int n_tensors, cudaStream_t s) {
  const int threads = StoreCfg<BLOCK>::RP * p.slots;
  const int64_t blocks = (int64_t(p.n_rows) + BLOCK - 1) / BLOCK;
  // Head groups by a count of 2048 threads an SM: each pays for the angles again
  // (25600 rows x 48 heads of 96, blocks of 64, when the call took 154 us: with twice
  // the groups 164, four times 193).  The registers of blocks of 32 and more admit
  // fewer (at d = 96 four blocks of 192 threads, or two from blocks of 64 on), so a
  // short call runs in more waves than this counts.
  const int64_t ctas = 148 * (2048 / threads);
  int64_t want = (ctas + blocks * B - 1) / (blocks * B);
  p.heads_per_group = int((n_heads + want - 1) / want);
  int64_t groups = 0;
  for (int t = 0; t < n_tensors; ++t) {
    groups += (p.heads[t] + p.heads_per_group - 1) / p.heads_per_group;
    p.group_end[t] = int(groups);
  }
  if (groups * blocks > INT32_MAX) return SAFEDIT_ERR_UNSUPPORTED;
  p.groups = int(groups);
  auto kern = state8_store_kernel<T, BLOCK, HALVES>;
  constexpr int kMost = kStoreDepth<T> * BLOCK * 128 * int(sizeof(T));
  static_assert(kMost <= 230000, "shared memory");
  const safedit_status st = set_smem(reinterpret_cast<const void*>(kern), kMost);
  if (st != SAFEDIT_OK) return st;
  const int ring_bytes = kStoreDepth<T> * BLOCK * p.slots * 8 * int(sizeof(T));
  kern<<<dim3(unsigned(blocks * groups), 1, unsigned(B)), threads, ring_bytes, s>>>(p);
  return after_launch(1);
}

template <typename T, bool HALVES>
static safedit_status store_by_block(StoreParams& p, int64_t B, int64_t n_heads, int n_tensors, int block, cudaStream_t s) {
  switch (block) {
    case 16: return launch_store<T, 16, HALVES>(p, B, n_heads, n_tensors, s);
    case 32: return launch_store<T, 32, HALVES>(p, B, n_heads, n_tensors, s);
    case 64: return launch_store<T, 64, HALVES>(p, B, n_heads, n_tensors, s);
    default: return launch_store<T, 128, HALVES>(p, B, n_heads, n_tensors, s);
  }
}

template <typename T>
static safedit_status store_by_form(StoreParams& p, int64_t B, int64_t n_heads, int n_tensors, int block, bool halves,
                                    cudaStream_t s) {
  return halves ? store_by_block<T, true>(p, B, n_heads, n_tensors, block, s)
                : store_by_block<T, false>(p, B, n_heads, n_tensors, block, s);
}

}  // namespace sd

using namespace sd;

extern "C" safedit_status safedit_state8_store(const safedit_tensor* src, const safedit_tensor* codes,
                                               const safedit_tensor* scales, int32_t n_tensors, int32_t block,
                                               int64_t row0, const int32_t* d_idx, int32_t n_idx,
                                               int32_t src_indexed, const int32_t* host_rotate,
                                               const safedit_tensor* pos, const safedit_rope* rope, void* stream) {
  if (!src || !codes || !scales || n_tensors < 1 || n_tensors > kMaxStoreTensors) return SAFEDIT_ERR_INVALID_ARG;
  if ((src_indexed != 0 && src_indexed != 1) || row0 < 0) return SAFEDIT_ERR_INVALID_ARG;
  if (d_idx ? n_idx < 0 : src_indexed) return SAFEDIT_ERR_INVALID_ARG;
  if (!state8_block_ok(block)) return SAFEDIT_ERR_UNSUPPORTED;
  if (row0 % block != 0) return SAFEDIT_ERR_ALIGNMENT;
  StoreParams p{};
  safedit_status st;
  int64_t B = -1, d = -1, n = -1, N = -1, heads = 0;
  for (int t = 0; t < n_tensors; ++t) {
    const safedit_tensor &x = src[t], &c = codes[t], &f = scales[t];
    if ((st = check_tensor(&x, 4)) != SAFEDIT_OK) return st;
    if ((st = check_codes(&c)) != SAFEDIT_OK) return st;
    if ((st = check_scales(&f, &c, block)) != SAFEDIT_OK) return st;
    if (x.dtype != SAFEDIT_BF16 && x.dtype != SAFEDIT_F16 && x.dtype != SAFEDIT_F32) return SAFEDIT_ERR_DTYPE;
    if (x.dtype != src[0].dtype || c.dtype != codes[0].dtype) return SAFEDIT_ERR_DTYPE;
    if (t == 0) B = x.dims[0], d = x.dims[3], n = d_idx ? int64_t(n_idx) : x.dims[2], N = c.dims[2];
    if (x.dims[0] != B || c.dims[0] != B || x.dims[3] != d || c.dims[3] != d || c.dims[1] != x.dims[1] ||
        c.dims[2] != N || (!src_indexed && x.dims[2] != n))
      return SAFEDIT_ERR_SHAPE;
    const int64_t vec = 16 / elt_size(x.dtype);
    if (x.strides[3] != 1 || !aligned16(x.data)) return SAFEDIT_ERR_ALIGNMENT;
    for (int k = 0; k < 3; ++k)
      if (x.strides[k] % vec != 0 || x.strides[k] < 0) return SAFEDIT_ERR_ALIGNMENT;
    heads += x.dims[1];
    if (heads > INT32_MAX / 2) return SAFEDIT_ERR_SHAPE;
    p.src[t] = x.data;
    p.code[t] = static_cast<uint8_t*>(c.data);
    p.scale[t] = static_cast<float*>(f.data);
    p.s_sb[t] = x.strides[0], p.s_sh[t] = x.strides[1], p.s_sr[t] = x.strides[2];
    p.c_sb[t] = c.strides[0], p.c_sh[t] = c.strides[1], p.c_sr[t] = c.strides[2];
    p.f_sb[t] = f.strides[0], p.f_sh[t] = f.strides[1];
    p.heads[t] = int(x.dims[1]);
    p.rotate[t] = host_rotate ? host_rotate[t] : 0;
    if (p.rotate[t] != 0 && p.rotate[t] != 1) return SAFEDIT_ERR_INVALID_ARG;
    p.any_rotate |= p.rotate[t];
  }
  if (d != 64 && d != 96 && d != 128) return SAFEDIT_ERR_UNSUPPORTED;
  if (row0 > N || n > N - row0 || N > INT32_MAX - 128) return SAFEDIT_ERR_SHAPE;
  if (B > 65535) return SAFEDIT_ERR_UNSUPPORTED;
  p.limit = INT32_MAX;
  if (p.any_rotate) {
    int64_t tokens = 0;
    if ((st = rope_setup(rope, pos, B, d, &p.tab, &p.pos, &tokens)) != SAFEDIT_OK) return st;
    if (rope->inverse) return SAFEDIT_ERR_INVALID_ARG;
    if (!d_idx && tokens < n) return SAFEDIT_ERR_SHAPE;
    p.limit = tokens;
  }
  if (src_indexed)
    for (int t = 0; t < n_tensors; ++t)
      if (src[t].dims[2] < p.limit) p.limit = src[t].dims[2];
  if (n == 0 || B == 0 || heads == 0) return SAFEDIT_OK;
  p.slots = int(d / 8);
  p.e4m3 = codes[0].dtype == SAFEDIT_E4M3;
  p.n_rows = int(n);
  p.row0 = int(row0);
  p.state_rows = int(N);
  p.idx = src_indexed || p.any_rotate ? d_idx : nullptr;  // nothing else reads it
  p.src_indexed = src_indexed;
  p.status = status_ptr();
  if (!p.status) return SAFEDIT_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool halves = p.any_rotate && rope->halves;
  switch (src[0].dtype) {
    case SAFEDIT_BF16: return store_by_form<__nv_bfloat16>(p, B, heads, n_tensors, block, halves, s);
    case SAFEDIT_F16: return store_by_form<__half>(p, B, heads, n_tensors, block, halves, s);
    default: return store_by_form<float>(p, B, heads, n_tensors, block, halves, s);
  }
}
