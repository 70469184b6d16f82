// rope.cu -- rows rotated at their tokens' positions on several axes.
//
//   (x, y) -> (x cos a - y sin a, x sin a + y cos a),
//   a = pos[b, i, axis] * theta_axis^(-2 m / s)
//
// Bound by memory: 2 * element size bytes for each element against three
// operations.  A thread owns one slot (four pairs) of one row and walks the
// heads of every tensor with it, so the fp64 angle reduction and the sine and
// cosine are paid once for all heads of Q and K, not once for each.  Heads go
// in groups over blockIdx.y, as few groups as still fill the GPU.  Q and K of
// 4096 tokens x 48 heads of 96 out of the fused projection (151 MB): 27.6 us
// in the kernel, 5.5 TB/s; 25600 tokens: 172 us, 5.5 TB/s.  Angles in 64-bit
// fixed point with a Taylor series in place of fp64 and sincospif measured no
// faster.
#include <cmath>
#include <type_traits>

#include <cuda_fp16.h>

#include "rope.cuh"

namespace sd {

safedit_status rope_setup(const safedit_rope* rope, const safedit_tensor* pos, int64_t B, int64_t d, RopeTable* tab,
                          RopePos* view, int64_t* tokens) {
  if (!rope) return SAFEDIT_ERR_INVALID_ARG;
  const int A = rope->n_axes;
  if (A < 1 || A > kMaxAxes) return SAFEDIT_ERR_INVALID_ARG;
  if ((rope->halves != 0 && rope->halves != 1) || (rope->inverse != 0 && rope->inverse != 1))
    return SAFEDIT_ERR_INVALID_ARG;
  safedit_status st = check_tensor(pos, 3);
  if (st != SAFEDIT_OK) return st;
  if (pos->dtype != SAFEDIT_I32 && pos->dtype != SAFEDIT_F32) return SAFEDIT_ERR_DTYPE;
  if ((pos->dims[0] != 1 && pos->dims[0] != B) || pos->dims[2] != A) return SAFEDIT_ERR_SHAPE;
  int64_t sum = 0;
  for (int a = 0; a < A; ++a) {
    const int64_t s = rope->axis_dim[a];
    if (s < 1) return SAFEDIT_ERR_INVALID_ARG;
    if (s % (rope->halves ? 8 : 2) != 0) return SAFEDIT_ERR_UNSUPPORTED;
    if (!(rope->theta[a] >= 1.0) || !std::isfinite(rope->theta[a])) return SAFEDIT_ERR_INVALID_ARG;
    sum += s;
  }
  if (sum > d) return SAFEDIT_ERR_SHAPE;
  constexpr long double kInv2Pi = 0.15915494309189533577L;
  const int halves = rope->halves;
  int at = 0, pair = 0;
  auto set = [&](int p, double turn, int axis, int lo, int hi) {
    RopeSlot& sl = tab->slot[p / 4];
    sl.turn[p % 4] = turn;
    sl.axes = (p % 4 ? sl.axes : 0u) | uint32_t(axis) << (8 * (p % 4));
    sl.runs = (p % 4 ? sl.runs : RopeSlot::pack(lo, hi)) | uint32_t(turn != 0.0) << (16 + p % 4);
  };
  for (int a = 0; a < A; ++a) {
    const int s = rope->axis_dim[a];
    // In more than fp64 where the host has it: in fp64 the steps of a segment of 256
    // add up to 2^-48.6 of a radian per unit of position, 5e-6 at 2^31.
    // The step is fp64's, corrected by one Newton step on step^(s/2) = 1 / theta (a
    // power in long double takes 0.3 us, fifteen times what this adds).
    long double step = std::pow(rope->theta[a], -2.0 / s), power = 1.0L, square = step;
    for (int e = s / 2; e; e >>= 1, square *= square)
      if (e & 1) power *= square;
    step *= 1.0L + (1.0L / (power * rope->theta[a]) - 1.0L) * (2.0L / s);
    long double f = 1.0L;
    for (int m = 0; m < s / 2; ++m, ++pair, f *= step) {
      set(pair, double(f * kInv2Pi), a, halves ? at + m : at + 2 * m, halves ? at + m + s / 2 : at + 2 * m + 4);
    }
    at += s;
  }
  // the rest of the row: pairs that do not turn, 8 consecutive elements a slot
  for (; pair < d / 2; ++pair) {
    set(pair, 0.0, 0, 2 * pair, 2 * pair + 4);
  }
  view->pos = pos->data;
  view->f32 = pos->dtype == SAFEDIT_F32;
  view->sb = pos->dims[0] == 1 ? 0 : pos->strides[0];
  view->st = pos->strides[1];
  view->sa = pos->strides[2];
  *tokens = pos->dims[1];
  return SAFEDIT_OK;
}

constexpr int kMaxRopeTensors = 4;
constexpr int kRopeThreads = 256;
// heads whose loads are in flight in one thread: 128 bytes of them
template <typename T>
constexpr int kRopeFlight = sizeof(T) == 4 ? 4 : 8;

struct RopeParams {
  RopeTable tab;
  RopePos pos;
  const void* src[kMaxRopeTensors];
  void* dst[kMaxRopeTensors];
  int64_t s_sb[kMaxRopeTensors], s_sh[kMaxRopeTensors], s_sr[kMaxRopeTensors];
  int64_t d_sb[kMaxRopeTensors], d_sh[kMaxRopeTensors], d_sr[kMaxRopeTensors];
  int head_end[kMaxRopeTensors];  // heads of tensors 0..t together
  int n_heads, heads_per_group, slots;
  int64_t n_rows, limit;  // rows of the call; tokens an index may name
  const int* idx;
  int src_indexed, dst_indexed;
  float sign;
  int* status;
};

template <typename T, bool HALVES>
__global__ void __launch_bounds__(kRopeThreads) rope_rows_kernel(const __grid_constant__ RopeParams p) {
  const int64_t u = int64_t(blockIdx.x) * kRopeThreads + threadIdx.x;
  const int64_t r = u / p.slots;
  const int slot = int(u - r * p.slots);
  if (r >= p.n_rows) return;
  const int b = blockIdx.z;
  int64_t i = r;
  if (p.idx) {
    i = __ldg(p.idx + r);
    if (i < 0 || i >= p.limit) {
      set_status(p.status, SAFEDIT_ERR_INDEX);
      return;
    }
  }
  const RopeSlot& sl = p.tab.slot[slot];
  const uint32_t runs = sl.runs, turning = RopeSlot::turning(runs);
  const int lo = RopeSlot::lo(runs), hi = RopeSlot::hi(runs);
  const int64_t rs = p.src_indexed ? i : r, rd = p.dst_indexed ? i : r;
  const int h_end = min(p.n_heads, int(blockIdx.y + 1) * p.heads_per_group);
  constexpr int F = kRopeFlight<T>;
  uint32_t w[F][SlotWords<T>::N];
  auto load = [&](int h0) {
#pragma unroll
    for (int e = 0; e < F; ++e) {
      const int hh = h0 + e;
      if (hh >= h_end) break;
      int t = 0;
      while (hh >= p.head_end[t]) ++t;
      const int h = t ? hh - p.head_end[t - 1] : hh;
      slot_load<T, HALVES>(w[e], static_cast<const T*>(p.src[t]) + b * p.s_sb[t] + h * p.s_sh[t] + rs * p.s_sr[t], lo, hi);
    }
  };
  load(blockIdx.y * p.heads_per_group);  // on their way while the angles are taken
  float c[4], s[4];
  rope_angles(sl, p.pos, b, i, p.sign, c, s);
  for (int h0 = blockIdx.y * p.heads_per_group; h0 < h_end; h0 += F) {
#pragma unroll
    for (int e = 0; e < F; ++e) {
      const int hh = h0 + e;
      if (hh >= h_end) break;
      int t = 0;
      while (hh >= p.head_end[t]) ++t;
      const int h = t ? hh - p.head_end[t - 1] : hh;
      T* const to = static_cast<T*>(p.dst[t]) + b * p.d_sb[t] + h * p.d_sh[t] + rd * p.d_sr[t];
      float x[8];
      slot_widen<T>(w[e], x);
      rope_turn<HALVES>(x, c, s, turning);
      if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(to + lo) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(to + hi) = make_float4(x[4], x[5], x[6], x[7]);
      } else {
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            o[k] = pack_bf16x2(x[2 * k], x[2 * k + 1]);
          } else {
            const __half2 y = __floats2half2_rn(x[2 * k], x[2 * k + 1]);
            o[k] = *reinterpret_cast<const uint32_t*>(&y);
          }
        }
        if constexpr (HALVES) {
          *reinterpret_cast<uint2*>(to + lo) = make_uint2(o[0], o[1]);
          *reinterpret_cast<uint2*>(to + hi) = make_uint2(o[2], o[3]);
        } else {
          *reinterpret_cast<uint4*>(to + lo) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
    if (h0 + F < h_end) load(h0 + F);
  }
}

template <typename T>
static safedit_status launch_rope(const RopeParams& p, dim3 grid, bool halves, cudaStream_t s) {
  if (halves)
    rope_rows_kernel<T, true><<<grid, kRopeThreads, 0, s>>>(p);
  else
    rope_rows_kernel<T, false><<<grid, kRopeThreads, 0, s>>>(p);
  return after_launch(1);
}

}  // namespace sd

using namespace sd;

extern "C" safedit_status safedit_rope_rows(const safedit_tensor* src, const safedit_tensor* dst, int32_t n_tensors,
                                            const safedit_tensor* pos, const safedit_rope* rope,
                                            const int32_t* d_idx, int32_t n_idx, int32_t src_indexed,
                                            int32_t dst_indexed, void* stream) {
  if (!src || !dst || n_tensors < 1 || n_tensors > kMaxRopeTensors) return SAFEDIT_ERR_INVALID_ARG;
  if ((src_indexed != 0 && src_indexed != 1) || (dst_indexed != 0 && dst_indexed != 1)) return SAFEDIT_ERR_INVALID_ARG;
  if (d_idx ? n_idx < 0 : (src_indexed || dst_indexed)) return SAFEDIT_ERR_INVALID_ARG;
  RopeParams p{};
  safedit_status st;
  int64_t B = -1, d = -1, n = -1, heads = 0;
  for (int t = 0; t < n_tensors; ++t) {
    const safedit_tensor &s = src[t], &o = dst[t];
    if ((st = check_tensor(&s, 4)) != SAFEDIT_OK) return st;
    if ((st = check_tensor(&o, 4)) != SAFEDIT_OK) return st;
    if (s.dtype != SAFEDIT_BF16 && s.dtype != SAFEDIT_F16 && s.dtype != SAFEDIT_F32) return SAFEDIT_ERR_DTYPE;
    if (o.dtype != s.dtype || s.dtype != src[0].dtype) return SAFEDIT_ERR_DTYPE;
    if (t == 0) B = s.dims[0], d = s.dims[3], n = d_idx ? int64_t(n_idx) : s.dims[2];
    if (d < 8 || d % 8 != 0 || d > 2 * kMaxPairs) return SAFEDIT_ERR_UNSUPPORTED;
    if (s.dims[0] != B || o.dims[0] != B || s.dims[3] != d || o.dims[3] != d || o.dims[1] != s.dims[1])
      return SAFEDIT_ERR_SHAPE;
    if (!src_indexed && s.dims[2] != n) return SAFEDIT_ERR_SHAPE;
    if (!dst_indexed && o.dims[2] != n) return SAFEDIT_ERR_SHAPE;
    const int64_t vec = 16 / elt_size(s.dtype);
    for (const safedit_tensor* x : {&s, &o}) {
      if (x->strides[3] != 1 || !aligned16(x->data)) return SAFEDIT_ERR_ALIGNMENT;
      for (int k = 0; k < 3; ++k)
        if (x->strides[k] % vec != 0 || x->strides[k] < 0) return SAFEDIT_ERR_ALIGNMENT;
    }
    heads += s.dims[1];
    p.src[t] = s.data;
    p.dst[t] = o.data;
    p.s_sb[t] = s.strides[0], p.s_sh[t] = s.strides[1], p.s_sr[t] = s.strides[2];
    p.d_sb[t] = o.strides[0], p.d_sh[t] = o.strides[1], p.d_sr[t] = o.strides[2];
    if (heads > INT32_MAX / 2) return SAFEDIT_ERR_SHAPE;
    p.head_end[t] = int(heads);
  }
  int64_t tokens = 0;
  if ((st = rope_setup(rope, pos, B, d, &p.tab, &p.pos, &tokens)) != SAFEDIT_OK) return st;
  if (!d_idx && tokens < n) return SAFEDIT_ERR_SHAPE;
  p.limit = tokens;
  for (int t = 0; t < n_tensors; ++t) {
    if (src_indexed && src[t].dims[2] < p.limit) p.limit = src[t].dims[2];
    if (dst_indexed && dst[t].dims[2] < p.limit) p.limit = dst[t].dims[2];
  }
  if (B > 65535) return SAFEDIT_ERR_UNSUPPORTED;
  p.slots = int(d / 8);
  const int64_t blocks = (n * p.slots + kRopeThreads - 1) / kRopeThreads;
  if (n > INT32_MAX || blocks > INT32_MAX) return SAFEDIT_ERR_UNSUPPORTED;
  if (n == 0 || B == 0 || heads == 0) return SAFEDIT_OK;
  p.n_rows = n;
  p.n_heads = int(heads);
  p.idx = d_idx;
  p.src_indexed = src_indexed;
  p.dst_indexed = dst_indexed;
  p.sign = rope->inverse ? -1.f : 1.f;
  p.status = status_ptr();
  if (!p.status) return SAFEDIT_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d_idx && dst_indexed && index_check_enabled() &&
      (st = launch_index_check(d_idx, int32_t(n), p.limit, p.status, s)) != SAFEDIT_OK)
    return st;
  // as few head groups as still give every SM eight blocks: each group pays
  // for the angles again, and few large blocks leave SMs idle at the end (4915
  // rows x 64 heads of 128: two blocks 41-43 us, four 41, eight 37, sixteen 40)
  const int64_t want = (8 * 148 + blocks * B - 1) / (blocks * B);
  int64_t groups = (heads + 3) / 4;
  if (groups > want) groups = want;
  p.heads_per_group = int((heads + groups - 1) / groups);
  groups = (heads + p.heads_per_group - 1) / p.heads_per_group;
  if (groups > 65535) return SAFEDIT_ERR_UNSUPPORTED;
  const dim3 grid{unsigned(blocks), unsigned(groups), unsigned(B)};
  switch (src[0].dtype) {
    case SAFEDIT_BF16: return launch_rope<__nv_bfloat16>(p, grid, rope->halves, s);
    case SAFEDIT_F16: return launch_rope<__half>(p, grid, rope->halves, s);
    default: return launch_rope<float>(p, grid, rope->halves, s);
  }
}
