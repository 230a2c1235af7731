// Routing of tokens to experts from their logits, and its gradient.
//
// Forward, per token (row) with logits l over E experts and the balance bias b:
//   s = softmax(l) or sigmoid(l)          the scores
//   c = s + b                              what selects (without b: l itself,
//                                          whose order is that of s)
//   groups of E / G consecutive experts, each ranked by its largest c or the
//   sum of its two largest; the best `kept` groups stay in the choice
//   idx = the k largest c, larger first, the lower expert on ties
//   w_j = scale * s_j, or scale * s_j / sum of the kept s
// Backward: with a_i the share of slot i (s_i over the kept sum) and g the
// gradient of w,
//   softmax:               dl_e = scale p_e (g_e - sum_i g_i p_i)
//   softmax, renormalised: dl_j = scale a_j (g_j - sum_i g_i a_i), others 0
//   sigmoid:               dl_j = scale g_j s_j (1 - s_j),          others 0
//   sigmoid, renormalised: dl_j = scale a_j (1 - s_j) (g_j - sum_i g_i a_i)
//
// One warp per row, its E logits in registers, lane i holding the VPL
// consecutive experts from i VPL: the lowest lane with the maximum is the
// lowest expert, so a selection round is one warp-wide integer maximum, one
// ballot and one shuffle.  Scores and sums are fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <new>
#include <type_traits>

#include "error.h"
#include "moe.h"

namespace {

constexpr int kMaxE = 256;
constexpr int kMaxK = 16;
constexpr int kMaxGroups = 32;
constexpr int kWarps = 8;           // rows a block works on at a time
constexpr int kGridCap = 152 * 8;   // blocks that fill the SMs; longer batches loop
constexpr unsigned kAll = 0xffffffffu;

struct Route {
  int E, k, score, groups, kept, group_score, renorm;
  float scale;
};

// Unsigned order of floats: larger value, larger key; NaN above everything,
// both zeros equal.  Keys up to kDead are -inf or nothing: never chosen.
constexpr uint32_t kDead = 0x007fffffu;

__device__ __forceinline__ uint32_t key_of(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t u = __float_as_uint(v + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t key) {
  if (key == 0xffffffffu) return __uint_as_float(0x7fffffffu);
  return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_float(float v, float* o) { *o = v; }
__device__ __forceinline__ void from_float(float v, __nv_bfloat16* o) { *o = __float2bfloat16(v); }

// VPL consecutive values from element e0 of a row; -inf past E.  VEC: E is a
// multiple of VPL and every row is aligned to VPL elements (at most 16 bytes).
template <typename L, int VPL, bool VEC>
__device__ __forceinline__ void load_row(const L* row, int e0, int E, float (&v)[VPL]) {
  if (VEC && e0 < E) {
    constexpr int bytes = VPL * sizeof(L) < 16 ? VPL * sizeof(L) : 16;
    constexpr int n = VPL * sizeof(L) / bytes;
    union {
      L l[VPL];
      uint4 q[n];
      uint2 d[1];
      uint32_t s;
    } u;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      if constexpr (bytes == 16) u.q[i] = __ldg(reinterpret_cast<const uint4*>(row + e0) + i);
      else if constexpr (bytes == 8) u.d[0] = __ldg(reinterpret_cast<const uint2*>(row + e0));
      else if constexpr (bytes == 4) u.s = __ldg(reinterpret_cast<const uint32_t*>(row + e0));
      else u.l[0] = row[e0];
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = to_float(u.l[i]);
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = e0 + i < E ? to_float(row[e0 + i]) : -INFINITY;
  }
}

template <typename L, int VPL, bool VEC>
__device__ __forceinline__ void store_row(L* row, int e0, int E, const float (&v)[VPL]) {
  if (VEC && e0 < E) {
    constexpr int bytes = VPL * sizeof(L) < 16 ? VPL * sizeof(L) : 16;
    constexpr int n = VPL * sizeof(L) / bytes;
    union {
      L l[VPL];
      uint4 q[n];
      uint2 d[1];
      uint32_t s;
    } u;
#pragma unroll
    for (int i = 0; i < VPL; ++i) from_float(v[i], &u.l[i]);
#pragma unroll
    for (int i = 0; i < n; ++i) {
      if constexpr (bytes == 16) reinterpret_cast<uint4*>(row + e0)[i] = u.q[i];
      else if constexpr (bytes == 8) *reinterpret_cast<uint2*>(row + e0) = u.d[0];
      else if constexpr (bytes == 4) *reinterpret_cast<uint32_t*>(row + e0) = u.s;
      else row[e0] = u.l[0];
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (e0 + i < E) from_float(v[i], row + e0 + i);
  }
}

// Softmax of the row held VPL a lane: p over v in place (0 where v is -inf);
// a row of -inf alone gives zeros.
template <int VPL>
__device__ __forceinline__ void row_softmax(float (&v)[VPL], float* top, float* inv) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) m = fmaxf(m, v[i]);
  m = warp_max(m);
  const float base = m == -INFINITY ? 0.f : m;
  float z = 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    v[i] = expf(v[i] - base);
    z += v[i];
  }
  z = warp_sum(z);
  *top = base;
  *inv = z == 0.f ? 0.f : 1.f / z;
#pragma unroll
  for (int i = 0; i < VPL; ++i) v[i] *= *inv;
}

__device__ __forceinline__ float sigmoid(float l) {
  const float e = expf(-fabsf(l));
  const float r = 1.f / (1.f + e);
  return l < 0.f ? e * r : l == l ? r : l;
}

// A kept slot's unnormalised share, the same factor off in all slots of the
// row: exp(l - m) for the softmax; for the sigmoid s / e^m with m = min(0,
// largest kept l), so that far negative logits keep their ratios.
__device__ __forceinline__ float share_of(int score, float l, float m) {
  if (score == MOE_SCORE_SOFTMAX) return expf(l - m);
  return l > 0.f ? 1.f / (1.f + expf(-l)) : expf(l - m) / (1.f + expf(l));
}

__device__ __forceinline__ float share_base(int score, float l, bool live) {
  const float m = warp_max(live ? l : -INFINITY);
  return score == MOE_SCORE_SOFTMAX ? m : fminf(m, 0.f);
}

template <typename L, int VPL, bool VEC>
__global__ void __launch_bounds__(kWarps * 32)
    route_forward(Route r, int T, const L* __restrict__ logits, long long stride,
                  const float* __restrict__ bias, int* __restrict__ idx, float* __restrict__ w,
                  int* __restrict__ counts) {
  __shared__ float s_level[kWarps][32 * VPL];
  __shared__ int s_count[kMaxE];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = r.E, k = r.k, e0 = lane * VPL;
  const int gs = E / r.groups;
  if (counts) {
    for (int e = threadIdx.x; e < E; e += kWarps * 32) s_count[e] = 0;
    __syncthreads();
  }
  float b[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) b[i] = bias && e0 + i < E ? __ldg(bias + e0 + i) : 0.f;
  // groups: `per` lanes walk each group; which group this lane's experts are in
  int per = 32;
  while (per * r.groups > 32) per >>= 1;
  const int my_group = lane / per, sub = lane & (per - 1);
  int in_group[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) in_group[i] = e0 + i < E ? (e0 + i) / gs : 0;
  const bool top2 = r.group_score == MOE_GROUP_TOP2;
  const bool by_level = r.groups > 1;
  const bool level_of_scores = by_level && top2;
  const bool need_p = r.score == MOE_SCORE_SOFTMAX && (!r.renorm || bias || level_of_scores);

  for (long long t = (long long)blockIdx.x * kWarps + warp; t < T; t += (long long)gridDim.x * kWarps) {
    const L* row = logits + t * stride;
    float l[VPL], s[VPL];
    load_row<L, VPL, VEC>(row, e0, E, l);
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] = l[i];
    float top = 0.f, inv = 0.f;
    if (need_p) {
      row_softmax<VPL>(s, &top, &inv);
    } else if (r.score == MOE_SCORE_SIGMOID && (bias || level_of_scores)) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) s[i] = sigmoid(l[i]);
    }
    uint32_t key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = l[i] == -INFINITY ? 0u : key_of(bias ? s[i] + b[i] : l[i]);
    if (by_level) {
      // the value each expert gives its group: c, s without a bias, or l where
      // the largest alone counts
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        s_level[warp][e0 + i] =
            key[i] == 0u ? -INFINITY : bias ? s[i] + b[i] : level_of_scores ? s[i] : l[i];
      __syncwarp();
      uint32_t m1 = 0u, m2 = 0u;
      if (my_group < r.groups) {
        // start each group elsewhere, so that groups of 32 experts read other banks
        const int n = (gs - sub + per - 1) / per;
        for (int i = 0, at = n > 0 ? my_group % n : 0; i < n; ++i, at = at + 1 == n ? 0 : at + 1) {
          const uint32_t v = key_of(s_level[warp][my_group * gs + sub + at * per]);
          m2 = max(m2, min(m1, v));
          m1 = max(m1, v);
        }
      }
      for (int o = per >> 1; o; o >>= 1) {
        const uint32_t o1 = __shfl_xor_sync(kAll, m1, o), o2 = __shfl_xor_sync(kAll, m2, o);
        m2 = max(max(m2, o2), min(m1, o1));
        m1 = max(m1, o1);
      }
      uint32_t level = m1;
      if (top2 && m1 > kDead && m2 > kDead) level = key_of(value_of(m1) + value_of(m2));
      int rank = 0;
      for (int g = 0; g < r.groups; ++g) {
        const uint32_t o = __shfl_sync(kAll, level, g * per);
        rank += o > level || (o == level && g < my_group);
      }
      const unsigned kept = __ballot_sync(kAll, rank < r.kept && my_group < r.groups);
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (!(kept >> (in_group[i] * per) & 1u)) key[i] = 0u;
      __syncwarp();
    }
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) best = max(best, key[i]);
    int my_e = -1;          // lane j: slot j's expert
    for (int j = 0; j < k; ++j) {
      const uint32_t m = __reduce_max_sync(kAll, best);
      if (m <= kDead) break;
      const int from = __ffs(__ballot_sync(kAll, best == m)) - 1;
      int e = 0;
      if (lane == from) {
        bool found = false;
        best = 0u;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          if (!found && key[i] == m) {
            found = true;
            e = e0 + i;
            key[i] = 0u;
          }
          best = max(best, key[i]);
        }
      }
      e = __shfl_sync(kAll, e, from);
      if (lane == j) my_e = e;
    }
    const bool live = my_e >= 0;
    const float lj = live ? to_float(row[my_e]) : -INFINITY;
    float wj = 0.f;
    if (r.renorm) {
      const float m = share_base(r.score, lj, live);
      const float a = live ? share_of(r.score, lj, m) : 0.f;
      const float z = warp_sum(a);
      if (live) wj = a / z;
    } else if (live) {
      wj = r.score == MOE_SCORE_SOFTMAX ? expf(lj - top) * inv : sigmoid(lj);
    }
    if (lane < k) {
      idx[t * k + lane] = my_e;
      w[t * k + lane] = live ? r.scale * wj : 0.f;
      if (counts && live) atomicAdd(&s_count[my_e], 1);
    }
  }
  if (counts) {
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kWarps * 32) {
      if (gridDim.x == 1) counts[e] = s_count[e];
      else if (s_count[e]) atomicAdd(counts + e, s_count[e]);
    }
  }
}

template <typename L, int VPL, bool VEC>
__global__ void __launch_bounds__(kWarps * 32)
    route_backward(Route r, int T, const L* __restrict__ logits, long long stride,
                   const int* __restrict__ idx, const float* __restrict__ grad_w,
                   L* __restrict__ grad, long long grad_stride) {
  __shared__ float s_row[kWarps][32 * VPL];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = r.E, k = r.k, e0 = lane * VPL;
  for (long long t = (long long)blockIdx.x * kWarps + warp; t < T; t += (long long)gridDim.x * kWarps) {
    const L* row = logits + t * stride;
    int e = lane < k ? idx[t * k + lane] : -1;
    const bool live = (unsigned)e < (unsigned)E;
    if (!live) e = -1 - lane;  // no two dead slots alike
    const float g = live ? grad_w[t * k + lane] : 0.f;
    const float lj = live ? to_float(row[e]) : -INFINITY;
    float v[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = 0.f;
    float add = 0.f;  // what slot `lane` adds to its expert's gradient
    if (r.renorm) {
      const float m = share_base(r.score, lj, live);
      float a = live ? share_of(r.score, lj, m) : 0.f;
      const float z = warp_sum(a);
      a = live ? a / z : 0.f;
      const float dot = warp_sum(live ? g * a : 0.f);
      if (live) add = r.scale * a * (g - dot);
      if (r.score == MOE_SCORE_SIGMOID) add *= sigmoid(-lj);
    } else if (r.score == MOE_SCORE_SIGMOID) {
      if (live) add = r.scale * g * sigmoid(lj) * sigmoid(-lj);
    } else {
      float top, inv;
      load_row<L, VPL, VEC>(row, e0, E, v);
      row_softmax<VPL>(v, &top, &inv);
      add = live ? r.scale * g * expf(lj - top) * inv : 0.f;
      const float dot = warp_sum(add);
#pragma unroll
      for (int i = 0; i < VPL; ++i) v[i] = -v[i] * dot;
    }
    if (!live) add = 0.f;
    // an expert named by several slots gets their sum, in slot order
    const unsigned same = __match_any_sync(kAll, e);
    if (__any_sync(kAll, live && (same & (same - 1)))) {
      float sum = 0.f;
      for (int j = 0; j < k; ++j) {
        const float o = __shfl_sync(kAll, add, j);
        if (same >> j & 1u) sum += o;
      }
      add = sum;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) s_row[warp][e0 + i] = v[i];
    __syncwarp();
    if (live && lane == __ffs(same) - 1) s_row[warp][e] += add;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = s_row[warp][e0 + i];
    store_row<L, VPL, VEC>(grad + t * grad_stride, e0, E, v);
    __syncwarp();
  }
}

int vpl_of(int E) {
  int v = 1;
  while (v * 32 < E) v <<= 1;
  return v;
}

bool rows_aligned(const void* p, long long stride, size_t size, int vpl) {
  const size_t a = size * vpl < 16 ? size * vpl : 16;
  return reinterpret_cast<uintptr_t>(p) % a == 0 && (size_t)stride * size % a == 0;
}

int blocks_of(int T) {
  const long long n = ((long long)T + kWarps - 1) / kWarps;
  return (int)(n < kGridCap ? n : kGridCap);
}

template <typename... A>
cudaError_t launch(void (*kernel)(A...), int T, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks_of(T));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// f(element type, experts per lane) for a router of E experts.
template <typename L, typename F>
cudaError_t by_vpl(int E, F&& f) {
  switch (vpl_of(E)) {
    case 1: return f(L{}, std::integral_constant<int, 1>{});
    case 2: return f(L{}, std::integral_constant<int, 2>{});
    case 4: return f(L{}, std::integral_constant<int, 4>{});
    default: return f(L{}, std::integral_constant<int, 8>{});
  }
}

}  // namespace

struct moe_router {
  Route r;
};

namespace {

size_t type_size(int type) { return type == MOE_TYPE_F32 ? 4 : 2; }

int check_logits(const moe_router* r, int T, const void* logits, int type, long long stride) {
  if (!r) return moe::set_error(MOE_E_INVAL, "null router handle");
  if (T < 0) return moe::set_error(MOE_E_INVAL, "T must not be negative");
  if (type != MOE_TYPE_F32 && type != MOE_TYPE_BF16)
    return moe::set_error(MOE_E_INVAL, "logits are MOE_TYPE_F32 or MOE_TYPE_BF16");
  if (T == 0) return MOE_OK;
  if (!logits) return moe::set_error(MOE_E_INVAL, "null logits");
  if (reinterpret_cast<uintptr_t>(logits) % type_size(type))
    return moe::set_error(MOE_E_INVAL, "logits must be aligned to their type");
  if (stride < r->r.E) return moe::set_error(MOE_E_INVAL, "rows of logits overlap: the row stride is below E");
  return MOE_OK;
}

bool aligned4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

}  // namespace

extern "C" {

moe_router_t* moe_router_create(int E, int k, int score, int groups, int groups_kept, int group_score,
                                int renormalise, float scale) {
  const char* bad = nullptr;
  if (E < 1 || E > kMaxE || k < 1 || k > E || k > kMaxK) bad = "need 1 <= k <= E <= 256 and k <= 16";
  else if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) bad = "score must be MOE_SCORE_*";
  else if (groups < 1 || groups > kMaxGroups || E % groups != 0) bad = "groups must divide E, 1 to 32 of them";
  else if (groups_kept < 1 || groups_kept > groups) bad = "need 1 <= groups_kept <= groups";
  else if (k > E / groups * groups_kept) bad = "k exceeds the experts of the kept groups";
  else if (group_score != MOE_GROUP_MAX && group_score != MOE_GROUP_TOP2) bad = "group_score must be MOE_GROUP_*";
  else if (renormalise != 0 && renormalise != 1) bad = "renormalise must be 0 or 1";
  else if (!isfinite(scale)) bad = "scale must be finite";
  if (bad) {
    moe::set_error(MOE_E_INVAL, bad);
    return nullptr;
  }
  moe_router_t* h = new (std::nothrow) moe_router();
  if (!h) {
    moe::set_error(MOE_E_NOMEM, "out of host memory");
    return nullptr;
  }
  h->r = Route{E, k, score, groups, groups_kept, group_score, renormalise, scale};
  moe::clear_error();
  return h;
}

void moe_router_destroy(moe_router_t* h) { delete h; }

int moe_router_forward(const moe_router_t* h, int T, const void* logits, int logits_type,
                       long long row_stride, const float* bias, int32_t* idx, float* w,
                       int32_t* counts, void* stream) {
  if (int rc = check_logits(h, T, logits, logits_type, row_stride)) return rc;
  if (T > 0 && (!idx || !w)) return moe::set_error(MOE_E_INVAL, "null idx or w");
  if (!aligned4(bias) || !aligned4(idx) || !aligned4(w) || !aligned4(counts))
    return moe::set_error(MOE_E_INVAL, "bias, idx, w and counts must be 4-byte aligned");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (counts && blocks_of(T) != 1) {  // a single block writes its counts, more add theirs
    cudaError_t e = cudaMemsetAsync(counts, 0, sizeof(int32_t) * h->r.E, s);
    if (e != cudaSuccess) return moe::set_cuda_error(e, "cudaMemsetAsync");
  }
  if (T == 0) return MOE_OK;
  auto go = [&](auto l, auto v) {
    using L = decltype(l);
    constexpr int VPL = decltype(v)::value;
    const L* p = static_cast<const L*>(logits);
    const bool vec = h->r.E % VPL == 0 && rows_aligned(p, row_stride, sizeof(L), VPL);
    return launch(vec ? route_forward<L, VPL, true> : route_forward<L, VPL, false>, T, s, h->r, T, p, row_stride,
                  bias, static_cast<int*>(idx), w, static_cast<int*>(counts));
  };
  cudaError_t e = logits_type == MOE_TYPE_F32 ? by_vpl<float>(h->r.E, go) : by_vpl<__nv_bfloat16>(h->r.E, go);
  return e == cudaSuccess ? MOE_OK : moe::set_cuda_error(e, "route_forward");
}

int moe_router_backward(const moe_router_t* h, int T, const void* logits, int logits_type,
                        long long row_stride, const int32_t* idx, const float* grad_w,
                        void* grad_logits, long long grad_row_stride, void* stream) {
  if (int rc = check_logits(h, T, logits, logits_type, row_stride)) return rc;
  if (T == 0) return MOE_OK;
  if (!idx || !grad_w || !grad_logits) return moe::set_error(MOE_E_INVAL, "null idx, grad_w or grad_logits");
  if (!aligned4(idx) || !aligned4(grad_w)) return moe::set_error(MOE_E_INVAL, "idx and grad_w must be 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(grad_logits) % type_size(logits_type))
    return moe::set_error(MOE_E_INVAL, "grad_logits must be aligned to its type");
  if (grad_row_stride < h->r.E)
    return moe::set_error(MOE_E_INVAL, "rows of grad_logits overlap: the row stride is below E");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto go = [&](auto l, auto v) {
    using L = decltype(l);
    constexpr int VPL = decltype(v)::value;
    const L* p = static_cast<const L*>(logits);
    L* g = static_cast<L*>(grad_logits);
    const bool vec = h->r.E % VPL == 0 && rows_aligned(p, row_stride, sizeof(L), VPL) &&
                     rows_aligned(g, grad_row_stride, sizeof(L), VPL);
    return launch(vec ? route_backward<L, VPL, true> : route_backward<L, VPL, false>, T, s, h->r, T, p, row_stride,
                  static_cast<const int*>(idx), grad_w, g, grad_row_stride);
  };
  cudaError_t e = logits_type == MOE_TYPE_F32 ? by_vpl<float>(h->r.E, go) : by_vpl<__nv_bfloat16>(h->r.E, go);
  return e == cudaSuccess ? MOE_OK : moe::set_cuda_error(e, "route_backward");
}

}  // extern "C"
