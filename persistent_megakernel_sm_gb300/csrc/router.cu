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
// A row's logits are in the registers of 4, 8, 16 or 32 lanes, 8 consecutive
// experts each, so a warp chooses for 8 to 1 rows at once; the lowest lane with
// the maximum is the lowest expert, so a selection round is a maximum over the
// row's lanes, one ballot and a search among 8 values.  The weights follow for
// the chosen alone, a lane a slot, for several rows together.  What bounds both
// kernels is instructions, not the 2 to 4 bytes a logit: at 8192 rows of 256
// experts in 8 groups, top 8, the selection rounds are half of them.  Scores
// and sums are fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <new>
#include <type_traits>

#include "error.h"
#include "moe.h"

namespace {

constexpr int kMaxE = 256;
constexpr int kMaxK = 16;
constexpr int kMaxGroups = 32;
constexpr int kWarps = 8;           // of a block
constexpr int kVals = 8;            // experts of a lane
constexpr int kSms = 152;
constexpr unsigned kAll = 0xffffffffu;

struct Route {
  int E, k, score, groups, kept, group_score, renorm;
  float scale;
};

// Rows a warp takes together, at most.
__host__ __device__ constexpr int max_rows(int lanes) { return lanes == 4 ? 8 : 4; }

// Unsigned order of floats: larger value, larger key; NaN above everything,
// both zeros equal.  Keys up to kDead are -inf or nothing: never chosen.
constexpr uint32_t kDead = 0x007fffffu;

__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);  // a sum's NaN is the positive one
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}

// Over aligned runs of n lanes, n a power of two.
__device__ __forceinline__ float run_max(float v, int n) {
  for (int o = n >> 1; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

__device__ __forceinline__ float run_sum(float v, int n) {
  for (int o = n >> 1; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

template <int LANES>
__device__ __forceinline__ uint32_t run_max(uint32_t v) {
  if constexpr (LANES == 32) {
    return __reduce_max_sync(kAll, v);
  } else {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
    return v;
  }
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

// Softmax of the row held by LANES lanes: p over v in place (0 where v is
// -inf); a row of -inf alone gives zeros.
template <int LANES, int VPL>
__device__ __forceinline__ void row_softmax(float (&v)[VPL], float* top, float* inv) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) m = fmaxf(m, v[i]);
  m = run_max(m, LANES);
  const float base = m == -INFINITY ? 0.f : m;
  float z = 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    v[i] = expf(v[i] - base);
    z += v[i];
  }
  z = run_sum(z, LANES);
  *top = base;
  *inv = z == 0.f ? 0.f : 1.f / z;
#pragma unroll
  for (int i = 0; i < VPL; ++i) v[i] *= *inv;
}

// For the choice alone: within 4e-7.
__device__ __forceinline__ float fast_sigmoid(float l) { return __fdividef(1.f, 1.f + __expf(-l)); }

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

__device__ __forceinline__ float share_base(int score, float l, bool live, int n) {
  const float m = run_max(live ? l : -INFINITY, n);
  return score == MOE_SCORE_SOFTMAX ? m : fminf(m, 0.f);
}

// `rows`: rows a warp takes together, a multiple of 32 / LANES; kpad: k rounded
// up to a power of two.
template <typename L, int LANES, bool VEC>
__global__ void __launch_bounds__(kWarps * 32, 3)
    route_forward(Route r, int T, int rows, int kpad, const L* __restrict__ logits, long long stride,
                  const float* __restrict__ bias, int* __restrict__ idx, float* __restrict__ w,
                  int* __restrict__ counts) {
  constexpr int kAtOnce = 32 / LANES, kMaxRows = max_rows(LANES);
  __shared__ float s_value[kWarps][32 * kVals];
  __shared__ uint32_t s_level[kWarps][kAtOnce][kMaxGroups];
  __shared__ int s_pick[kWarps][kMaxRows][kMaxK];
  __shared__ float2 s_norm[kWarps][kMaxRows];
  __shared__ int s_count[kMaxE];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & (LANES - 1), at_once = lane / LANES;
  const int E = r.E, k = r.k, e0 = sub * kVals;
  const int gs = E / r.groups;
  if (counts) {
    for (int e = threadIdx.x; e < E; e += kWarps * 32) s_count[e] = 0;
    __syncthreads();
  }
  float b[kVals];
#pragma unroll
  for (int i = 0; i < kVals; ++i) b[i] = bias && e0 + i < E ? __ldg(bias + e0 + i) : 0.f;
  const bool top2 = r.group_score == MOE_GROUP_TOP2;
  const bool by_level = r.groups > 1;
  const bool level_of_scores = by_level && top2;
  const bool need_p = r.score == MOE_SCORE_SOFTMAX && (!r.renorm || bias || level_of_scores);
  // groups: `per` lanes walk each group (one lane several groups if there are
  // more groups than lanes); which group this lane's experts are in
  int per = LANES;
  while (per > 1 && per * r.groups > LANES) per >>= 1;
  int in_group[kVals];
#pragma unroll
  for (int i = 0; i < kVals; ++i) in_group[i] = by_level && e0 + i < E ? (e0 + i) / gs : 0;

  for (long long t0 = ((long long)blockIdx.x * kWarps + warp) * rows; t0 < T; t0 += (long long)gridDim.x * kWarps * rows) {
    for (int r0 = 0; r0 < rows && t0 + r0 < T; r0 += kAtOnce) {
      const long long t = t0 + r0 + at_once;
      const L* row = logits + (t < T ? t : T - 1) * stride;
      float l[kVals], s[kVals];
      load_row<L, kVals, VEC>(row, e0, E, l);
#pragma unroll
      for (int i = 0; i < kVals; ++i) s[i] = l[i];
      if (need_p) {
        float top, inv;
        row_softmax<LANES, kVals>(s, &top, &inv);
        if (sub == 0) s_norm[warp][r0 + at_once] = make_float2(top, inv);
      } else if (r.score == MOE_SCORE_SIGMOID && (bias || level_of_scores)) {
#pragma unroll
        for (int i = 0; i < kVals; ++i) s[i] = fast_sigmoid(l[i]);
      }
      uint32_t key[kVals];
#pragma unroll
      for (int i = 0; i < kVals; ++i) key[i] = l[i] == -INFINITY ? 0u : key_of(bias ? s[i] + b[i] : l[i]);
      if (by_level) {
        // the value each expert gives its group: c, s without a bias, or l where
        // the largest alone counts
        uint32_t* value = reinterpret_cast<uint32_t*>(s_value[warp]) + at_once * LANES * kVals;
#pragma unroll
        for (int i = 0; i < kVals; ++i)
          value[e0 + i] = key[i] != 0u && level_of_scores && !bias ? key_of(s[i]) : key[i];
        __syncwarp();
        for (int g0 = 0; g0 < r.groups; g0 += LANES / per) {
          const int g = g0 + sub / per, step = sub & (per - 1);
          uint32_t m1 = 0u, m2 = 0u;
          if (g < r.groups) {
            // start each group elsewhere, so that groups of 32 experts read other banks
            const int n = (gs - step + per - 1) / per;
            for (int i = 0, at = n > 0 ? g % n : 0; i < n; ++i, at = at + 1 == n ? 0 : at + 1) {
              const uint32_t v = value[g * gs + step + at * per];
              m2 = max(m2, min(m1, v));
              m1 = max(m1, v);
            }
          }
          for (int o = per >> 1; o; o >>= 1) {
            const uint32_t o1 = __shfl_xor_sync(kAll, m1, o), o2 = __shfl_xor_sync(kAll, m2, o);
            m2 = max(max(m2, o2), min(m1, o1));
            m1 = max(m1, o1);
          }
          if (top2 && m1 > kDead && m2 > kDead) m1 = key_of(value_of(m1) + value_of(m2));
          if (g < r.groups && step == 0) s_level[warp][at_once][g] = max(m1, kDead);
        }
        __syncwarp();
        uint32_t kept = 0u;
        for (int g = sub; g < r.groups; g += LANES) {
          const uint32_t level = s_level[warp][at_once][g];
          int rank = 0;
          for (int o = 0; o < r.groups; ++o) {
            const uint32_t v = s_level[warp][at_once][o];
            rank += v > level || (v == level && o < g);
          }
          if (rank < r.kept) kept |= 1u << g;
        }
        for (int o = LANES / 2; o; o >>= 1) kept |= __shfl_xor_sync(kAll, kept, o);
#pragma unroll
        for (int i = 0; i < kVals; ++i)
          if (!(kept >> in_group[i] & 1u)) key[i] = 0u;
      }
      uint32_t best = key[0];
#pragma unroll
      for (int i = 1; i < kVals; ++i) best = max(best, key[i]);
      int* pick = s_pick[warp][r0 + at_once];
      for (int j = 0; j < k; ++j) {
        const uint32_t m = run_max<LANES>(best);
        unsigned with = __ballot_sync(kAll, best == m);
        if (LANES < 32) with = with >> (at_once * LANES) & ((1u << (LANES & 31)) - 1u);
        const bool mine = sub == __ffs(with) - 1;
        const uint32_t hit = mine && m > kDead ? m : 1u;  // no key is 1
        int e = -1;
#pragma unroll
        for (int i = kVals - 1; i >= 0; --i) e = key[i] == hit ? i : e;
#pragma unroll
        for (int i = 0; i < kVals; ++i) key[i] = e == i ? 0u : key[i];
        if (mine) {
          pick[j] = e < 0 ? -1 : e0 + e;
          best = max(max(max(key[0], key[1]), max(key[2], key[3])), max(max(key[4], key[5]), max(key[6], key[7])));
        }
      }
    }
    __syncwarp();
    for (int q0 = 0; q0 < rows * kpad; q0 += 32) {
      const int row_of = (q0 + lane) / kpad, j = lane & (kpad - 1);
      const long long t = t0 + row_of;
      const bool slot = row_of < rows && t < T && j < k;
      const int e = slot ? s_pick[warp][row_of][j] : -1;
      const bool live = e >= 0;
      const float lj = live ? to_float(logits[t * stride + e]) : -INFINITY;
      float wj = 0.f;
      if (r.renorm) {
        const float m = share_base(r.score, lj, live, kpad);
        const float a = live ? share_of(r.score, lj, m) : 0.f;
        const float z = run_sum(a, kpad);
        if (live) wj = a / z;
      } else if (live) {
        const float2 norm = s_norm[warp][row_of];
        wj = r.score == MOE_SCORE_SOFTMAX ? expf(lj - norm.x) * norm.y : sigmoid(lj);
      }
      if (slot) {
        idx[t * k + j] = e;
        w[t * k + j] = live ? r.scale * wj : 0.f;
        if (counts && live) atomicAdd(&s_count[e], 1);
      }
    }
    __syncwarp();
  }
  if (counts) {
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kWarps * 32) {
      if (gridDim.x == 1) counts[e] = s_count[e];
      else if (s_count[e]) atomicAdd(counts + e, s_count[e]);
    }
  }
}

// A lane a slot for `rows` rows together (rows kpad <= 32), then a row at a
// time by 32 / LANES rows: what the softmax gives every expert, or zero, with
// the slots' shares added.
template <typename L, int LANES, bool VEC>
__global__ void __launch_bounds__(kWarps * 32, 3)
    route_backward(Route r, int T, int rows, int kpad, const L* __restrict__ logits, long long stride,
                   const int* __restrict__ idx, const float* __restrict__ grad_w,
                   L* __restrict__ grad, long long grad_stride) {
  constexpr int kAtOnce = 32 / LANES, kMaxRows = max_rows(LANES);
  __shared__ float s_row[kWarps][kMaxRows][LANES * kVals];
  __shared__ float2 s_norm[kWarps][kMaxRows];
  __shared__ float s_dot[kWarps][kMaxRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & (LANES - 1), at_once = lane / LANES;
  const int E = r.E, k = r.k, e0 = sub * kVals;
  const bool dense = r.score == MOE_SCORE_SOFTMAX && !r.renorm;
  // rows of zeros to add to; the entries added to are set back below
  for (int i = lane; i < kMaxRows * LANES * kVals; i += 32) (&s_row[warp][0][0])[i] = 0.f;
  __syncwarp();
  for (long long t0 = ((long long)blockIdx.x * kWarps + warp) * rows; t0 < T; t0 += (long long)gridDim.x * kWarps * rows) {
    if (dense) {
      for (int r0 = 0; r0 < rows && t0 + r0 < T; r0 += kAtOnce) {
        const long long t = t0 + r0 + at_once;
        float v[kVals], top, inv;
        load_row<L, kVals, VEC>(logits + (t < T ? t : T - 1) * stride, e0, E, v);
        row_softmax<LANES, kVals>(v, &top, &inv);
        if (sub == 0 && r0 + at_once < rows) s_norm[warp][r0 + at_once] = make_float2(top, inv);
      }
      __syncwarp();
    }
    const int row_of = lane / kpad, j = lane & (kpad - 1);
    const long long ts = t0 + row_of;
    const bool slot = row_of < rows && ts < T && j < k;
    const int e = slot ? idx[ts * k + j] : -1;
    const float lj = (unsigned)e < (unsigned)E ? to_float(logits[ts * stride + e]) : -INFINITY;
    const bool live = lj != -INFINITY;  // nor a masked expert, whose score is 0
    const float g = live ? grad_w[ts * k + j] : 0.f;
    float add = 0.f;  // what this slot adds to its expert's gradient
    if (r.renorm) {
      const float m = share_base(r.score, lj, live, kpad);
      float a = live ? share_of(r.score, lj, m) : 0.f;
      const float z = run_sum(a, kpad);
      a = live ? a / z : 0.f;
      const float dot = run_sum(live ? g * a : 0.f, kpad);
      if (live) add = r.scale * a * (g - dot);
      if (r.score == MOE_SCORE_SIGMOID) add *= sigmoid(-lj);
    } else if (r.score == MOE_SCORE_SIGMOID) {
      if (live) add = r.scale * g * sigmoid(lj) * sigmoid(-lj);
    } else {
      const float2 norm = s_norm[warp][row_of < rows ? row_of : 0];
      add = live ? r.scale * g * expf(lj - norm.x) * norm.y : 0.f;
      const float dot = run_sum(add, kpad);
      if (j == 0 && row_of < rows) s_dot[warp][row_of] = dot;
    }
    // an expert named by several slots of a row gets their sum, in slot order
    const int key = live ? row_of * kMaxE + e : -1 - lane;  // no two dead slots alike
    const unsigned same = __match_any_sync(kAll, key);
    if (__any_sync(kAll, (same & (same - 1)) != 0u)) {
      float sum = 0.f;
      for (int q = 0; q < 32; ++q) {
        const float o = __shfl_sync(kAll, add, q);
        if (same >> q & 1u) sum += o;
      }
      add = sum;
    }
    const bool leads = live && lane == __ffs(same) - 1;
    if (leads) s_row[warp][row_of][e] = add;
    __syncwarp();
    for (int r0 = 0; r0 < rows && t0 + r0 < T; r0 += kAtOnce) {
      const long long t = t0 + r0 + at_once;
      const bool mine = r0 + at_once < rows && t < T;  // rows of fewer than the lanes hold
      const int at = mine ? r0 + at_once : 0;
      float v[kVals];
      const float4* from = reinterpret_cast<const float4*>(&s_row[warp][at][e0]);
      const float4 x = from[0], y = from[1];
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
      if (dense) {
        float p[kVals];
        load_row<L, kVals, VEC>(logits + (t < T ? t : T - 1) * stride, e0, E, p);
        const float2 norm = s_norm[warp][at];
        const float dot = s_dot[warp][at];
#pragma unroll
        for (int i = 0; i < kVals; ++i) v[i] -= expf(p[i] - norm.x) * norm.y * dot;
      }
      if (mine) store_row<L, kVals, VEC>(grad + t * grad_stride, e0, E, v);
    }
    __syncwarp();
    if (leads) s_row[warp][row_of][e] = 0.f;
    __syncwarp();
  }
}

// Rows that vectors of 8 elements (16 bytes at most) can be read from.
bool rows_aligned(const void* p, long long stride, size_t size) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (size_t)stride * size % 16 == 0;
}

int pow2_from(int n) {
  int p = 1;
  while (p < n) p <<= 1;
  return p;
}

int lanes_of(int E) { return std::max(4, pow2_from((E + kVals - 1) / kVals)); }

// How many rows a warp takes together, and blocks.
struct Shape {
  int rows, kpad, blocks;
};

Shape shape_of(const Route& r, int T, bool backward) {
  const int lanes = lanes_of(r.E), at_once = 32 / lanes;
  Shape s;
  s.kpad = pow2_from(r.k);
  const int together = std::min(max_rows(lanes), std::max(1, 32 / s.kpad));
  auto tasks_of = [&](int rows) { return ((long long)T + rows - 1) / rows; };
  int cap;
  if (backward) {
    // a slot a lane is most of the work: all the rows a warp has lanes for, once
    // there are several rows for every warp of the device (32768 rows of 256
    // experts: 12.9 us at 4 rows a warp, 27.6 at 1)
    s.rows = T > kSms * kWarps * 2 * at_once ? together : std::min(at_once, together);
    cap = kSms * 8;
  } else {
    // three blocks an SM are resident and take rows by turns: the rows together
    // that give the fullest warp the least to do, its slots costing about a
    // sixth of a choice each pass (32768 rows of 64 experts: 14.5 us so, 16.5
    // with as many blocks as there is work for)
    cap = kSms * 3;
    s.rows = at_once;
    float least = INFINITY;
    for (int rows = at_once; rows <= std::max(at_once, together); rows *= 2) {
      const long long passes = (tasks_of(rows) + cap * kWarps - 1) / (cap * kWarps);
      const float cost = (float)passes * ((float)rows / at_once + 0.17f);
      if (cost < least) least = cost, s.rows = rows;
    }
  }
  s.blocks = (int)std::min<long long>((tasks_of(s.rows) + kWarps - 1) / kWarps, cap);
  return s;
}

template <typename... A>
cudaError_t launch(void (*kernel)(A...), int blocks, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// f(element type, lanes of a row) for a router of E experts.
template <typename L, typename F>
cudaError_t by_lanes(int E, F&& f) {
  switch (lanes_of(E)) {
    case 4: return f(L{}, std::integral_constant<int, 4>{});
    case 8: return f(L{}, std::integral_constant<int, 8>{});
    case 16: return f(L{}, std::integral_constant<int, 16>{});
    default: return f(L{}, std::integral_constant<int, 32>{});
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
  const Shape shape = shape_of(h->r, T, false);
  if (counts && shape.blocks != 1) {  // a single block writes its counts, more add theirs
    cudaError_t e = cudaMemsetAsync(counts, 0, sizeof(int32_t) * h->r.E, s);
    if (e != cudaSuccess) return moe::set_cuda_error(e, "cudaMemsetAsync");
  }
  if (T == 0) return MOE_OK;
  auto go = [&](auto l, auto n) {
    using L = decltype(l);
    constexpr int LANES = decltype(n)::value;
    const L* p = static_cast<const L*>(logits);
    const bool vec = h->r.E % kVals == 0 && rows_aligned(p, row_stride, sizeof(L));
    return launch(vec ? route_forward<L, LANES, true> : route_forward<L, LANES, false>, shape.blocks, s, h->r, T,
                  shape.rows, shape.kpad, p, row_stride, bias, static_cast<int*>(idx), w, static_cast<int*>(counts));
  };
  cudaError_t e = logits_type == MOE_TYPE_F32 ? by_lanes<float>(h->r.E, go) : by_lanes<__nv_bfloat16>(h->r.E, go);
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
  const Shape shape = shape_of(h->r, T, true);
  auto go = [&](auto l, auto n) {
    using L = decltype(l);
    constexpr int LANES = decltype(n)::value;
    const L* p = static_cast<const L*>(logits);
    L* g = static_cast<L*>(grad_logits);
    const bool vec = h->r.E % kVals == 0 && rows_aligned(p, row_stride, sizeof(L)) &&
                     rows_aligned(g, grad_row_stride, sizeof(L));
    return launch(vec ? route_backward<L, LANES, true> : route_backward<L, LANES, false>, shape.blocks, s, h->r, T,
                  shape.rows, shape.kpad, p, row_stride, static_cast<const int*>(idx), grad_w, g, grad_row_stride);
  };
  cudaError_t e = logits_type == MOE_TYPE_F32 ? by_lanes<float>(h->r.E, go) : by_lanes<__nv_bfloat16>(h->r.E, go);
  return e == cudaSuccess ? MOE_OK : moe::set_cuda_error(e, "route_backward");
}

}  // extern "C"
