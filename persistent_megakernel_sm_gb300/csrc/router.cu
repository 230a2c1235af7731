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
// experts each, so a warp chooses for 8 to 1 rows at once, from few candidates
// (choose below).  The weights follow for the chosen alone, a lane a slot, for
// several rows together.  What bounds the choice is instructions, not the 2 to 4
// bytes a logit: 920 of a warp for a row of 256 experts in 8 groups, top 8 (8192
// rows 14.4 us, their bytes 1.2); the gradient waits for the gathered logits,
// then writes every expert (32768 rows of 256 fp32 10.5 us, those writes 4.9).
// Scores and sums are fp32.
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
// Blocks resident on an SM.  More hide more latency, fewer leave a warp more rows
// together: 8192 rows of 256 grouped experts 14.4 us at 2 and 3, 16.4 at 4, 32768
// of 64 experts 14.4, 12.8 and 14.4; the gradient of 32768 rows of 256 11.5 at 3,
// 10.5 at 4, 11.7 at 5.
constexpr int kForward = 3, kBackward = 4;
constexpr unsigned kAll = 0xffffffffu;

struct Route {
  int E, k, score, groups, kept, group_score, renorm;
  float scale;
  int span;  // log2 of the lanes of a group, if it is 8 experts of each of 1, 2, 4 ... lanes, or -1
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

// For the choice alone: within 4e-7 of the score (which is at most 1), by the
// device's 2^x and reciprocal; a far negative logit's score keeps fewer bits.
__device__ __forceinline__ float fast_sigmoid(float l) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(l * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
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

__device__ __forceinline__ float share_base(int score, float l, bool live, int n) {
  const float m = run_max(live ? l : -INFINITY, n);
  return score == MOE_SCORE_SOFTMAX ? m : fminf(m, 0.f);
}

// The two largest of this lane's and the lane o away's.
__device__ __forceinline__ void merge_top2(uint32_t& m1, uint32_t& m2, int o) {
  const uint32_t o1 = __shfl_xor_sync(kAll, m1, o), o2 = __shfl_xor_sync(kAll, m2, o);
  m2 = max(max(m2, o2), min(m1, o1));
  m1 = max(m1, o1);
}

// What ranks a group of these two largest keys; at least kDead.
__device__ __forceinline__ uint32_t level_of(uint32_t m1, uint32_t m2, bool top2) {
  if (top2 && m1 > kDead && m2 > kDead) m1 = key_of(value_of(m1) + value_of(m2));
  return max(m1, kDead);
}

// pick[0..k) = the experts of the k largest keys of the row held by LANES
// lanes, larger first, the lower expert on ties; -1 where none is left.
//
// k rounds on the lanes' largest keys alone give a bound that at least k keys
// (of as many lanes) reach and few others do (k = 8 of 256: 9 to 11 on
// average); these candidates are listed in the experts' order and each is
// ranked against the others, in about 170 instructions where k rounds of a
// maximum, its expert and its removal over all keys took 500 (8192 rows 20.6 us
// so, 16.5 with candidates).  Rows with more candidates than kHold a lane (many
// equal logits) are still chosen by such rounds.
constexpr int kHold = 2;

template <int LANES>
__device__ __forceinline__ void choose(uint32_t (&key)[kVals], int k, int e0, int sub, int at_once, uint2* cand,
                                       int* pick) {
  constexpr unsigned kRun = LANES == 32 ? kAll : (1u << (LANES & 31)) - 1u;
  uint32_t best = key[0];
#pragma unroll
  for (int i = 1; i < kVals; ++i) best = max(best, key[i]);
  uint32_t bound = 0u, rest = best;
  for (int j = 0; j < k; ++j) {
    bound = run_max<LANES>(rest);
    rest = rest == bound ? 0u : rest;
  }
  bound = max(bound, kDead + 1u);
  int mine = 0, before = 0;
#pragma unroll
  for (int i = 0; i < kVals; ++i) mine += key[i] >= bound;
  const int shift = LANES == 32 ? 0 : at_once * LANES;
  int n = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) {  // the lanes' counts, 0 to 8, added bit by bit
    const unsigned with = __ballot_sync(kAll, mine >> b & 1) >> shift & kRun;
    before += __popc(with & ((1u << sub) - 1u)) << b;
    n += __popc(with) << b;
  }
  if (!__any_sync(kAll, n > kHold * LANES)) {
#pragma unroll
    for (int i = 0; i < kVals; ++i)
      if (key[i] >= bound) cand[before++] = make_uint2(key[i], e0 + i);
    __syncwarp();
    uint2 c[kHold];
    int rank[kHold];
#pragma unroll
    for (int h = 0; h < kHold; ++h) {
      const int q = h * LANES + sub;
      c[h] = q < n ? cand[q] : make_uint2(0u, 0u);
      rank[h] = 0;
    }
    const int most = LANES == 32 ? n : __reduce_max_sync(kAll, n);
    if (most <= LANES) {
      for (int o = 0; o < most; ++o)
        rank[0] += __shfl_sync(kAll, c[0].x, o, LANES) > (o < sub ? c[0].x - 1u : c[0].x);
    } else {
#pragma unroll
      for (int f = 0; f < kHold; ++f) {
        for (int o = 0; o < LANES && f * LANES + o < most; ++o) {
          const uint32_t v = __shfl_sync(kAll, c[f].x, o, LANES);
#pragma unroll
          for (int h = 0; h < kHold; ++h) rank[h] += v > (f < h || (f == h && o < sub) ? c[h].x - 1u : c[h].x);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < kHold; ++h)
      if (h * LANES + sub < n && rank[h] < k) pick[rank[h]] = (int)c[h].y;
    for (int j = n + sub; j < k; j += LANES) pick[j] = -1;
    __syncwarp();  // the candidates' place is free again
    return;
  }
  for (int j = 0; j < k; ++j) {
    const uint32_t m = run_max<LANES>(best);
    const unsigned with = __ballot_sync(kAll, best == m) >> shift & kRun;
    const bool here = sub == __ffs(with) - 1;
    const uint32_t hit = here && m > kDead ? m : 1u;  // no key is 1
    int e = -1;
#pragma unroll
    for (int i = kVals - 1; i >= 0; --i) e = key[i] == hit ? i : e;
#pragma unroll
    for (int i = 0; i < kVals; ++i) key[i] = e == i ? 0u : key[i];
    if (here) {
      pick[j] = e < 0 ? -1 : e0 + e;
      best = max(max(max(key[0], key[1]), max(key[2], key[3])), max(max(key[4], key[5]), max(key[6], key[7])));
    }
  }
}

// What a warp takes of the rows, in units of `unit` rows: `base` units, the first
// `extra` warps one more, at most `units` of them together.  klog: log2 of kpad,
// k rounded up to a power of two.
struct Share {
  int unit, base, extra, units, klog;
};

template <typename L, int LANES, bool VEC>
__global__ void __launch_bounds__(kWarps * 32, kForward)
    route_forward(Route r, int T, Share share, const L* __restrict__ logits, long long stride,
                  const float* __restrict__ bias, int* __restrict__ idx, float* __restrict__ w,
                  int* __restrict__ counts) {
  constexpr int kAtOnce = 32 / LANES, kMaxRows = max_rows(LANES);
  __shared__ float s_value[kWarps][32 * kVals];
  __shared__ uint32_t s_level[kWarps][kAtOnce][kMaxGroups];
  __shared__ uint2 s_cand[kWarps][32 * kHold];
  __shared__ int s_pick[kWarps][kMaxRows][kMaxK];
  __shared__ float2 s_norm[kWarps][kMaxRows];
  __shared__ int s_count[kMaxE];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & (LANES - 1), at_once = lane / LANES;
  const int E = r.E, k = r.k, klog = share.klog, kpad = 1 << klog, e0 = sub * kVals;
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
  // groups that are not whole lanes: `per` lanes walk each group (one lane
  // several groups if there are more groups than lanes); which group this
  // lane's experts are in
  int per = LANES;
  int in_group[kVals];
  if (by_level && r.span < 0) {
    while (per > 1 && per * r.groups > LANES) per >>= 1;
#pragma unroll
    for (int i = 0; i < kVals; ++i) in_group[i] = e0 + i < E ? (e0 + i) / gs : 0;
  }

  const int w_id = blockIdx.x * kWarps + warp;
  int left = share.base + (w_id < share.extra);
  long long t0 = ((long long)w_id * share.base + min(w_id, share.extra)) * share.unit;
  for (int now; left > 0; left -= now, t0 += now * share.unit) {
    now = min(left, share.units);
    const int rows = now * share.unit;
    for (int r0 = 0; r0 < rows; r0 += kAtOnce) {
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
      if (bias) {  // masked by either, even if the other is NaN (which fminf passes over)
#pragma unroll
        for (int i = 0; i < kVals; ++i) key[i] = fminf(l[i], b[i]) == -INFINITY ? 0u : key_of(s[i] + b[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kVals; ++i) key[i] = key_of(l[i]);
      }
      if (by_level && r.span >= 0) {
        // a group is some lanes: its two largest by exchanges among them
        uint32_t m1 = 0u, m2 = 0u;
#pragma unroll
        for (int i = 0; i < kVals; ++i) {
          const uint32_t v = key[i] > kDead && level_of_scores && !bias ? key_of(s[i]) : key[i];
          m2 = max(m2, min(m1, v));
          m1 = max(m1, v);
        }
        for (int o = (1 << r.span) >> 1; o; o >>= 1) merge_top2(m1, m2, o);
        const uint32_t level = level_of(m1, m2, top2);
        const int g = sub >> r.span;
        int rank = 0;
        for (int o = 0; o < r.groups; ++o)
          rank += __shfl_sync(kAll, level, o << r.span, LANES) > (o < g ? level - 1u : level);
        if (rank >= r.kept) {
#pragma unroll
          for (int i = 0; i < kVals; ++i) key[i] = 0u;
        }
      } else if (by_level) {
        // the value each expert gives its group: c, s without a bias, or l where
        // the largest alone counts
        uint32_t* value = reinterpret_cast<uint32_t*>(s_value[warp]) + at_once * LANES * kVals;
#pragma unroll
        for (int i = 0; i < kVals; ++i)
          value[e0 + i] = key[i] > kDead && level_of_scores && !bias ? key_of(s[i]) : key[i];
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
          for (int o = per >> 1; o; o >>= 1) merge_top2(m1, m2, o);
          if (g < r.groups && step == 0) s_level[warp][at_once][g] = level_of(m1, m2, top2);
        }
        __syncwarp();
        uint32_t kept = 0u;
        for (int g = sub; g < r.groups; g += LANES) {
          const uint32_t level = s_level[warp][at_once][g];
          int rank = 0;
          for (int o = 0; o < r.groups; ++o) rank += s_level[warp][at_once][o] > (o < g ? level - 1u : level);
          if (rank < r.kept) kept |= 1u << g;
        }
        for (int o = LANES / 2; o; o >>= 1) kept |= __shfl_xor_sync(kAll, kept, o);
#pragma unroll
        for (int i = 0; i < kVals; ++i)
          if (!(kept >> in_group[i] & 1u)) key[i] = 0u;
      }
      choose<LANES>(key, k, e0, sub, at_once, s_cand[warp] + at_once * LANES * kHold, s_pick[warp][r0 + at_once]);
    }
    __syncwarp();
    for (int q0 = 0; q0 < rows * kpad; q0 += 32) {
      const int row_of = (q0 + lane) >> klog, j = lane & (kpad - 1);
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
__global__ void __launch_bounds__(kWarps * 32, kBackward)
    route_backward(Route r, int T, Share share, const L* __restrict__ logits, long long stride,
                   const int* __restrict__ idx, const float* __restrict__ grad_w,
                   L* __restrict__ grad, long long grad_stride) {
  constexpr int kAtOnce = 32 / LANES, kMaxRows = max_rows(LANES);
  __shared__ float s_row[kWarps][kMaxRows][LANES * kVals];
  __shared__ float2 s_norm[kWarps][kMaxRows];
  __shared__ float s_dot[kWarps][kMaxRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & (LANES - 1), at_once = lane / LANES;
  const int E = r.E, k = r.k, klog = share.klog, kpad = 1 << klog, e0 = sub * kVals;
  const bool dense = r.score == MOE_SCORE_SOFTMAX && !r.renorm;
  // rows of zeros to add to; the entries added to are set back below
  for (int i = lane; i < kMaxRows * LANES * kVals; i += 32) (&s_row[warp][0][0])[i] = 0.f;
  __syncwarp();
  const int w_id = blockIdx.x * kWarps + warp;
  int left = share.base + (w_id < share.extra);
  long long t0 = ((long long)w_id * share.base + min(w_id, share.extra)) * share.unit;
  const int row_of = lane >> klog, j = lane & (kpad - 1);
  int rows = min(left, share.units) * share.unit;
  bool slot = row_of < rows && t0 + row_of < T && j < k;
  int e = slot ? idx[(t0 + row_of) * k + j] : -1;
  float g = slot ? grad_w[(t0 + row_of) * k + j] : 0.f;
  float lj = (unsigned)e < (unsigned)E ? to_float(logits[(t0 + row_of) * stride + e]) : -INFINITY;
  while (left > 0) {
    // the next slots are on their way while these are worked on
    left -= share.units;
    const long long t1 = t0 + rows;
    const int rows1 = max(min(left, share.units) * share.unit, 0);
    slot = row_of < rows1 && t1 + row_of < T && j < k;
    const int e1 = slot ? idx[(t1 + row_of) * k + j] : -1;
    const float g1 = slot ? grad_w[(t1 + row_of) * k + j] : 0.f;
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
    const bool live = lj != -INFINITY;  // not a masked expert, whose score is 0
    if (!live) g = 0.f;
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
    // an expert named by several slots of a row gets their sum, in slot order:
    // each slot leaves its mark, and one that does not find it has a double (a
    // match of all slots with each other every time: 11.6 us in place of 10.5)
    unsigned same = 1u << lane;
    if (live) s_row[warp][row_of][e] = __int_as_float(lane);
    __syncwarp();
    if (__any_sync(kAll, live && __float_as_int(s_row[warp][row_of][e]) != lane)) {
      same = __match_any_sync(kAll, live ? row_of * kMaxE + e : -1 - lane);  // no two dead slots alike
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
    lj = (unsigned)e1 < (unsigned)E ? to_float(logits[(t1 + row_of) * stride + e1]) : -INFINITY;
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
    e = e1, g = g1, t0 = t1, rows = rows1;
  }
}

// Rows that vectors of 8 elements (16 bytes at most) can be read from.
bool rows_aligned(const void* p, long long stride, size_t size) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (size_t)stride * size % 16 == 0;
}

int log2_from(int n) {  // rounded up
  int l = 0;
  while (1 << l < n) ++l;
  return l;
}

int lanes_of(int E) { return std::max(4, 1 << log2_from((E + kVals - 1) / kVals)); }

// Route::span
int span_of(int E, int groups) {
  const int lanes = E / groups / kVals;
  return E / groups % kVals == 0 && (lanes & (lanes - 1)) == 0 ? log2_from(lanes) : -1;
}

// The resident warps share the rows, to within one unit of each other, so that
// each weighs the slots of its few rows together and all end at about the same
// time: 8192 rows of 256 grouped experts 14.4 us, 16.5 with a grid's stride of
// single rows; 32768 of 64 experts 12.8 and 14.4.
Share split_of(const Route& r, int T, bool backward, int* blocks) {
  const int lanes = lanes_of(r.E);
  Share s;
  s.klog = log2_from(r.k);
  // as many rows together as have a lane for each slot; the choice takes all the
  // rows that a warp holds even so
  const int together = std::min(max_rows(lanes), 32 >> s.klog);
  s.unit = backward ? std::min(32 / lanes, together) : 32 / lanes;
  s.units = std::max(1, together / s.unit);
  const int units = (int)(((long long)T + s.unit - 1) / s.unit);
  *blocks = std::min((units + kWarps - 1) / kWarps, kSms * (backward ? kBackward : kForward));
  s.base = units / (*blocks * kWarps), s.extra = units % (*blocks * kWarps);
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
  h->r = Route{E, k, score, groups, groups_kept, group_score, renormalise, scale,
               span_of(E, groups)};
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
  int blocks = 0;
  const Share share = T ? split_of(h->r, T, false, &blocks) : Share{};
  if (counts && blocks != 1) {  // a single block writes its counts, more add theirs
    cudaError_t e = cudaMemsetAsync(counts, 0, sizeof(int32_t) * h->r.E, s);
    if (e != cudaSuccess) return moe::set_cuda_error(e, "cudaMemsetAsync");
  }
  if (T == 0) return MOE_OK;
  auto go = [&](auto l, auto n) {
    using L = decltype(l);
    constexpr int LANES = decltype(n)::value;
    const L* p = static_cast<const L*>(logits);
    const bool vec = h->r.E % kVals == 0 && rows_aligned(p, row_stride, sizeof(L));
    return launch(vec ? route_forward<L, LANES, true> : route_forward<L, LANES, false>, blocks, s, h->r, T, share, p, row_stride, bias, static_cast<int*>(idx), w, static_cast<int*>(counts));
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
  int blocks;
  const Share share = split_of(h->r, T, true, &blocks);
  auto go = [&](auto l, auto n) {
    using L = decltype(l);
    constexpr int LANES = decltype(n)::value;
    const L* p = static_cast<const L*>(logits);
    L* g = static_cast<L*>(grad_logits);
    const bool vec = h->r.E % kVals == 0 && rows_aligned(p, row_stride, sizeof(L)) &&
                     rows_aligned(g, grad_row_stride, sizeof(L));
    return launch(vec ? route_backward<L, LANES, true> : route_backward<L, LANES, false>, blocks, s, h->r, T, share, p, row_stride, static_cast<const int*>(idx), grad_w, g, grad_row_stride);
  };
  cudaError_t e = logits_type == MOE_TYPE_F32 ? by_lanes<float>(h->r.E, go) : by_lanes<__nv_bfloat16>(h->r.E, go);
  return e == cudaSuccess ? MOE_OK : moe::set_cuda_error(e, "route_backward");
}

}  // extern "C"
