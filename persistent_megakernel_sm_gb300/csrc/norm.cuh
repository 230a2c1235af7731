// The norms about a block, with its gate and the residual stream, and their
// gradient.  Per token (row), with the residual r, the block's output y, a gate g
// and a factor s:
//   p   = N_post(y)                  or y itself
//   out = r + s g p                  rounded to r's type
//   n   = N_pre(out)                 of the rounded sum: what the next block reads
//   N(x) = (x - m) / sqrt(mean (x - m)^2 + eps) * gain + shift, m the mean (layer)
//   or 0 (rms)
// Backward, with u = (x - m) rstd of a norm, t = (gradient) * gain:
//   through the norm  rstd (t - u mean(t u) - [layer] mean(t))
//   G = grad_out + (that of n),  grad_r = G,  grad of p = s g G, again through the
//   post norm; grad gain = sum over rows of (gradient) u, grad shift of (gradient),
//   grad g = s G p over the rows, the columns or neither.
// The second norm's means are linear in G, which is grad_out + rstd t less multiples
// of 1 and u, so all of a row's sums are taken in one go, before either norm's
// means are known: one exchange a row.
//
// What bounds both is HBM, so the rest is kept out of its way.  A block holds a row (a
// cluster of 2, 4 or 8 blocks one that is too wide), a lane one or two times 8
// consecutive columns of it, in registers; while it works on a row, the next ones are on
// their way: by asynchronous 16-byte copies into slots of shared memory that belong to
// the thread that reads them, so that no barrier guards them.  Rows that are not aligned
// come as the 16-byte pieces that they lie in, shifted when they are read (the piece that
// two lanes share is read by both), and leave a warp's 256 columns at a time, each store
// along the row.  The forward pass exchanges sums between
// the block's warps twice a row, a layer norm once more for each norm (the mean first,
// then the squares about it); the gradient once.  Sums over rows are kept in
// registers, written once a block and added by a second kernel in a fixed order.
//
// 8192 x 7168 in bf16, root mean squares on both sides, fp32 gains, a gate of columns:
// forward 88 us, 5.3 TB/s (with one norm alone 72, 6.5); with both kept in 8 bits 160; the
// gradient 173 us, 4.1 TB/s, from 8-bit rows 222; layer norms 144 and 299; in fp32 154
// and 358.  What is left to HBM's time (69 and 104, in fp32 104 and 156) is instructions,
// 200 to 660 of a warp for 256 columns, and the wait for a row's exchange: 14 warps an SM
// issue 1.7 of them a cycle forward and 1.9 in the gradient, where 4 could be, and the 7 that
// a wide gradient in fp32 has 0.9.  4099 x 2047 in rows that are not aligned, layer norms,
// a gate of rows, fp32: forward 46 us, gradient 84 (HBM's time 17 and 27), for the shifts
// and the stores of single values.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <new>
#include <type_traits>

#include "error.h"
#include "moe.h"
#include "ptx.cuh"
#include "rows8.cuh"

namespace {

using bf16 = __nv_bfloat16;

constexpr int kMaxD = 32768;
constexpr int kMaxT = 1 << 30;            // a row index and a few strides of the grid stay in 32 bits
constexpr int kThreads = 512;            // of a block, at most
constexpr int kMaxStages = 4;            // rows under way
constexpr int kSms = 152;
constexpr int kRing = 200 * 1024;        // shared memory of an SM for all of it
constexpr int kMaxSmem = 227 * 1024;     // of a block
constexpr int kMaxCluster = 8;           // blocks of a row
constexpr unsigned kAll = 0xffffffffu;
constexpr int kNone = MOE_NORM_NONE, kRms = MOE_NORM_RMS, kLayer = MOE_NORM_LAYER;

__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ------------------------------------------------------------------------ pairs

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }

// 8 columns.
struct Eight {
  float2 v[4];
  __device__ __forceinline__ float get(int i) const { return i & 1 ? v[i >> 1].y : v[i >> 1].x; }
  __device__ __forceinline__ void set(int i, float x) { (i & 1 ? v[i >> 1].y : v[i >> 1].x) = x; }
  __device__ __forceinline__ void cut(int n) {  // zeros from column n on
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i >= n) set(i, 0.f);
  }
};

__device__ __forceinline__ Eight unpack(const uint32_t (&w)[4]) {
  Eight e;
#pragma unroll
  for (int i = 0; i < 4; ++i) e.v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  return e;
}
__device__ __forceinline__ uint4 pack(const Eight& e) {
  union {
    __nv_bfloat162 b[4];
    uint4 q;
  } u;
#pragma unroll
  for (int i = 0; i < 4; ++i) u.b[i] = __floats2bfloat162_rn(e.v[i].x, e.v[i].y);
  return u.q;
}

// ------------------------------------------------------------------------ slots

// cp.async of 16 or 8 bytes, of which n are read and the rest zero, and of 4.
__device__ __forceinline__ void copy16(void* to, const void* from, int n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(moe::smem_u32(to)), "l"(from), "r"(n) : "memory");
}
__device__ __forceinline__ void copy8(void* to, const void* from, int n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(moe::smem_u32(to)), "l"(from), "r"(n) : "memory");
}
__device__ __forceinline__ void copy4(void* to, const void* from, int n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(moe::smem_u32(to)), "l"(from), "r"(n) : "memory");
}

// Rows of a tensor: where row 0 begins and how far the next is, in bytes.
template <typename T>
struct Rows {
  T* p;
  uint32_t stride;
  __device__ __forceinline__ T* at(int t) const {  // one multiply-add
    return reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(p) + (uint64_t)(uint32_t)t * stride);
  }
};

struct Rows8 {
  int8_t* codes;  // null: none
  bf16* scales;
};

struct Shape {
  int T, d, stages;
  int field[5];    // offsets of a stage's fields, in bytes
  int stage;       // bytes of a stage
  int vec;         // where the gains and shifts begin
  int out;         // where the warps' rows for unaligned stores begin
  int parts;       // where the warps' parts of the sums begin, for this row and the one before
  int groups, group_lanes, group_log;  // of 8-bit rows: of a row; a group's eights, and the logarithm of its columns
  float scale, eps, one;    // one: 1 where gains are stored less 1
};

// `units`: threads times a thread's eights; unit: chunk * threads + thread.  A field is
// one plane of 16 bytes a unit for 8 bf16, two for 8 fp32 (codes: of 8 bytes, and one of
// 4 for a scale).  Rows that are not aligned come as the pieces of 16 bytes that they lie
// in, each unit's from the one that its first column is in; the piece behind them that
// it may need is the next lane's first, for a warp's last lane one more behind the
// planes.  So a warp's lanes read what others copied: __syncwarp stands behind
// the wait for the copies, and before the slots are given to another row.
template <typename T>
__host__ __device__ constexpr int pieces() {
  return (int)sizeof(T) / 2;
}

template <typename T, bool VEC>
__device__ __forceinline__ void fetch(char* field, int units, int unit, const T* row, int col, int d) {
  uint4* slot = reinterpret_cast<uint4*>(field) + unit;
  constexpr int k = pieces<T>();
  if constexpr (VEC) {
    if (col >= d) return;
#pragma unroll
    for (int i = 0; i < k; ++i) moe::cp_async16(slot + i * units, row + col + i * (16 / sizeof(T)));
  } else {
    const uintptr_t from = reinterpret_cast<uintptr_t>(row + col) & ~(uintptr_t)15;
    const int left = (int)(reinterpret_cast<uintptr_t>(row + d) - from);  // to the row's end; none: nothing of it is here
#pragma unroll
    for (int i = 0; i < k; ++i)
      if (left > 16 * i) copy16(slot + i * units, reinterpret_cast<const char*>(from) + 16 * i, min(16, left - 16 * i));
    if ((unit & 31) == 31 && left > 16 * k)
      copy16(reinterpret_cast<uint4*>(field) + k * units + unit / 32, reinterpret_cast<const char*>(from) + 16 * k, min(16, left - 16 * k));
  }
}

// N words from byte `shift` of the words before on; `shift` is a row's.
template <int N, int M>
__device__ __forceinline__ void shifted(const uint32_t (&w)[M], int shift, uint32_t (&out)[N]) {
  uint32_t a[M + 1], b[M + 1];
#pragma unroll
  for (int i = 0; i < M; ++i) a[i] = w[i];
  a[M] = 0;
  if (M - N >= 3) {
#pragma unroll
    for (int i = 0; i < M; ++i) b[i] = shift & 8 ? (i + 2 < M ? a[i + 2] : 0u) : a[i];
  } else {
#pragma unroll
    for (int i = 0; i < M; ++i) b[i] = a[i];
  }
#pragma unroll
  for (int i = 0; i < M; ++i) a[i] = shift & 4 ? (i + 1 < M ? b[i + 1] : 0u) : b[i];
#pragma unroll
  for (int i = 0; i < N; ++i) out[i] = __funnelshift_r(a[i], a[i + 1], (shift & 3) * 8);
}

__device__ __forceinline__ void put_words(uint4 q, uint32_t* w) { w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w; }

// What was fetched.  n: the columns that are there.
template <typename T, bool VEC>
__device__ __forceinline__ Eight read(const char* field, int units, int unit, const T* row, int n) {
  constexpr int k = pieces<T>(), kWords = (int)sizeof(T) * 2;
  const uint4* slot = reinterpret_cast<const uint4*>(field) + unit;
  uint32_t in[4 * (k + 1)], w[kWords];
#pragma unroll
  for (int i = 0; i < k; ++i) put_words(slot[i * units], in + 4 * i);
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = in[i];
  } else {
    const uint4* next = (unit & 31) == 31 ? reinterpret_cast<const uint4*>(field) + k * units + unit / 32 : slot + 1;
    put_words(*next, in + 4 * k);
    shifted(in, (int)(reinterpret_cast<uintptr_t>(row) & 15), w);
  }
  Eight e;
  if constexpr (sizeof(T) == 2) {
    e = unpack(w);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) e.v[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  }
  if (!VEC && n < 8) e.cut(n);
  return e;
}

// Where the scales of a field of codes begin: behind a plane of 8 bytes a unit, and one a warp.
template <bool VEC>
__device__ __forceinline__ int scales_at(int units) {
  return 8 * units + (VEC ? 0 : units / 4);
}

template <bool VEC>
__device__ __forceinline__ void fetch8(char* field, int units, int unit, const Rows8& r, int t, const Shape& a, int col) {
  uint2* slot = reinterpret_cast<uint2*>(field) + unit;
  const int8_t* row = r.codes + (long long)t * a.d;
  if constexpr (VEC) {
    if (col < a.d) copy8(slot, row + col, 8);
  } else {
    const uintptr_t from = reinterpret_cast<uintptr_t>(row + col) & ~(uintptr_t)7;
    const int left = (int)(reinterpret_cast<uintptr_t>(row + a.d) - from);
    if (left > 0) copy8(slot, reinterpret_cast<const char*>(from), min(8, left));
    if ((unit & 31) == 31 && left > 8)
      copy8(reinterpret_cast<uint2*>(field) + units + unit / 32, reinterpret_cast<const char*>(from) + 8, min(8, left - 8));
  }
  if (col >= a.d) return;
  // the word that the scale is in; the tensor may end in its middle
  const long long scale = (long long)t * a.groups + (col >> a.group_log);
  const bool last = scale == (long long)a.T * a.groups - 1 && !(scale & 1);
  copy4(field + scales_at<VEC>(units) + 4 * unit, r.scales + (scale & ~1ll), last ? 2 : 4);
}

template <bool VEC>
__device__ __forceinline__ Eight read8(const char* field, int units, int unit, const Rows8& r, int t, const Shape& a, int col,
                                       int n) {
  const uint2* slot = reinterpret_cast<const uint2*>(field) + unit;
  uint32_t w[2];
  const uint2 q = slot[0];
  if constexpr (VEC) {
    w[0] = q.x, w[1] = q.y;
  } else {
    const uint2 q2 = (unit & 31) == 31 ? reinterpret_cast<const uint2*>(field)[units + unit / 32] : slot[1];
    const uint32_t in[4] = {q.x, q.y, q2.x, q2.y};
    shifted(in, (int)(reinterpret_cast<uintptr_t>(r.codes + (long long)t * a.d) & 7), w);
  }
  const uint32_t word = *reinterpret_cast<const uint32_t*>(field + scales_at<VEC>(units) + 4 * unit);
  const bool odd = ((uint32_t)t * (uint32_t)a.groups + (uint32_t)(col >> a.group_log)) & 1;  // the low bit alone: any width will do
  const float s = __uint_as_float(odd ? word & 0xffff0000u : word << 16);
  Eight e;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float2 x[2];
    moe::rows8_floats(w[h], x);
    e.v[2 * h] = mul2(x[0], two(s)), e.v[2 * h + 1] = mul2(x[1], two(s));
  }
  if (!VEC && n < 8) e.cut(n);
  return e;
}

// ----------------------------------------------------------------------- stores

// A thread's 8 columns to a row.  VEC: at once; else by way of the warp's own 1 KB,
// each store along the row (lane_col: the warp's first column and the lane).
template <bool VEC>
__device__ __forceinline__ void store_row(bf16* row, uint4 q, int col, int d, float* warp_row) {
  if constexpr (VEC) {
    if (col < d) __stcs(reinterpret_cast<uint4*>(row + col), q);
  } else {
    const int lane = threadIdx.x & 31, lane_col = col - 7 * lane;
    __syncwarp();
    reinterpret_cast<uint4*>(warp_row)[lane] = q;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane_col + 32 * i < d) row[lane_col + 32 * i] = reinterpret_cast<bf16*>(warp_row)[lane + 32 * i];
  }
}
template <bool VEC>
__device__ __forceinline__ void store_row(float* row, const Eight& e, int col, int d, float* warp_row) {
  const float4 a = make_float4(e.v[0].x, e.v[0].y, e.v[1].x, e.v[1].y), b = make_float4(e.v[2].x, e.v[2].y, e.v[3].x, e.v[3].y);
  if constexpr (VEC) {
    if (col >= d) return;
    __stcs(reinterpret_cast<float4*>(row + col), a);
    __stcs(reinterpret_cast<float4*>(row + col) + 1, b);
  } else {
    const int lane = threadIdx.x & 31, lane_col = col - 7 * lane;
    __syncwarp();
    reinterpret_cast<float4*>(warp_row)[lane * 2] = a;
    reinterpret_cast<float4*>(warp_row)[lane * 2 + 1] = b;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane_col + 32 * i < d) row[lane_col + 32 * i] = warp_row[lane + 32 * i];
  }
}
template <bool VEC>
__device__ __forceinline__ void store_row(bf16* row, const Eight& e, int col, int d, float* warp_row) {
  store_row<VEC>(row, pack(e), col, d, warp_row);
}

// The thread's 8 columns of a row of T, held in 8 bits; zeros behind the row's end.
template <typename T, bool VEC>
__device__ __forceinline__ void store_rows8(const Rows8& r, int t, const Shape& a, const Eight& e, int col, float* warp_row) {
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) most = max(most, moe::abs_bits(e.get(i)));
  for (int o = a.group_lanes >> 1; o; o >>= 1) most = max(most, __shfl_xor_sync(kAll, most, o));
  const bf16 s = moe::rows8_scale<T>(most);
  const uint2 word = moe::rows8_codes<T>(e.v, s);
  const int lane = threadIdx.x & 31;
  if constexpr (VEC) {
    if (col < a.d) __stcs(reinterpret_cast<uint2*>(r.codes + (long long)t * a.d + col), word);
  } else {
    const int lane_col = col - 7 * lane;
    __syncwarp();
    reinterpret_cast<uint2*>(warp_row)[lane] = word;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane_col + 32 * i < a.d) r.codes[(long long)t * a.d + lane_col + 32 * i] = reinterpret_cast<int8_t*>(warp_row)[lane + 32 * i];
  }
  if (col < a.d && (lane & (a.group_lanes - 1)) == 0) r.scales[(long long)t * a.groups + (col >> a.group_log)] = s;
}

// ------------------------------------------------------------------- parameters

__device__ __forceinline__ Eight load_params(const void* p, int f32, int col, int n, float none, float plus) {
  Eight e{};
  if (!p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) e.v[i] = two(none);
  } else if (n == 8 && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
    uint32_t w[4];
    if (f32) {
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + col);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        put_words(q[h], w);
        e.v[2 * h] = make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
        e.v[2 * h + 1] = make_float2(__uint_as_float(w[2]), __uint_as_float(w[3]));
      }
    } else {
      put_words(*reinterpret_cast<const uint4*>(static_cast<const bf16*>(p) + col), w);
      e = unpack(w);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) e.v[i] = add2(e.v[i], two(plus));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) e.set(i, plus + (f32 ? static_cast<const float*>(p)[col + i] : __bfloat162float(static_cast<const bf16*>(p)[col + i])));
  }
  return e;
}

// Eight numbers a unit in shared memory, in two planes.
struct Kept {
  float4* base;
  int units;
  __device__ __forceinline__ void write(int i, int unit, const Eight& e) const {
    base[(2 * i) * units + unit] = make_float4(e.v[0].x, e.v[0].y, e.v[1].x, e.v[1].y);
    base[(2 * i + 1) * units + unit] = make_float4(e.v[2].x, e.v[2].y, e.v[3].x, e.v[3].y);
  }
  __device__ __forceinline__ Eight read(int i, int unit) const {
    const float4 a = base[(2 * i) * units + unit], b = base[(2 * i + 1) * units + unit];
    Eight e;
    e.v[0] = make_float2(a.x, a.y), e.v[1] = make_float2(a.z, a.w), e.v[2] = make_float2(b.x, b.y), e.v[3] = make_float2(b.z, b.w);
    return e;
  }
};

// ------------------------------------------------------------------------- sums

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// Four sums over a warp at once: two exchanges hand the lanes one of the four each,
// three more add it up; lanes 0, 8, 16 and 24 have v.x, v.y, v.z, v.w.
__device__ __forceinline__ float warp_sum4(float4 v) {
  const int lane = threadIdx.x & 31;
  const bool up = lane & 16, right = lane & 8;
  float a = (up ? v.z : v.x) + __shfl_xor_sync(kAll, up ? v.x : v.z, 16);
  const float b = (up ? v.w : v.y) + __shfl_xor_sync(kAll, up ? v.y : v.w, 16);
  a = (right ? b : a) + __shfl_xor_sync(kAll, right ? a : b, 8);
#pragma unroll
  for (int o = 4; o; o >>= 1) a += __shfl_xor_sync(kAll, a, o);
  return a;
}

// The blocks of a cluster exchange their warps' sums; a single block's warps too.
struct Team {
  float4* parts;                 // of all warps, twice: for this exchange and the last one
  int blocks, rank, warps, warp; // warps: of the whole team; warp: of all
  int turn = 0;

  __device__ __forceinline__ Team(char* at) : parts(reinterpret_cast<float4*>(at)) {
    uint32_t n, r;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    blocks = (int)n, rank = (int)r, warps = (int)(n * blockDim.x / 32);
    warp = (int)(r * (blockDim.x / 32) + threadIdx.x / 32);
  }
  // What a warp's lane (of every eighth, or the first alone) has of its sums to every
  // block, and the wait for all of them.
  __device__ __forceinline__ void put(float* to, float v, bool mine) const {
    if (blocks == 1) {
      if (mine) *to = v;
    } else if (mine) {
      for (int b = 0; b < blocks; ++b)
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(moe::mapa_shared(moe::smem_u32(to), (uint32_t)b)), "f"(v) : "memory");
    }
  }
  __device__ __forceinline__ void exchange() const {
    if (blocks > 1) asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    else __syncthreads();
  }
  // N fours of sums over all threads of the team
  template <int N>
  __device__ __forceinline__ void sum(float4 (&v)[N]) {
    const int lane = threadIdx.x & 31;
    float mine[N];
#pragma unroll
    for (int q = 0; q < N; ++q) mine[q] = warp_sum4(v[q]);
    if (warps > 1) {
      float4* at = parts + turn * N * warps;
      turn ^= 1;
#pragma unroll
      for (int q = 0; q < N; ++q) put(reinterpret_cast<float*>(at + q * warps + warp) + (lane >> 3), mine[q], (lane & 7) == 0);
      exchange();
#pragma unroll
      for (int q = 0; q < N; ++q) {
        float4 t = lane < warps ? at[q * warps + lane] : make_float4(0.f, 0.f, 0.f, 0.f);
        if (blocks > 1)
          for (int w = lane + 32; w < warps; w += 32) {
            const float4 p = at[q * warps + w];
            t.x += p.x, t.y += p.y, t.z += p.z, t.w += p.w;
          }
        mine[q] = warp_sum4(t);
      }
    }
#pragma unroll
    for (int q = 0; q < N; ++q)
      v[q] = make_float4(__shfl_sync(kAll, mine[q], 0), __shfl_sync(kAll, mine[q], 8), __shfl_sync(kAll, mine[q], 16),
                         __shfl_sync(kAll, mine[q], 24));
  }
  // one sum
  __device__ __forceinline__ float sum(float v) {
    const int lane = threadIdx.x & 31;
    v = warp_sum(v);
    if (warps == 1) return v;
    float* at = reinterpret_cast<float*>(parts) + turn * warps;
    turn ^= 1;
    put(at + warp, v, lane == 0);
    exchange();
    if (blocks == 1 && warps <= 16) {
      float s = (lane & 15) < warps ? at[lane & 15] : 0.f;
#pragma unroll
      for (int o = 8; o; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
      return s;
    }
    float s = 0.f;
    for (int w = lane; w < warps; w += 32) s += at[w];
    return warp_sum(s);
  }
};

// A norm's mean and rstd of the team's row, CH eights of it in each thread, zeros behind
// its end; n: how many of them are columns.
template <bool LAYER, int CH>
__device__ __forceinline__ float2 moments(Team& team, const Eight (&e)[CH], const int (&n)[CH], float inv_d, float eps) {
  float mean = 0.f;
  if (LAYER) {
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) s = add2(s, e[c].v[j]);
    mean = team.sum(s.x + s.y) * inv_d;
  }
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    Eight off = e[c];
    if (LAYER) {
#pragma unroll
      for (int j = 0; j < 4; ++j) off.v[j] = add2(off.v[j], two(-mean));
      if (n[c] < 8) off.cut(n[c]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) s = fma2(off.v[j], off.v[j], s);
  }
  return make_float2(mean, rsqrtf(fmaf(team.sum(s.x + s.y), inv_d, eps)));
}

// Before anything is under way: slots of columns behind the row's end, which no copy
// reaches, are read as zeros; and a cluster's blocks all have to run before one writes
// to another.
__device__ __forceinline__ void begin(const Shape& a, const Team& team, char* smem, int columns) {
  if (columns > a.d) {
    for (int o = threadIdx.x; o < a.stages * a.stage / 16; o += blockDim.x) reinterpret_cast<uint4*>(smem)[o] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
  if (team.blocks > 1) moe::cluster_sync();
}

// Until the oldest of a.stages rows under way has come.
template <bool VEC>
__device__ __forceinline__ void wait_copies(int stages) {
  if (stages == 2) moe::cp_async_wait<1>();
  else if (stages == 3) moe::cp_async_wait<2>();
  else moe::cp_async_wait<3>();
  if (!VEC) __syncwarp();
}

// ------------------------------------------------------------------------- host

template <typename T>
bool rows_aligned(const Rows<T>& r) {  // for 16-byte vectors
  return reinterpret_cast<uintptr_t>(r.p) % 16 == 0 && r.stride % 16 == 0;
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t type_size(int type) { return type == MOE_TYPE_F32 ? 4 : 2; }

// How a kernel is laid over rows: eights of a lane, blocks of a row, their threads, and
// how many of them an SM is given.
struct Plan {
  int chunks, blocks, threads, per_sm, smem;
};

// A block's threads and shared memory for `chunks` eights a lane: as many blocks to a
// row as it takes for two stages to fit, as many blocks to an SM as it then has
// room for, up to sm_threads threads, and as many stages, up to kMaxStages.
Plan lay_out(Shape* a, int chunks, int block_threads, int sm_threads, const int (&field_bytes)[5], int kept, int quads, bool vec) {
  constexpr int least = 2;
  Plan p;
  p.chunks = chunks;
  const int lanes = (a->d + 7) / 8;
  int rest = 0, parts = 0, units = 0;
  auto with = [&](int blocks) {
    p.blocks = blocks;
    p.threads = ((lanes + blocks * chunks - 1) / (blocks * chunks) + 31) / 32 * 32;
    units = p.threads * chunks;
    a->stage = 0;
    // a unit's bytes, and behind them a warp's piece (16 bytes, 8 of codes) of rows that are not aligned
    for (int i = 0; i < 5; ++i) a->field[i] = a->stage, a->stage += field_bytes[i] * units + (vec || !field_bytes[i] ? 0 : units / 2);
    parts = 2 * quads * p.blocks * p.threads / 32 * 16;
    rest = kept * 32 * units + (vec ? 0 : p.threads * 32) + parts;
    return p.threads <= block_threads && least * a->stage + rest <= kRing;
  };
  int blocks = 1;
  while (!with(blocks) && blocks < kMaxCluster) blocks *= 2;
  p.per_sm = std::max(1, std::min({32, sm_threads / p.threads, kRing / (least * a->stage + rest)}));
  a->stages = std::max(least, std::min(kMaxStages, (kRing / p.per_sm - rest) / std::max(1, a->stage)));
  a->vec = a->stages * a->stage;
  a->out = a->vec + kept * 32 * units;
  a->parts = a->vec + rest - parts;
  p.smem = a->vec + rest;
  return p;
}

template <typename, bool, bool, int, int, bool>
struct ForwardKernel;
template <typename, bool, bool, int, int>
struct BackwardKernel;

// Shared memory beyond 48 KB is asked for once a kernel and device.
template <typename Kernel, typename F>
cudaError_t allow_smem(F* kernel) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <typename... A>
cudaError_t launch(void (*kernel)(A...), unsigned grid, int cluster, int threads, int smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // kernels wait themselves
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

struct moe_norm {
  int d, pre, post, gate, group;
  float eps, scale, one;
  float* sums = nullptr;  // of the teams of a backward pass
  int device = -1;
};

namespace {

// Rows that a gradient takes at once, at most: its teams.
int most_teams(const moe_norm* h) {
  int most = kSms;
  for (int chunks = 1; chunks <= 2; ++chunks)
    most = std::max(most, kSms * std::min(32, kThreads / (((h->d + 8 * chunks - 1) / (8 * chunks) + 31) / 32 * 32)));
  return most;
}

Shape shape_of(const moe_norm* h, int T) {
  Shape a = {};
  a.T = T;
  a.d = h->d;
  a.scale = h->scale;
  a.eps = h->eps;
  a.one = h->one;
  a.groups = (h->d + h->group - 1) / h->group;
  a.group_lanes = h->group / 8;
  a.group_log = h->group == 32 ? 5 : h->group == 64 ? 6 : 7;
  return a;
}

// Eights of a lane.  What a row costs a thread beside its columns (the exchanges, the
// root, finding its tensors) is shared by two of them (8192 x 4096, gradient: 108 us
// with one, 95 with two); with few rows more threads are sooner done (512 x 4096: 16.1
// and 17.7), unless a second block would have to join them (1024 x 16384: 150 and 73).
int chunks_of(int d, int T, int most) {
  const int lanes = (d + 7) / 8;
  if (T <= 2 * kSms || (T <= 8 * kSms && lanes <= kThreads)) return 1;
  int c = 1;
  while (c < most && c * 32 < lanes) c *= 2;
  return c;
}

// f(aligned, pre norm a layer norm, post norm, eights of a lane), as types.
template <typename F>
cudaError_t by_kind(const moe_norm* h, bool vec, int chunks, F&& f) {
  constexpr std::integral_constant<int, kNone> none{};
  constexpr std::integral_constant<int, kRms> rms{};
  constexpr std::integral_constant<int, kLayer> layer{};
  auto by_post = [&](auto v, auto pre, auto c) {
    return h->post == kNone ? f(v, pre, none, c) : h->post == kRms ? f(v, pre, rms, c) : f(v, pre, layer, c);
  };
  auto by_chunks = [&](auto v, auto pre) {
    constexpr std::integral_constant<int, 1> one{};
    if constexpr (decltype(v)::value) return chunks == 1 ? by_post(v, pre, one) : by_post(v, pre, std::integral_constant<int, 2>{});
    else return by_post(v, pre, one);  // rows that are not aligned keep more registers busy
  };
  auto by_pre = [&](auto v) { return h->pre == kLayer ? by_chunks(v, std::true_type{}) : by_chunks(v, std::false_type{}); };
  return vec ? by_pre(std::true_type{}) : by_pre(std::false_type{});
}

const char* check_rows(const moe_norm* h, const void* p, int type, long long stride) {
  if (!p) return nullptr;
  if (!aligned(p, type_size(type))) return "tensors must be aligned to their type";
  if (stride < h->d) return "rows overlap: a row stride is below d";
  if (stride >= (1ll << 32) / (long long)type_size(type)) return "a row stride must be below 4 GB";
  return nullptr;
}

// Without rows (T = 0) what has one a token is an empty tensor, whose pointer may be null.
const char* check_params(const moe_norm* h, const moe_norm_params* p, int T) {
  if (!p) return "null params";
  if (p->type != MOE_TYPE_F32 && p->type != MOE_TYPE_BF16) return "gains and shifts are MOE_TYPE_F32 or MOE_TYPE_BF16";
  const void* all[] = {p->pre_gain, p->pre_shift, p->post_gain, p->post_shift};
  for (const void* q : all)
    if (!aligned(q, type_size(p->type))) return "gains and shifts must be aligned to their type";
  if (h->pre == kNone && p->pre_gain) return "a gain for a norm that the handle does not have";
  if (h->post == kNone && p->post_gain) return "a gain for a norm that the handle does not have";
  if ((h->pre != kLayer && p->pre_shift) || (h->post != kLayer && p->post_shift)) return "only layer norms have a shift";
  const bool empty_gate = T == 0 && !p->gate && (h->gate == MOE_GATE_TOKEN || h->gate == MOE_GATE_ELEMENT);
  if ((h->gate != MOE_GATE_NONE) != (p->gate != nullptr) && !empty_gate) return "the gate must be given as the handle has it";
  const size_t gate_size = h->gate == MOE_GATE_CHANNEL ? type_size(p->type) : h->gate == MOE_GATE_TOKEN ? 4 : 2;
  if (!aligned(p->gate, gate_size)) return "the gate must be aligned to its type";
  if (h->gate == MOE_GATE_ELEMENT) return check_rows(h, p->gate, MOE_TYPE_BF16, p->gate_stride);
  return nullptr;
}

const char* check_rows8(const moe_rows8* r, int T) {
  if (!r || T == 0) return nullptr;
  if (!r->codes || !r->scales) return "null codes or scales of 8-bit rows";
  if (!aligned(r->scales, 4)) return "scales of 8-bit rows must be 4-byte aligned";
  return nullptr;
}

Rows8 rows8_of(const moe_rows8* r) {
  return r ? Rows8{static_cast<int8_t*>(r->codes), static_cast<bf16*>(r->scales)} : Rows8{nullptr, nullptr};
}

template <typename T>
Rows<T> rows_of(const void* p, long long stride) {
  return Rows<T>{static_cast<T*>(const_cast<void*>(p)), (uint32_t)(stride * (long long)sizeof(T))};
}

}  // namespace

