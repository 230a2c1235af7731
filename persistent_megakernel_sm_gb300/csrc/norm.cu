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
// What bounds both is HBM.  A block holds a row (a cluster of 2, 4 or 8 blocks one
// of more than 4096, 8192, 16384 columns), a lane 8 consecutive columns of it, and
// goes over its rows as a pipeline: while one row is finished, the next one's sums
// are taken and the rows behind are on their way.  Rows that are aligned come by
// asynchronous 16-byte copies into slots that belong to the thread that reads them
// (so that no barrier guards them), others a warp's 256 columns at a time, each
// load along the row.  Gains and shifts stay in shared memory.  Sums over rows are
// kept in registers, written once a block and added by a second kernel in a fixed
// order.
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
constexpr int kThreads = 512;            // of a block, at most: 4096 columns
constexpr int kMaxStages = 4;            // rows under way
constexpr int kSms = 152;
constexpr int kRing = 196 * 1024;        // shared memory of an SM for slots, gains and shifts
constexpr unsigned kAll = 0xffffffffu;
constexpr int kNone = MOE_NORM_NONE, kRms = MOE_NORM_RMS, kLayer = MOE_NORM_LAYER;

__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ void from_float(float v, float* o) { *o = v; }
__device__ __forceinline__ void from_float(float v, bf16* o) { *o = __float2bfloat16_rn(v); }
__device__ __forceinline__ float rounded(float v, const float*) { return v; }
__device__ __forceinline__ float rounded(float v, const bf16*) { return __bfloat162float(__float2bfloat16_rn(v)); }

__device__ __forceinline__ void unpack(uint4 q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
}

__device__ __forceinline__ uint4 pack(const float (&v)[8]) {
  union {
    __nv_bfloat162 b[4];
    uint4 q;
  } u;
#pragma unroll
  for (int i = 0; i < 4; ++i) u.b[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  return u.q;
}

// cp.async of 16, 8 or (n of them read, the rest zero) 4 bytes.
__device__ __forceinline__ void copy8(void* to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(moe::smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(void* to, const void* from, int n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(moe::smem_u32(to)), "l"(from), "r"(n) : "memory");
}

// Rows of a tensor: where row 0 begins and how far the next is, in elements.
template <typename T>
struct Rows {
  T* p;
  long long stride;
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
  int groups, group_lanes;  // of 8-bit rows
  int pre, post, gate;
  float scale, eps, one;    // one: 1 where gains are stored less 1
};

// ------------------------------------------------------------- a thread's slots

// Where a thread finds the 8 columns of the rows under way.  A field is one plane
// of 16 bytes a thread (8 bf16), two (fp32: columns 0 to 3 and 4 to 7), or 8 bytes
// and 4 (codes and their scale).
struct Slots {
  char* base;      // of the stage
  int threads;

  __device__ __forceinline__ uint4* plane(int field, int half = 0) const {
    return reinterpret_cast<uint4*>(base + field) + half * threads;
  }
  __device__ __forceinline__ void read(int field, int tid, const bf16*, float (&v)[8]) const { unpack(plane(field)[tid], v); }
  __device__ __forceinline__ void read(int field, int tid, const float*, float (&v)[8]) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 q = reinterpret_cast<const float4*>(plane(field, h))[tid];
      v[4 * h] = q.x, v[4 * h + 1] = q.y, v[4 * h + 2] = q.z, v[4 * h + 3] = q.w;
    }
  }
  __device__ __forceinline__ uint2* codes(int field) const { return reinterpret_cast<uint2*>(base + field); }
  __device__ __forceinline__ uint32_t* scales(int field) const {
    return reinterpret_cast<uint32_t*>(base + field + 8 * threads);
  }
  // `odd`: which half of the word the scale is in
  __device__ __forceinline__ void read8(int field, int tid, int odd, float (&v)[8]) const {
    const uint2 q = codes(field)[tid];
    moe::rows8_floats(q.x, v);
    moe::rows8_floats(q.y, v + 4);
    const uint32_t w = scales(field)[tid];
    const float s = __uint_as_float(odd ? w & 0xffff0000u : w << 16);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= s;
  }
};

// One tensor's part of a row on its way into a field: `start` asks for it, `end`
// puts it in place.  VEC: by asynchronous copies, `end` has nothing to do.
template <typename T, bool VEC>
struct Fetch {
  T v[VEC ? 1 : 8];

  // `col`: the thread's first column, `lane_col`: the warp's first plus the lane
  __device__ __forceinline__ void start(const Slots& s, int field, int tid, const T* row, int col, int lane_col, int d) {
    if constexpr (VEC) {
      if (col < d) {
        moe::cp_async16(s.plane(field) + tid, row + col);
        if (sizeof(T) == 4) moe::cp_async16(s.plane(field, 1) + tid, row + col + 4);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = lane_col + 32 * i < d ? row[lane_col + 32 * i] : T(0.f);
    }
  }
  __device__ __forceinline__ void end(const Slots& s, int field, int tid) const {
    if constexpr (!VEC) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = (tid & ~31) * 8 + 32 * i + (tid & 31);  // the block's column
        char* to = sizeof(T) == 4 ? reinterpret_cast<char*>(s.plane(field, e >> 2 & 1)) + (e >> 3) * 16 + (e & 3) * 4
                                  : reinterpret_cast<char*>(s.plane(field)) + e * 2;
        *reinterpret_cast<T*>(to) = v[i];
      }
    }
  }
};

template <bool VEC>
struct Fetch8 {
  int8_t v[VEC ? 1 : 8];
  bf16 s;

  __device__ __forceinline__ void start(const Slots& at, int field, int tid, const Rows8& r, long long row, const Shape& a,
                                        int col, int lane_col) {
    const long long scale = row * a.groups + col / (8 * a.group_lanes);
    if constexpr (VEC) {
      if (col < a.d) {
        copy8(at.codes(field) + tid, r.codes + row * a.d + col);
        // the word that the scale is in; the tensor may end in its middle
        const bool last = scale == (long long)a.T * a.groups - 1 && !(scale & 1);
        copy4(at.scales(field) + tid, r.scales + (scale & ~1ll), last ? 2 : 4);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = lane_col + 32 * i < a.d ? r.codes[row * a.d + lane_col + 32 * i] : (int8_t)0;
      s = col < a.d ? r.scales[scale] : bf16(0.f);
    }
  }
  __device__ __forceinline__ void end(const Slots& at, int field, int tid) const {
    if constexpr (!VEC) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        reinterpret_cast<int8_t*>(at.codes(field))[(tid & ~31) * 8 + 32 * i + (tid & 31)] = v[i];
      at.scales(field)[tid] = (uint32_t)__bfloat16_as_ushort(s) * 0x00010001u;  // whichever half is read
    }
  }
};

// A thread's 8 columns to a row.  VEC: at once; else by way of the warp's own 1 KB,
// each store along the row.
template <bool VEC, typename T>
__device__ __forceinline__ void store_row(T* row, const float (&v)[8], int col, int lane_col, int d, float* warp_row) {
  if constexpr (VEC) {
    if (col >= d) return;
    if constexpr (sizeof(T) == 2) {
      __stcs(reinterpret_cast<uint4*>(row + col), pack(v));
    } else {
      __stcs(reinterpret_cast<float4*>(row + col), make_float4(v[0], v[1], v[2], v[3]));
      __stcs(reinterpret_cast<float4*>(row + col) + 1, make_float4(v[4], v[5], v[6], v[7]));
    }
  } else {
    const int lane = threadIdx.x & 31;
    float4* mine = reinterpret_cast<float4*>(warp_row) + lane * 2;
    __syncwarp();
    mine[0] = make_float4(v[0], v[1], v[2], v[3]);
    mine[1] = make_float4(v[4], v[5], v[6], v[7]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane_col + 32 * i < d) from_float(warp_row[lane + 32 * i], row + lane_col + 32 * i);
  }
}

// The thread's 8 columns of a row of T, held in 8 bits; zeros behind the row's end.
template <typename T, bool VEC>
__device__ __forceinline__ void store_rows8(const Rows8& r, long long row, const Shape& a, const float (&v)[8], int col,
                                            int lane_col, float* warp_row) {
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) most = max(most, moe::abs_bits(v[i]));
  for (int o = a.group_lanes >> 1; o; o >>= 1) most = max(most, __shfl_xor_sync(kAll, most, o));
  const bf16 s = moe::rows8_scale(most);
  uint32_t word[2];
  moe::rows8_codes<T>(v, s, word);
  const int lane = threadIdx.x & 31;
  if constexpr (VEC) {
    if (col < a.d) __stcs(reinterpret_cast<uint2*>(r.codes + row * a.d + col), make_uint2(word[0], word[1]));
  } else {
    uint2* bytes = reinterpret_cast<uint2*>(warp_row);
    __syncwarp();
    bytes[lane] = make_uint2(word[0], word[1]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane_col + 32 * i < a.d) r.codes[row * a.d + lane_col + 32 * i] = reinterpret_cast<int8_t*>(bytes)[lane + 32 * i];
  }
  if (col < a.d && (lane & (a.group_lanes - 1)) == 0) r.scales[row * a.groups + col / (8 * a.group_lanes)] = s;
}

// ------------------------------------------------------------------------- sums

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// Mean and summed squares about it of n values, put together with another n's
// (Chan, Golub and LeVeque): no large sums are taken from one another.
struct Moments {
  float n, mean, m2;
};

__device__ __forceinline__ Moments both(const Moments& a, const Moments& b) {
  if (a.n == 0.f) return b;  // an empty side's square could overflow
  if (b.n == 0.f) return a;
  const float n = a.n + b.n;
  const float part = __fdividef(b.n, n), off = b.mean - a.mean;
  return Moments{n, fmaf(off, part, a.mean), a.m2 + fmaf(off * off, a.n * part, b.m2)};
}

__device__ __forceinline__ Moments warp_moments(Moments m) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
    m = both(m, Moments{__shfl_xor_sync(kAll, m.n, o), __shfl_xor_sync(kAll, m.mean, o), __shfl_xor_sync(kAll, m.m2, o)});
  // the two sides of an exchange round differently: one lane's for all
  return Moments{m.n, __shfl_sync(kAll, m.mean, 0), __shfl_sync(kAll, m.m2, 0)};
}

// A warp's part of what a norm is made of: (sum of squares, -) or (mean, squares about it).
__device__ __forceinline__ float2 warp_part(const float (&v)[8], int n, int kind) {
  if (kind == kLayer) {
    float mean = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) mean += i < n ? v[i] : 0.f;
    mean = n ? mean / (float)n : 0.f;
    float m2 = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m2 += i < n ? (v[i] - mean) * (v[i] - mean) : 0.f;
    const Moments m = warp_moments(Moments{(float)n, mean, m2});
    return make_float2(m.mean, m.m2);
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(v[i], v[i], s);  // zeros behind the row's end
  return make_float2(warp_sum(s), 0.f);
}

// (mean, rstd) from every warp's part.
__device__ __forceinline__ float2 whole(const float2* parts, int stride, int warps, int kind, int d, float eps) {
  const int lane = threadIdx.x & 31;
  float mean = 0.f, m2;
  if (kind == kLayer) {
    Moments m{0.f, 0.f, 0.f};
    for (int w = lane; w < warps; w += 32) {
      const float2 p = parts[w * stride];
      m = both(m, Moments{(float)max(0, min(256, d - 256 * w)), p.x, p.y});
    }
    m = warp_moments(m);
    mean = m.mean, m2 = m.m2;
  } else {
    float s = 0.f;
    for (int w = lane; w < warps; w += 32) s += parts[w * stride].x;
    m2 = warp_sum(s);
  }
  return make_float2(mean, __frsqrt_rn(m2 / (float)d + eps));
}

// ---------------------------------------------------------------------- forward

template <typename R>
struct Forward {
  Shape a;
  Rows<const R> residual;
  Rows<const bf16> y, gate_rows;  // null: none
  const float* gate_tokens;
  const void *pre_gain, *pre_shift, *post_gain, *post_shift, *gate_columns;  // null: none
  int params_f32;
  Rows<R> out;
  Rows<bf16> norm;
  float4* stats;
  Rows8 out8, y8;
};

__device__ __forceinline__ void load_params(const void* p, int f32, int col, int n, float none, float plus, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = !p ? none : i >= n ? 0.f
                              : plus + (f32 ? static_cast<const float*>(p)[col + i]
                                            : __bfloat162float(static_cast<const bf16*>(p)[col + i]));
}

// Eight numbers a thread keeps in shared memory, in two planes.
struct Kept {
  float4* base;
  int threads, tid;
  __device__ __forceinline__ void write(int i, const float (&v)[8]) const {
    base[(2 * i) * threads + tid] = make_float4(v[0], v[1], v[2], v[3]);
    base[(2 * i + 1) * threads + tid] = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ __forceinline__ void read(int i, float (&v)[8]) const {
    const float4 a = base[(2 * i) * threads + tid], b = base[(2 * i + 1) * threads + tid];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};

// The blocks of a cluster exchange their warps' parts; a single block's warps too.
struct Team {
  int blocks, rank, warps;  // warps: of the whole team

  __device__ __forceinline__ Team() {
    uint32_t n, r;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    blocks = (int)n, rank = (int)r, warps = (int)(n * blockDim.x / 32);
  }
  // one lane writes to every block
  __device__ __forceinline__ void write(float4* at, float4 v) const {
    if (blocks == 1) {
      *at = v;
    } else {
      for (int b = 0; b < blocks; ++b) {
        const uint32_t to = moe::mapa_shared(moe::smem_u32(at), (uint32_t)b);
        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                     : "memory");
      }
    }
  }
  __device__ __forceinline__ void arrive() const {
    if (blocks > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  }
  __device__ __forceinline__ void wait() const {
    if (blocks > 1)
      asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    else
      __syncthreads();
  }
};

__device__ __forceinline__ void wait_copies(int stages) {  // the row to be read next has come
  if (stages == 2) moe::cp_async_wait<0>();
  else if (stages == 3) moe::cp_async_wait<1>();
  else moe::cp_async_wait<2>();
}

// Before anything is under way: the copies leave the slots of columns behind the
// row's end alone, which are read as zeros; and a cluster's blocks all have to run
// before one writes to another.
template <bool VEC>
__device__ __forceinline__ void begin(const Shape& a, const Team& team, char* smem, int tid, int threads) {
  if (VEC && team.blocks * threads * 8 > a.d) {
    for (int o = tid; o < a.stages * a.stage / 16; o += threads) reinterpret_cast<uint4*>(smem)[o] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
  if (team.blocks > 1) moe::cluster_sync();
}

// Of the rows team, team + teams, ...: iteration i takes the post norm's sums of
// row i, writes row i - 2's norm, and row i - 1's sum with the sums of its norm.
template <typename R, bool VEC>
__global__ void __launch_bounds__(kThreads, VEC ? 2 : 1) norm_forward(const __grid_constant__ Forward<R> f) {
  extern __shared__ __align__(16) char smem[];
  const Shape& a = f.a;
  const Team team;
  const int tid = threadIdx.x, lane = tid & 31, threads = blockDim.x, warp = team.rank * (threads / 32) + (tid >> 5);
  const int col = (team.rank * threads + tid) * 8, lane_col = (team.rank * threads + (tid & ~31)) * 8 + lane;
  const int n = max(0, min(8, a.d - col));
  const int first = blockIdx.x / team.blocks, step = gridDim.x / team.blocks;
  const int rows = first < a.T ? (a.T - first - 1) / step + 1 : 0;
  float* warp_row = reinterpret_cast<float*>(smem + a.out) + (tid >> 5) * 256;
  const Kept kept{reinterpret_cast<float4*>(smem + a.vec), threads, tid};
  auto row_at = [&](int i) { return (long long)first + (long long)i * step; };
  auto slots = [&](int i) { return Slots{smem + i % a.stages * a.stage, threads}; };

  wait_for_previous_kernel();
  let_next_kernel_start();
  begin<VEC>(a, team, smem, tid, threads);
  Fetch<R, VEC> fr;
  Fetch<bf16, VEC> fy, fg;
  auto start = [&](int i) {
    if (i < rows) {
      const long long t = row_at(i);
      const Slots s = slots(i);
      fr.start(s, a.field[0], tid, f.residual.p + t * f.residual.stride, col, lane_col, a.d);
      if (f.y.p) fy.start(s, a.field[1], tid, f.y.p + t * f.y.stride, col, lane_col, a.d);
      if (f.gate_rows.p) fg.start(s, a.field[2], tid, f.gate_rows.p + t * f.gate_rows.stride, col, lane_col, a.d);
    }
    if (VEC) moe::cp_async_commit();
  };
  auto end = [&](int i) {
    if (VEC || i >= rows) return;
    const Slots s = slots(i);
    __syncwarp();
    fr.end(s, a.field[0], tid);
    if (f.y.p) fy.end(s, a.field[1], tid);
    if (f.gate_rows.p) fg.end(s, a.field[2], tid);
    __syncwarp();
  };
  for (int i = 0; i < a.stages - 1; ++i) start(i), end(i);

  {  // s g gain and s g shift of the post norm, gain and shift of the pre norm
    float gate[8], v[8];
    load_params(f.gate_columns, f.params_f32, col, n, 1.f, 0.f, gate);
    load_params(f.post_gain, f.params_f32, col, n, 1.f, a.one, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= gate[i] * a.scale;
    kept.write(0, v);
    load_params(f.pre_gain, f.params_f32, col, n, 1.f, a.one, v);
    kept.write(1, v);
    if (f.post_shift) {
      load_params(f.post_shift, f.params_f32, col, n, 0.f, 0.f, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= gate[i] * a.scale;
      kept.write(2, v);
    }
    if (f.pre_shift) {
      load_params(f.pre_shift, f.params_f32, col, n, 0.f, 0.f, v);
      kept.write(3, v);
    }
  }

  float sum[8];                          // row i - 2's, then row i - 1's
  float2 post = make_float2(0.f, 1.f), pre = make_float2(0.f, 1.f), post_before = post;
  float gate_t = 1.f, gate_next = 1.f;
#pragma unroll 1
  for (int i = 0; i < rows + 2; ++i) {
    if (!VEC) start(i - 1 + a.stages);
    float2 post_part = make_float2(0.f, 0.f), pre_part = make_float2(0.f, 0.f);
    if (VEC) wait_copies(a.stages);
    if (i < rows) {
      if (f.gate_tokens) gate_next = f.gate_tokens[row_at(i)];
      if (f.y.p && (a.post != kNone || f.y8.codes)) {
        float y[8];
        slots(i).read(a.field[1], tid, (const bf16*)nullptr, y);
        if (a.post != kNone) post_part = warp_part(y, n, a.post);
        if (f.y8.codes) store_rows8<bf16, VEC>(f.y8, row_at(i), a, y, col, lane_col, warp_row);
      }
    }
    if (i >= 2) {
      const long long t = row_at(i - 2);
      if (f.norm.p) {
        float gain[8], v[8];
        kept.read(1, gain);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (sum[j] - pre.x) * pre.y * gain[j];
        if (f.pre_shift) {
          kept.read(3, gain);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] += gain[j];
        }
        store_row<VEC>(f.norm.p + t * f.norm.stride, v, col, lane_col, a.d, warp_row);
      }
      if (f.stats && warp == 0 && lane == 0) f.stats[t] = make_float4(post_before.x, post_before.y, pre.x, pre.y);
    }
    if (i >= 1 && i <= rows) {
      const long long t = row_at(i - 1);
      const Slots s = slots(i - 1);
      s.read(a.field[0], tid, (const R*)nullptr, sum);
      if (f.y.p) {
        float y[8], k[8];
        s.read(a.field[1], tid, (const bf16*)nullptr, y);
        kept.read(0, k);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = (y[j] - post.x) * post.y * k[j];
        if (f.post_shift) {
          kept.read(2, k);
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] += k[j];
        }
        if (f.gate_rows.p) {
          s.read(a.field[2], tid, (const bf16*)nullptr, k);
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] *= k[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = j < n ? rounded(fmaf(y[j], gate_t, sum[j]), (const R*)nullptr) : 0.f;
        store_row<VEC>(f.out.p + t * f.out.stride, sum, col, lane_col, a.d, warp_row);
      }
      if (f.out8.codes) store_rows8<R, VEC>(f.out8, t, a, sum, col, lane_col, warp_row);
      if (a.pre != kNone) pre_part = warp_part(sum, n, a.pre);
    }
    if (VEC) start(i - 1 + a.stages);
    else end(i - 1 + a.stages);
    float4* at = reinterpret_cast<float4*>(smem + a.parts) + (i & 1) * team.warps;
    if (lane == 0) team.write(&at[warp], make_float4(post_part.x, post_part.y, pre_part.x, pre_part.y));
    team.arrive();
    team.wait();
    post_before = post;
    gate_t = gate_next;
    if (a.post != kNone) post = whole(reinterpret_cast<const float2*>(at), 2, team.warps, a.post, a.d, a.eps);
    if (a.pre != kNone) pre = whole(reinterpret_cast<const float2*>(at) + 1, 2, team.warps, a.pre, a.d, a.eps);
  }
}

// --------------------------------------------------------------------- backward

template <typename R>
struct Backward {
  Shape a;
  Rows<const R> grad_out, kept_out;  // null: none; kept_out, y: null where they are kept in 8 bits
  Rows<const bf16> grad_norm, y, gate_rows;
  Rows8 out8, y8;
  const float4* stats;
  const float* gate_tokens;
  const void *pre_gain, *post_gain, *post_shift, *gate_columns;
  int params_f32;
  Rows<R> grad_residual;  // null: not wanted
  Rows<bf16> grad_y, grad_gate_rows;
  float* grad_gate_tokens;
  float* sums;            // [teams, 4, d]: gradient times u and gradient, of the pre norm and of the post norm
};

// The sums of a row, in the order in which they are reduced.
enum { kTU, kUV, kXV, kT, kV, kUW, kXW, kW, kUB, kXB, kB, kSums };

// Fours of them that a row has: kTU, kUV and kXV, with layer norms up to all.
__host__ __device__ constexpr int quads_of(bool pre_layer, int post) { return pre_layer || post == kLayer ? 3 : 1; }

template <typename R, bool VEC, bool PRE_LAYER, int POST>
__global__ void __launch_bounds__(kThreads) norm_backward(const __grid_constant__ Backward<R> f) {
  extern __shared__ __align__(16) char smem[];
  const Shape& a = f.a;
  const Team team;
  const int tid = threadIdx.x, lane = tid & 31, threads = blockDim.x, warp = team.rank * (threads / 32) + (tid >> 5);
  const int col = (team.rank * threads + tid) * 8, lane_col = (team.rank * threads + (tid & ~31)) * 8 + lane;
  const int n = max(0, min(8, a.d - col));
  const int first = blockIdx.x / team.blocks, step = gridDim.x / team.blocks;
  const int rows = first < a.T ? (a.T - first - 1) / step + 1 : 0;
  float* warp_row = reinterpret_cast<float*>(smem + a.out) + (tid >> 5) * 256;
  const Kept kept{reinterpret_cast<float4*>(smem + a.vec), threads, tid};
  auto row_at = [&](int i) { return (long long)first + (long long)i * step; };
  auto slots = [&](int i) { return Slots{smem + i % a.stages * a.stage, threads}; };
  const bool has_y = f.y.p || f.y8.codes;
  const bool has_norm = f.grad_norm.p != nullptr;
  const bool token_shift = POST == kLayer && f.grad_gate_tokens && f.post_shift;
  const int scale_group = col / (8 * a.group_lanes);

  wait_for_previous_kernel();
  let_next_kernel_start();
  begin<VEC>(a, team, smem, tid, threads);
  Fetch<R, VEC> fgo, fx;
  Fetch<bf16, VEC> fgn, fy, fg;
  Fetch8<VEC> fx8, fy8;
  auto start = [&](int i) {
    if (i < rows) {
      const long long t = row_at(i);
      const Slots s = slots(i);
      if (f.grad_out.p) fgo.start(s, a.field[0], tid, f.grad_out.p + t * f.grad_out.stride, col, lane_col, a.d);
      if (has_norm) {
        fgn.start(s, a.field[1], tid, f.grad_norm.p + t * f.grad_norm.stride, col, lane_col, a.d);
        if (f.out8.codes) fx8.start(s, a.field[2], tid, f.out8, t, a, col, lane_col);
        else fx.start(s, a.field[2], tid, f.kept_out.p + t * f.kept_out.stride, col, lane_col, a.d);
      }
      if (f.y8.codes) fy8.start(s, a.field[3], tid, f.y8, t, a, col, lane_col);
      else if (f.y.p) fy.start(s, a.field[3], tid, f.y.p + t * f.y.stride, col, lane_col, a.d);
      if (f.gate_rows.p) fg.start(s, a.field[4], tid, f.gate_rows.p + t * f.gate_rows.stride, col, lane_col, a.d);
    }
    if (VEC) moe::cp_async_commit();
  };
  auto end = [&](int i) {
    if (VEC || i >= rows) return;
    const Slots s = slots(i);
    __syncwarp();
    if (f.grad_out.p) fgo.end(s, a.field[0], tid);
    if (has_norm) {
      fgn.end(s, a.field[1], tid);
      if (f.out8.codes) fx8.end(s, a.field[2], tid);
      else fx.end(s, a.field[2], tid);
    }
    if (f.y8.codes) fy8.end(s, a.field[3], tid);
    else if (f.y.p) fy.end(s, a.field[3], tid);
    if (f.gate_rows.p) fg.end(s, a.field[4], tid);
    __syncwarp();
  };
  for (int i = 0; i < a.stages - 1; ++i) start(i), end(i);

  {  // the pre norm's gain; the post norm's, its shift and the gate's columns
    float v[8];
    load_params(f.pre_gain, f.params_f32, col, n, 1.f, a.one, v);
    kept.write(0, v);
    load_params(f.post_gain, f.params_f32, col, n, 1.f, a.one, v);
    kept.write(1, v);
    load_params(f.gate_columns, f.params_f32, col, n, 1.f, 0.f, v);
    kept.write(2, v);
    if (f.post_shift) {
      load_params(f.post_shift, f.params_f32, col, n, 0.f, 0.f, v);
      kept.write(3, v);
    }
  }

  // u of the pre norm and of the post norm (y itself where there is none)
  auto read_u = [&](int i, float4 st, float (&x)[8], float (&y)[8]) {
    const Slots s = slots(i);
    const long long t = row_at(i);
    const int odd = (int)((t * a.groups + scale_group) & 1);
    if (has_norm) {
      if (f.out8.codes) s.read8(a.field[2], tid, odd, x);
      else s.read(a.field[2], tid, (const R*)nullptr, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = PRE_LAYER ? (x[j] - st.z) * st.w : x[j] * st.w;
    }
    if (has_y) {
      if (f.y8.codes) s.read8(a.field[3], tid, odd, y);
      else s.read(a.field[3], tid, (const bf16*)nullptr, y);
      if (POST != kNone) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = POST == kLayer ? (y[j] - st.x) * st.y : y[j] * st.y;
      }
    }
  };
  // the gate's part that a thread's columns have of their own
  auto read_gate = [&](int i, float (&g)[8]) {
    if (f.gate_rows.p) slots(i).read(a.field[4], tid, (const bf16*)nullptr, g);
    else kept.read(2, g);
  };

  float acc_tu[8] = {}, acc_t[PRE_LAYER ? 8 : 1] = {}, acc_v[8] = {}, acc_g[POST == kLayer ? 8 : 1] = {};
  float4 st = make_float4(0.f, 1.f, 0.f, 1.f), st_next = st, st_ahead = st;
  float gate_t = 1.f, gate_next = 1.f, gate_ahead = 1.f;
  auto ahead = [&](int i) {  // a row's numbers, an iteration before its sums
    if (i >= rows) return;
    if (f.stats) st_ahead = __ldg(f.stats + row_at(i));
    if (f.gate_tokens) gate_ahead = __ldg(f.gate_tokens + row_at(i));
  };
  ahead(0);
  float total[kSums] = {};
  const bool sums_post = POST != kNone || f.grad_gate_tokens;
  const float inv_d = 1.f / (float)a.d;
#pragma unroll 1
  for (int i = 0; i < rows + 1; ++i) {
    if (!VEC) start(i - 1 + a.stages);
    st = st_next, gate_t = gate_next;
    st_next = st_ahead, gate_next = gate_ahead;
    ahead(i + 1);
    if (VEC) wait_copies(a.stages);
    float sum[kSums] = {};
    if (i < rows) {  // row i's sums
      const Slots s = slots(i);
      float x[8], y[8], gn[8], go[8], k[8];
      read_u(i, st_next, x, y);
      if (f.grad_out.p) {
        s.read(a.field[0], tid, (const R*)nullptr, go);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) go[j] = 0.f;
      }
      if (has_norm) {
        s.read(a.field[1], tid, (const bf16*)nullptr, gn);
        kept.read(0, k);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float t = gn[j] * k[j];
          sum[kTU] = fmaf(t, x[j], sum[kTU]);
          if (PRE_LAYER) sum[kT] += t;
          go[j] = fmaf(t, st_next.w, go[j]);
        }
        if (PRE_LAYER) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j >= n) x[j] = 0.f;  // 0 - mean behind the row's end
        }
      }
      if (sums_post) {
        float w[8];
        kept.read(1, k);
        read_gate(i, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          w[j] *= k[j];
          const float v = y[j] * w[j];
          sum[kUV] = fmaf(go[j], v, sum[kUV]);
          if (has_norm) sum[kXV] = fmaf(x[j], v, sum[kXV]);
          if (PRE_LAYER) sum[kV] += j < n ? v : 0.f;
          if (POST == kLayer) {
            sum[kUW] = fmaf(go[j], w[j], sum[kUW]);
            if (has_norm) sum[kXW] = fmaf(x[j], w[j], sum[kXW]);
            if (PRE_LAYER) sum[kW] += j < n ? w[j] : 0.f;
          }
        }
        if (token_shift) {
          kept.read(3, k);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            sum[kUB] = fmaf(go[j], k[j], sum[kUB]);
            if (has_norm) sum[kXB] = fmaf(x[j], k[j], sum[kXB]);
            if (PRE_LAYER) sum[kB] += k[j];
          }
        }
      }
    }
    if (i >= 1) {  // row i - 1's gradients
      const long long t = row_at(i - 1);
      const Slots s = slots(i - 1);
      const float c1 = total[kTU] * inv_d, c2 = PRE_LAYER ? total[kT] * inv_d : 0.f;
      float x[8], y[8], g[8], k[8];
      read_u(i - 1, st, x, y);
      if (f.grad_out.p) {
        s.read(a.field[0], tid, (const R*)nullptr, g);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = 0.f;
      }
      if (has_norm) {
        float gn[8];
        s.read(a.field[1], tid, (const bf16*)nullptr, gn);
        kept.read(0, k);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          acc_tu[j] = fmaf(gn[j], x[j], acc_tu[j]);
          if (PRE_LAYER) acc_t[PRE_LAYER ? j : 0] += gn[j];
          float v = gn[j] * k[j] - x[j] * c1;
          if (PRE_LAYER) v -= c2;
          g[j] = fmaf(st.w, v, g[j]);
        }
      }
      if (f.grad_residual.p) store_row<VEC>(f.grad_residual.p + t * f.grad_residual.stride, g, col, lane_col, a.d, warp_row);
      // from here on s G; with v, w, b for y gain g, gain g and shift:
      // sum of G v = sum of u v - rstd (c2 sum of v + c1 sum of x v), and so on
      auto of = [&](int uv, int xv, int ones) {
        return total[uv] - (has_norm ? st.w * (c1 * total[xv] + (PRE_LAYER ? c2 * total[ones] : 0.f)) : 0.f);
      };
      const float e1 = sums_post ? a.scale * of(kUV, kXV, kV) : 0.f;
      if (f.grad_gate_tokens && warp == 0 && lane == 0)
        f.grad_gate_tokens[t] = e1 + (token_shift ? a.scale * of(kUB, kXB, kB) : 0.f);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] *= a.scale;
      float w[8];
      read_gate(i - 1, w);
      if (f.grad_gate_rows.p) {
        float p[8];
        kept.read(1, k);
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = POST != kNone ? y[j] * k[j] : y[j];
        if (POST == kLayer && f.post_shift) {
          kept.read(3, k);
#pragma unroll
          for (int j = 0; j < 8; ++j) p[j] += k[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] *= g[j];
        store_row<VEC>(f.grad_gate_rows.p + t * f.grad_gate_rows.stride, p, col, lane_col, a.d, warp_row);
      }
      // a gate of columns is put on the sums over rows, and their gradient taken
      // from them, at the end: here without it
      if (!f.gate_columns) {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] *= w[j] * gate_t;
      }
      if (has_y) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          acc_v[j] = fmaf(g[j], y[j], acc_v[j]);
          if (POST == kLayer) acc_g[POST == kLayer ? j : 0] += g[j];
        }
      }
      if (f.gate_columns) {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] *= w[j];
      }
      if (f.grad_y.p) {
        if (POST != kNone) {
          const float m1 = e1 * gate_t * inv_d, m2 = POST == kLayer ? a.scale * gate_t * of(kUW, kXW, kW) * inv_d : 0.f;
          kept.read(1, k);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float v = g[j] * k[j] - y[j] * m1;
            if (POST == kLayer) v -= m2;
            g[j] = st.y * v;
          }
        }
        store_row<VEC>(f.grad_y.p + t * f.grad_y.stride, g, col, lane_col, a.d, warp_row);
      }
    }
    if (VEC) start(i - 1 + a.stages);
    else end(i - 1 + a.stages);
    constexpr int quads = quads_of(PRE_LAYER, POST);
    float4* at = reinterpret_cast<float4*>(smem + a.parts) + (i & 1) * quads * team.warps;
#pragma unroll
    for (int q = 0; q < quads; ++q) {
      float4 v;
      float* p = reinterpret_cast<float*>(&v);
#pragma unroll
      for (int j = 0; j < 4; ++j) p[j] = 4 * q + j < kSums ? warp_sum(sum[4 * q + j < kSums ? 4 * q + j : 0]) : 0.f;
      if (lane == 0) team.write(&at[q * team.warps + warp], v);
    }
    team.arrive();
    team.wait();
#pragma unroll
    for (int q = 0; q < quads; ++q) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = lane; w < team.warps; w += 32) {
        const float4 p = at[q * team.warps + w];
        v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
      }
      const float* p = reinterpret_cast<const float*>(&v);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (4 * q + j < kSums) total[4 * q + j] = warp_sum(p[j]);
    }
  }

  if (!f.sums) return;
  float* to = f.sums + (long long)first * 4 * a.d + col;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j >= n) break;
    to[j] = acc_tu[j];
    if (PRE_LAYER) to[a.d + j] = acc_t[PRE_LAYER ? j : 0];
    to[2 * a.d + j] = acc_v[j];
    if (POST == kLayer) to[3 * a.d + j] = acc_g[POST == kLayer ? j : 0];
  }
}

struct Columns {
  int d, teams, post_layer, pre_layer, params_f32;
  const float* sums;
  const void *post_gain, *post_shift, *gate_columns;
  float one;
  float *pre_gain_grad, *pre_shift_grad, *post_gain_grad, *post_shift_grad, *gate_grad;  // null: not wanted
};

// The teams' sums of 32 columns, added in order by 32 warps' shares.
__global__ void __launch_bounds__(1024) norm_columns(const Columns c) {
  __shared__ float part[4][32][33];
  wait_for_previous_kernel();
  let_next_kernel_start();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float v[4] = {};
  if (col < c.d) {
    const bool wanted[4] = {c.pre_gain_grad != nullptr, c.pre_layer && c.pre_shift_grad,
                            c.post_gain_grad || c.gate_grad, c.post_layer && (c.post_shift_grad || c.gate_grad)};
    for (int t = warp; t < c.teams; t += 32) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (wanted[q]) v[q] += __ldcg(c.sums + ((long long)t * 4 + q) * c.d + col);
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) part[q][warp][lane] = v[q];
  __syncthreads();
  if (warp >= 4) return;
  float s = 0.f;
  for (int w = 0; w < 32; ++w) s += part[warp][w][lane];
  __syncwarp();
  part[warp][0][lane] = s;
  __threadfence_block();
  asm volatile("bar.sync 1, 128;" ::: "memory");
  if (warp != 0 || col >= c.d) return;
  const float pre_gain = part[0][0][lane], pre_shift = part[1][0][lane];
  const float with_u = part[2][0][lane], alone = part[3][0][lane];
  auto param = [&](const void* p, float none) {
    return !p ? none : c.params_f32 ? static_cast<const float*>(p)[col] : __bfloat162float(static_cast<const bf16*>(p)[col]);
  };
  if (c.pre_gain_grad) c.pre_gain_grad[col] = pre_gain;
  if (c.pre_shift_grad) c.pre_shift_grad[col] = pre_shift;
  const float gate = param(c.gate_columns, 1.f);
  if (c.post_gain_grad) c.post_gain_grad[col] = gate * with_u;
  if (c.post_shift_grad) c.post_shift_grad[col] = gate * alone;
  if (c.gate_grad) {
    const float gain = c.post_gain ? param(c.post_gain, 1.f) + c.one : 1.f;
    c.gate_grad[col] = gain * with_u + (c.post_shift ? param(c.post_shift, 0.f) * alone : 0.f);
  }
}

// ------------------------------------------------------------------------- host

template <typename T>
bool rows_aligned(const Rows<T>& r) {  // for 16-byte vectors
  return reinterpret_cast<uintptr_t>(r.p) % 16 == 0 && (size_t)r.stride * sizeof(T) % 16 == 0;
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t type_size(int type) { return type == MOE_TYPE_F32 ? 4 : 2; }

// Blocks of a row, their threads, and how many of them an SM is given.
struct Plan {
  int blocks, threads, per_sm;
};

Plan plan_of(int d, int sm_threads) {
  const int lanes = (d + 7) / 8;
  Plan p;
  p.blocks = 1;
  while (p.blocks * kThreads < lanes) p.blocks *= 2;
  p.threads = ((lanes + p.blocks - 1) / p.blocks + 31) / 32 * 32;
  p.per_sm = std::max(1, std::min(16, sm_threads / p.threads));
  return p;
}

// The shared memory of a block: as many stages as an SM has room for, 2 at least.
int lay_out(Shape* a, const Plan& p, const int (&field_bytes)[5], int kept, int quads, bool vec) {
  a->stage = 0;
  for (int i = 0; i < 5; ++i) a->field[i] = a->stage, a->stage += field_bytes[i] * p.threads;
  const int parts = 2 * quads * p.blocks * p.threads / 32 * 16;
  const int rest = kept * 32 * p.threads + (vec ? 0 : p.threads * 32) + parts;
  a->stages = std::max(2, std::min(kMaxStages, (kRing / p.per_sm - rest) / std::max(1, a->stage)));
  a->vec = a->stages * a->stage;
  a->out = a->vec + kept * 32 * p.threads;
  a->parts = a->vec + rest - parts;
  return a->vec + rest;
}

template <typename, bool>
struct ForwardKernel;
template <typename, bool, bool, int>
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
  e = cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 208 * 1024);
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

// Teams of blocks of a backward pass, at most.
int most_teams(const moe_norm* h) {
  const Plan p = plan_of(h->d, kThreads);
  return kSms * p.per_sm / p.blocks;
}

Shape shape_of(const moe_norm* h, int T) {
  Shape a = {};
  a.T = T;
  a.d = h->d;
  a.pre = h->pre;
  a.post = h->post;
  a.gate = h->gate;
  a.scale = h->scale;
  a.eps = h->eps;
  a.one = h->one;
  a.groups = (h->d + h->group - 1) / h->group;
  a.group_lanes = h->group / 8;
  return a;
}

const char* check_params(const moe_norm* h, const moe_norm_params* p) {
  if (!p) return "null params";
  if (p->type != MOE_TYPE_F32 && p->type != MOE_TYPE_BF16) return "gains and shifts are MOE_TYPE_F32 or MOE_TYPE_BF16";
  const void* all[] = {p->pre_gain, p->pre_shift, p->post_gain, p->post_shift};
  for (const void* q : all)
    if (!aligned(q, type_size(p->type))) return "gains and shifts must be aligned to their type";
  if (h->pre == kNone && p->pre_gain) return "a gain for a norm that the handle does not have";
  if (h->post == kNone && p->post_gain) return "a gain for a norm that the handle does not have";
  if ((h->pre != kLayer && p->pre_shift) || (h->post != kLayer && p->post_shift)) return "only layer norms have a shift";
  if ((h->gate != MOE_GATE_NONE) != (p->gate != nullptr)) return "the gate must be given as the handle has it";
  const size_t gate_size = h->gate == MOE_GATE_CHANNEL ? type_size(p->type) : h->gate == MOE_GATE_TOKEN ? 4 : 2;
  if (!aligned(p->gate, gate_size)) return "the gate must be aligned to its type";
  if (h->gate == MOE_GATE_ELEMENT && p->gate_stride < h->d) return "rows of the gate overlap: the row stride is below d";
  return nullptr;
}

const char* check_rows8(const moe_rows8* r) {
  if (!r) return nullptr;
  if (!r->codes || !r->scales) return "null codes or scales of 8-bit rows";
  if (!aligned(r->scales, 4)) return "scales of 8-bit rows must be 4-byte aligned";
  return nullptr;
}

const char* check_rows(const moe_norm* h, const void* p, int type, long long stride) {
  if (!p) return nullptr;
  if (!aligned(p, type_size(type))) return "tensors must be aligned to their type";
  if (stride < h->d) return "rows overlap: a row stride is below d";
  return nullptr;
}

Rows8 rows8_of(const moe_rows8* r) {
  return r ? Rows8{static_cast<int8_t*>(r->codes), static_cast<bf16*>(r->scales)} : Rows8{nullptr, nullptr};
}

template <typename T>
Rows<T> rows_of(const void* p, long long stride) {
  return Rows<T>{static_cast<T*>(const_cast<void*>(p)), stride};
}

}  // namespace

extern "C" {

moe_norm_t* moe_norm_create(int d, int pre, int post, int gate, float eps, float scale, int unit_offset, int group) {
  const char* bad = nullptr;
  if (d < 1 || d > kMaxD) bad = "need 1 <= d <= 32768";
  else if (pre < kNone || pre > kLayer || post < kNone || post > kLayer) bad = "norms must be MOE_NORM_*";
  else if (gate < MOE_GATE_NONE || gate > MOE_GATE_ELEMENT) bad = "gate must be MOE_GATE_*";
  else if (!(eps >= 0.f) || !isfinite(eps)) bad = "eps must be finite and not negative";
  else if (!isfinite(scale)) bad = "scale must be finite";
  else if (unit_offset != 0 && unit_offset != 1) bad = "unit_offset must be 0 or 1";
  else if (group != 32 && group != 64 && group != 128) bad = "group must be 32, 64 or 128";
  if (bad) {
    moe::set_error(MOE_E_INVAL, bad);
    return nullptr;
  }
  moe_norm_t* h = new (std::nothrow) moe_norm_t();
  if (!h) {
    moe::set_error(MOE_E_NOMEM, "out of host memory");
    return nullptr;
  }
  h->d = d;
  h->pre = pre;
  h->post = post;
  h->gate = gate;
  h->group = group;
  h->eps = eps;
  h->scale = scale;
  h->one = unit_offset ? 1.f : 0.f;
  moe::clear_error();
  return h;
}

void moe_norm_destroy(moe_norm_t* h) {
  if (!h) return;
  if (h->sums) cudaFree(h->sums);
  delete h;
}

long long moe_norm_workspace_bytes(const moe_norm_t* h) {
  return h ? (long long)most_teams(h) * 4 * h->d * (long long)sizeof(float) : -1;
}

int moe_norm_reserve(moe_norm_t* h, void* stream) {
  (void)stream;
  if (!h) return moe::set_error(MOE_E_INVAL, "null handle");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return moe::set_cuda_error(e, "moe_norm_reserve");
  if (h->sums)
    return h->device == dev ? MOE_OK : moe::set_error(MOE_E_STATE, "the handle was reserved on another device");
  if (cudaMalloc(&h->sums, (size_t)moe_norm_workspace_bytes(h)) != cudaSuccess) {
    h->sums = nullptr;
    cudaGetLastError();
    return moe::set_error(MOE_E_NOMEM, "workspace allocation failed");
  }
  h->device = dev;
  moe::clear_error();
  return MOE_OK;
}

int moe_norm_forward(const moe_norm_t* h, int T, int residual_type, const void* residual, long long residual_stride,
                     const void* y, long long y_stride, const moe_norm_params* params, void* out, long long out_stride,
                     void* norm, long long norm_stride, float* stats, const moe_rows8* out8, const moe_rows8* y8,
                     void* stream) {
  if (!h) return moe::set_error(MOE_E_INVAL, "null handle");
  if (T < 0) return moe::set_error(MOE_E_INVAL, "T must not be negative");
  if (residual_type != MOE_TYPE_F32 && residual_type != MOE_TYPE_BF16)
    return moe::set_error(MOE_E_INVAL, "the residual is MOE_TYPE_F32 or MOE_TYPE_BF16");
  const char* bad = check_params(h, params);
  if (!bad) bad = check_rows8(out8);
  if (!bad) bad = check_rows8(y8);
  if (bad) return moe::set_error(MOE_E_INVAL, bad);
  if (T == 0) return MOE_OK;
  if (!residual) bad = "null residual";
  else if (!y != !out) bad = "y and out: both or neither";
  else if (!y && (h->post != kNone || h->gate != MOE_GATE_NONE || y8)) bad = "without y there is nothing to norm, to gate or to keep";
  else if ((h->pre != kNone) != (norm != nullptr)) bad = "norm must be given where the handle has one, and only there";
  else if (!y && !norm && !out8) bad = "nothing to do";
  else if (!aligned(stats, 16)) bad = "stats must be 16-byte aligned";
  if (!bad) bad = check_rows(h, residual, residual_type, residual_stride);
  if (!bad) bad = check_rows(h, y, MOE_TYPE_BF16, y_stride);
  if (!bad) bad = check_rows(h, out, residual_type, out_stride);
  if (!bad) bad = check_rows(h, norm, MOE_TYPE_BF16, norm_stride);
  if (!bad && out == residual && out_stride != residual_stride) bad = "out in residual's place needs its row stride";
  if (bad) return moe::set_error(MOE_E_INVAL, bad);
  auto go = [&](auto r) {
    using R = decltype(r);
    Forward<R> f = {};
    f.a = shape_of(h, T);
    f.residual = rows_of<const R>(residual, residual_stride);
    f.y = rows_of<const bf16>(y, y_stride);
    f.out = rows_of<R>(out, out_stride);
    f.norm = rows_of<bf16>(norm, norm_stride);
    f.pre_gain = params->pre_gain, f.pre_shift = params->pre_shift;
    f.post_gain = params->post_gain, f.post_shift = params->post_shift;
    f.params_f32 = params->type == MOE_TYPE_F32;
    if (h->gate == MOE_GATE_CHANNEL) f.gate_columns = params->gate;
    if (h->gate == MOE_GATE_TOKEN) f.gate_tokens = static_cast<const float*>(params->gate);
    if (h->gate == MOE_GATE_ELEMENT) f.gate_rows = rows_of<const bf16>(params->gate, params->gate_stride);
    f.stats = reinterpret_cast<float4*>(stats);
    f.out8 = rows8_of(out8), f.y8 = rows8_of(y8);
    const bool vec = h->d % 8 == 0 && rows_aligned(f.residual) && rows_aligned(f.y) && rows_aligned(f.out) &&
                     rows_aligned(f.norm) && rows_aligned(f.gate_rows) && aligned(f.out8.codes, 8) && aligned(f.y8.codes, 8);
    const Plan p = plan_of(h->d, vec ? 2 * kThreads : kThreads);
    const int bytes[5] = {(int)sizeof(R) * 8, y ? 16 : 0, f.gate_rows.p ? 16 : 0, 0, 0};
    const int smem = lay_out(&f.a, p, bytes, f.pre_shift ? 4 : f.post_shift ? 3 : 2, 1, vec);
    const int teams = std::min(T, kSms * p.per_sm / p.blocks);
    auto with = [&](auto v) {
      auto* kernel = norm_forward<R, decltype(v)::value>;
      cudaError_t e = allow_smem<ForwardKernel<R, decltype(v)::value>>(kernel);
      return e == cudaSuccess ? launch(kernel, (unsigned)(teams * p.blocks), p.blocks, p.threads, smem,
                                       static_cast<cudaStream_t>(stream), f) : e;
    };
    return vec ? with(std::true_type{}) : with(std::false_type{});
  };
  const cudaError_t e = residual_type == MOE_TYPE_F32 ? go(0.f) : go(bf16());
  return e == cudaSuccess ? MOE_OK : moe::set_cuda_error(e, "norm_forward");
}

int moe_norm_backward(const moe_norm_t* h, int T, int residual_type, const void* grad_out, long long grad_out_stride,
                      const void* grad_norm, long long grad_norm_stride, const moe_norm_params* params,
                      const moe_norm_kept* kept, void* grad_residual, long long grad_residual_stride, void* grad_y,
                      long long grad_y_stride, const moe_norm_grads* grads, void* stream) {
  if (!h) return moe::set_error(MOE_E_INVAL, "null handle");
  if (T < 0) return moe::set_error(MOE_E_INVAL, "T must not be negative");
  if (residual_type != MOE_TYPE_F32 && residual_type != MOE_TYPE_BF16)
    return moe::set_error(MOE_E_INVAL, "the residual is MOE_TYPE_F32 or MOE_TYPE_BF16");
  if (!kept || !grads) return moe::set_error(MOE_E_INVAL, "null kept or grads");
  const char* bad = check_params(h, params);
  if (!bad) bad = check_rows8(kept->out8);
  if (!bad) bad = check_rows8(kept->y8);
  if (bad) return moe::set_error(MOE_E_INVAL, bad);
  const moe_norm_grads& g = *grads;
  // a gradient is of something that is there
  if ((g.pre_gain && !params->pre_gain) || (g.pre_shift && !params->pre_shift) || (g.post_gain && !params->post_gain) ||
      (g.post_shift && !params->post_shift) || (g.gate && !params->gate))
    return moe::set_error(MOE_E_INVAL, "a gradient of something that was not given");
  float* const columns[] = {g.pre_gain, g.pre_shift, g.post_gain, g.post_shift,
                            h->gate == MOE_GATE_CHANNEL ? static_cast<float*>(g.gate) : nullptr};
  bool any = false;
  for (const float* c : columns) {
    if (!aligned(c, 4)) return moe::set_error(MOE_E_INVAL, "gradients must be aligned to their type");
    any = any || c;
  }
  if (any && !h->sums) return moe::set_error(MOE_E_STATE, "moe_norm_reserve was not called");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    for (float* c : columns)
      if (c)
        if (cudaError_t e = cudaMemsetAsync(c, 0, sizeof(float) * h->d, s)) return moe::set_cuda_error(e, "cudaMemsetAsync");
    return MOE_OK;
  }
  const bool has_norm = grad_norm != nullptr;
  const bool has_y = kept->y || kept->y8;
  if (!grad_out && !grad_norm) bad = "no gradient to start from";
  else if (has_norm && h->pre == kNone) bad = "the gradient of a norm that the handle does not have";
  else if (!has_norm && (g.pre_gain || g.pre_shift)) bad = "gradients of the pre norm need that of its output";
  else if (kept->out && kept->out8) bad = "out is kept in one form";
  else if (kept->y && kept->y8) bad = "y is kept in one form";
  else if (has_norm && !kept->out && !kept->out8) bad = "the gradient of the norm needs what was kept of out";
  else if (!has_y && ((h->post != kNone && grad_y) || g.post_gain || g.post_shift || g.gate)) bad = "these gradients need what was kept of y";
  else if ((has_norm || h->post != kNone) && !kept->stats) bad = "the gradients of norms need stats";
  else if (!grad_residual && !grad_y && !any && !g.gate) bad = "no gradient is wanted";
  else if (!aligned(kept->stats, 16)) bad = "stats must be 16-byte aligned";
  else if (h->gate == MOE_GATE_TOKEN && !aligned(g.gate, 4)) bad = "gradients must be aligned to their type";
  if (!bad) bad = check_rows(h, grad_out, residual_type, grad_out_stride);
  if (!bad) bad = check_rows(h, grad_norm, MOE_TYPE_BF16, grad_norm_stride);
  if (!bad) bad = check_rows(h, kept->out, residual_type, kept->out_stride);
  if (!bad) bad = check_rows(h, kept->y, MOE_TYPE_BF16, kept->y_stride);
  if (!bad) bad = check_rows(h, grad_residual, residual_type, grad_residual_stride);
  if (!bad) bad = check_rows(h, grad_y, MOE_TYPE_BF16, grad_y_stride);
  if (!bad && h->gate == MOE_GATE_ELEMENT) bad = check_rows(h, g.gate, MOE_TYPE_BF16, g.gate_stride);
  if (!bad && grad_out && grad_out == grad_residual && grad_out_stride != grad_residual_stride)
    bad = "grad_residual in grad_out's place needs its row stride";
  if (bad) return moe::set_error(MOE_E_INVAL, bad);
  const Plan p = plan_of(h->d, kThreads);
  const int teams = std::min(T, kSms * p.per_sm / p.blocks);
  auto go = [&](auto r) {
    using R = decltype(r);
    Backward<R> f = {};
    f.a = shape_of(h, T);
    f.grad_out = rows_of<const R>(grad_out, grad_out_stride);
    f.grad_norm = rows_of<const bf16>(grad_norm, grad_norm_stride);
    if (has_norm) {
      f.kept_out = rows_of<const R>(kept->out, kept->out_stride);
      f.out8 = rows8_of(kept->out8);
    }
    f.y = rows_of<const bf16>(kept->y, kept->y_stride);
    f.y8 = rows8_of(kept->y8);
    f.stats = reinterpret_cast<const float4*>(kept->stats);
    f.pre_gain = params->pre_gain, f.post_gain = params->post_gain, f.post_shift = params->post_shift;
    f.params_f32 = params->type == MOE_TYPE_F32;
    if (h->gate == MOE_GATE_CHANNEL) f.gate_columns = params->gate;
    if (h->gate == MOE_GATE_TOKEN) {
      f.gate_tokens = static_cast<const float*>(params->gate);
      f.grad_gate_tokens = static_cast<float*>(g.gate);
    }
    if (h->gate == MOE_GATE_ELEMENT) {
      f.gate_rows = rows_of<const bf16>(params->gate, params->gate_stride);
      f.grad_gate_rows = rows_of<bf16>(g.gate, g.gate_stride);
    }
    f.grad_residual = rows_of<R>(grad_residual, grad_residual_stride);
    f.grad_y = rows_of<bf16>(grad_y, grad_y_stride);
    f.sums = any ? h->sums : nullptr;
    const bool vec = h->d % 8 == 0 && rows_aligned(f.grad_out) && rows_aligned(f.grad_norm) && rows_aligned(f.kept_out) &&
                     rows_aligned(f.y) && rows_aligned(f.gate_rows) && rows_aligned(f.grad_residual) &&
                     rows_aligned(f.grad_y) && rows_aligned(f.grad_gate_rows) && aligned(f.out8.codes, 8) &&
                     aligned(f.y8.codes, 8);
    const int size = (int)sizeof(R) * 8;
    const int bytes[5] = {grad_out ? size : 0, has_norm ? 16 : 0, !has_norm ? 0 : f.out8.codes ? 16 : size,
                          has_y ? 16 : 0, f.gate_rows.p ? 16 : 0};
    const int smem = lay_out(&f.a, p, bytes, f.post_shift ? 4 : 3, quads_of(h->pre == kLayer, h->post), vec);
    auto with = [&](auto v, auto layer, auto post) {
      constexpr bool VEC = decltype(v)::value, LAYER = decltype(layer)::value;
      constexpr int POST = decltype(post)::value;
      auto* kernel = norm_backward<R, VEC, LAYER, POST>;
      cudaError_t e = allow_smem<BackwardKernel<R, VEC, LAYER, POST>>(kernel);
      return e == cudaSuccess ? launch(kernel, (unsigned)(teams * p.blocks), p.blocks, p.threads, smem, s, f) : e;
    };
    auto by_post = [&](auto v, auto layer) {
      return h->post == kNone  ? with(v, layer, std::integral_constant<int, kNone>{})
             : h->post == kRms ? with(v, layer, std::integral_constant<int, kRms>{})
                               : with(v, layer, std::integral_constant<int, kLayer>{});
    };
    auto by_pre = [&](auto v) {
      return h->pre == kLayer ? by_post(v, std::true_type{}) : by_post(v, std::false_type{});
    };
    return vec ? by_pre(std::true_type{}) : by_pre(std::false_type{});
  };
  cudaError_t e = residual_type == MOE_TYPE_F32 ? go(0.f) : go(bf16());
  if (e == cudaSuccess && any) {
    Columns c = {};
    c.d = h->d, c.teams = teams;
    c.post_layer = h->post == kLayer, c.pre_layer = h->pre == kLayer;
    c.params_f32 = params->type == MOE_TYPE_F32;
    c.sums = h->sums;
    c.post_gain = params->post_gain, c.post_shift = params->post_shift;
    if (h->gate == MOE_GATE_CHANNEL) c.gate_columns = params->gate;
    c.one = h->one;
    c.pre_gain_grad = columns[0], c.pre_shift_grad = columns[1], c.post_gain_grad = columns[2];
    c.post_shift_grad = columns[3], c.gate_grad = columns[4];
    e = launch(norm_columns, (unsigned)((h->d + 31) / 32), 1, 1024, 0, s, c);
  }
  return e == cudaSuccess ? MOE_OK : moe::set_cuda_error(e, "norm_backward");
}

}  // extern "C"
