// Experts on 4-bit weights with group scales: the conversion of bf16 weights,
// the way back, and the experts' SwiGLU product for decode batches.
//
// A weight matrix [rows, cols] is held as codes (two 4-bit numbers to a byte,
// the even column in the low half), one bf16 scale for each group of 32, 64
// or 128 consecutive columns of a row and, optionally, one zero point (0..15,
// a byte) for each group: value = (code - zero) * scale, zero 8 where there
// are no zero points.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <new>

#include "error.h"
#include "moe.h"

namespace {

constexpr int kMaxE = 256;
constexpr int kMaxK = 16;
constexpr int kMaxD = 32768;
constexpr int kMaxT = 1024;

struct Weight {
  const uint8_t* codes;          // [E + S, rows, cols / 2]
  const __nv_bfloat16* scales;   // [E + S, rows, cols / group]
  const uint8_t* zeros;          // the same, or null
};

// ------------------------------------------------------------------ conversion

// One warp lane holds 8 consecutive weights; the G / 8 lanes of a group share
// its range by shuffles.
template <int G, bool Z>
__global__ void __launch_bounds__(256)
    w4_quantize(long long n8, const uint4* __restrict__ w, uint32_t* __restrict__ codes,
                __nv_bfloat16* __restrict__ scales, uint8_t* __restrict__ zeros) {
  constexpr int kLanes = G / 8;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n8; i += (long long)gridDim.x * 256) {
    // n8 is a multiple of kLanes, so the lanes of a group are here together
    const unsigned mask = ((1u << kLanes) - 1u) << (threadIdx.x & 31 & ~(kLanes - 1));
    union {
      uint4 q;
      __nv_bfloat16 b[8];
    } u;
    u.q = w[i];
    float v[8], lo = 0.f, hi = 0.f;
    bool finite = true;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = __bfloat162float(u.b[j]);
      finite &= fabsf(v[j]) < INFINITY;
      lo = fminf(lo, v[j]);
      hi = fmaxf(hi, v[j]);
    }
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(mask, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(mask, hi, o));
      finite &= __shfl_xor_sync(mask, (int)finite, o) != 0;
    }
    // (hi - lo) / 15, halved first so that no range overflows
    const float range = Z ? (hi * 0.5f - lo * 0.5f) / 7.5f : fmaxf(hi, -lo) / 7.f;
    const __nv_bfloat16 sb = __float2bfloat16(finite ? range : __uint_as_float(0x7fffffffu));
    const float s = __bfloat162float(sb);
    const float div = s == 0.f || !finite ? 1.f : s;
    const float z = !finite ? 8.f : Z ? fminf(fmaxf(rintf(-lo / div), 0.f), 15.f) : 8.f;
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float q = fminf(fmaxf(rintf((finite ? v[j] : 0.f) / div) + z, 0.f), 15.f);
      word |= (uint32_t)q << (4 * j);
    }
    codes[i] = word;
    if (i % kLanes == 0) {
      scales[i / kLanes] = sb;
      if (Z) zeros[i / kLanes] = (uint8_t)z;
    }
  }
}

template <int G, bool Z>
__global__ void __launch_bounds__(256)
    w4_dequantize(long long n8, const uint32_t* __restrict__ codes,
                  const __nv_bfloat16* __restrict__ scales, const uint8_t* __restrict__ zeros,
                  uint4* __restrict__ w) {
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n8; i += (long long)gridDim.x * 256) {
    const uint32_t word = codes[i];
    const float s = __bfloat162float(scales[i / (G / 8)]);
    const float z = Z ? (float)zeros[i / (G / 8)] : 8.f;
    union {
      uint4 q;
      __nv_bfloat16 b[8];
    } u;
#pragma unroll
    for (int j = 0; j < 8; ++j) u.b[j] = __float2bfloat16(((float)(word >> (4 * j) & 15u) - z) * s);
    w[i] = u.q;
  }
}

// --------------------------------------------------------------------- experts

struct Experts {
  int T, d, f, E, k, S, group;
  Weight gate, up, down;
  const __nv_bfloat16* x;   // [T, d]
  const int* idx;           // [T, k]
  const float* w;           // [T, k]
  __nv_bfloat16* h;         // [T k + T S, f]
  __nv_bfloat16* out;       // [T, d]
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Dot product of row r of expert e with v [cols], by one warp.
__device__ float w4_dot(const Weight& m, long long r, int cols, int group, const __nv_bfloat16* v) {
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(m.codes + r * (cols / 2));
  const long long g0 = r * (cols / group);
  float sum = 0.f;
  for (int i = threadIdx.x & 31; i < cols / 8; i += 32) {
    const uint32_t word = codes[i];
    const int g = i * 8 / group;
    const float s = __bfloat162float(m.scales[g0 + g]), z = m.zeros ? (float)m.zeros[g0 + g] : 8.f;
    float part = 0.f;
    for (int j = 0; j < 8; ++j)
      part += ((float)(word >> (4 * j) & 15u) - z) * __bfloat162float(v[i * 8 + j]);
    sum += s * part;
  }
  return warp_sum(sum);
}

// The expert of row p of h: slot p of idx, or the shared expert behind them.
__device__ __forceinline__ int expert_of(const Experts& a, int p) {
  return p < a.T * a.k ? a.idx[p] : a.E;
}

__global__ void w4_gate_up(Experts a) {
  const int n = blockIdx.x * 8 + (threadIdx.x >> 5), p = blockIdx.y;
  const int e = expert_of(a, p);
  if (e < 0 || e > a.E || (e == a.E && p < a.T * a.k)) return;
  const __nv_bfloat16* x = a.x + (size_t)(p < a.T * a.k ? p / a.k : p - a.T * a.k) * a.d;
  const long long r = (long long)e * a.f + n;
  const float z = w4_dot(a.gate, r, a.d, a.group, x), u = w4_dot(a.up, r, a.d, a.group, x);
  if ((threadIdx.x & 31) == 0) a.h[(size_t)p * a.f + n] = __float2bfloat16(z / (1.f + expf(-z)) * u);
}

__global__ void w4_down(Experts a) {
  const int n = blockIdx.x * 8 + (threadIdx.x >> 5), t = blockIdx.y;
  float sum = 0.f;
  for (int j = 0; j < a.k + a.S; ++j) {
    const int p = j < a.k ? t * a.k + j : a.T * a.k + t;
    const int e = j < a.k ? a.idx[p] : a.E;
    if (e < 0 || (j < a.k && e >= a.E)) continue;
    const float y = w4_dot(a.down, (long long)e * a.d + n, a.f, a.group, a.h + (size_t)p * a.f);
    sum += j < a.k ? a.w[p] * y : y;
  }
  if ((threadIdx.x & 31) == 0) a.out[(size_t)t * a.d + n] = __float2bfloat16(sum);
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int check_matrix(long long rows, int cols, int group, const void* codes, const void* scales, const void* w) {
  if (group != 32 && group != 64 && group != 128) return moe::set_error(MOE_E_INVAL, "group must be 32, 64 or 128");
  if (rows < 0 || cols < 0 || cols % group != 0)
    return moe::set_error(MOE_E_INVAL, "cols must be a multiple of the group, rows and cols not negative");
  if (rows == 0 || cols == 0) return MOE_OK;
  if (!codes || !scales || !w) return moe::set_error(MOE_E_INVAL, "null tensor pointer");
  if (!aligned(codes, 16) || !aligned(w, 16) || !aligned(scales, 2))
    return moe::set_error(MOE_E_INVAL, "weights and codes must be 16-byte aligned, scales 2-byte");
  return MOE_OK;
}

template <typename... A>
cudaError_t launch(void (*kernel)(A...), dim3 grid, int threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

dim3 convert_grid(long long n8) { return dim3((unsigned)std::min<long long>((n8 + 255) / 256, 152 * 8)); }

}  // namespace

struct moe_w4 {
  int d, f, E, k, S, group;
  int T_max = 0;
  Weight gate{}, up{}, down{};
  char* ws = nullptr;
};

namespace {

long long workspace(const moe_w4* h, int T) { return (long long)T * (h->k + h->S) * h->f * 2; }

}  // namespace

extern "C" {

int moe_w4_quantize(long long rows, int cols, int group, const void* w, void* codes, void* scales,
                    void* zeros, void* stream) {
  if (int rc = check_matrix(rows, cols, group, codes, scales, w)) return rc;
  const long long n8 = rows * (cols / 8);
  if (n8 == 0) return MOE_OK;
  auto kernel = zeros ? (group == 32 ? w4_quantize<32, true> : group == 64 ? w4_quantize<64, true> : w4_quantize<128, true>)
                      : (group == 32 ? w4_quantize<32, false> : group == 64 ? w4_quantize<64, false> : w4_quantize<128, false>);
  cudaError_t e = launch(kernel, convert_grid(n8), 256, static_cast<cudaStream_t>(stream), n8,
                         static_cast<const uint4*>(w), static_cast<uint32_t*>(codes),
                         static_cast<__nv_bfloat16*>(scales), static_cast<uint8_t*>(zeros));
  return e == cudaSuccess ? MOE_OK : moe::set_cuda_error(e, "w4_quantize");
}

int moe_w4_dequantize(long long rows, int cols, int group, const void* codes, const void* scales,
                      const void* zeros, void* w, void* stream) {
  if (int rc = check_matrix(rows, cols, group, codes, scales, w)) return rc;
  const long long n8 = rows * (cols / 8);
  if (n8 == 0) return MOE_OK;
  auto kernel = zeros ? (group == 32 ? w4_dequantize<32, true> : group == 64 ? w4_dequantize<64, true> : w4_dequantize<128, true>)
                      : (group == 32 ? w4_dequantize<32, false> : group == 64 ? w4_dequantize<64, false> : w4_dequantize<128, false>);
  cudaError_t e = launch(kernel, convert_grid(n8), 256, static_cast<cudaStream_t>(stream), n8,
                         static_cast<const uint32_t*>(codes), static_cast<const __nv_bfloat16*>(scales),
                         static_cast<const uint8_t*>(zeros), static_cast<uint4*>(w));
  return e == cudaSuccess ? MOE_OK : moe::set_cuda_error(e, "w4_dequantize");
}

moe_w4_t* moe_w4_create(int d, int f, int E, int k, int shared_experts, int group) {
  const char* bad = nullptr;
  if (d <= 0 || d % 128 != 0 || d > kMaxD) bad = "d must be a positive multiple of 128, at most 32768";
  else if (f <= 0 || f % 128 != 0 || f > kMaxD) bad = "f must be a positive multiple of 128, at most 32768";
  else if (E < 1 || E > kMaxE || k < 1 || k > E || k > kMaxK) bad = "need 1 <= k <= E <= 256 and k <= 16";
  else if (shared_experts < 0 || shared_experts > 1) bad = "shared_experts must be 0 or 1";
  else if (group != 32 && group != 64 && group != 128) bad = "group must be 32, 64 or 128";
  if (bad) {
    moe::set_error(MOE_E_INVAL, bad);
    return nullptr;
  }
  moe_w4_t* h = new (std::nothrow) moe_w4_t();
  if (!h) {
    moe::set_error(MOE_E_NOMEM, "out of host memory");
    return nullptr;
  }
  h->d = d;
  h->f = f;
  h->E = E;
  h->k = k;
  h->S = shared_experts;
  h->group = group;
  moe::clear_error();
  return h;
}

long long moe_w4_workspace_bytes(const moe_w4_t* h, int T_max) {
  return !h || T_max < 0 || T_max > kMaxT ? -1 : workspace(h, T_max);
}

int moe_w4_reserve(moe_w4_t* h, int T_max, void* stream) {
  if (!h) return moe::set_error(MOE_E_INVAL, "null handle");
  if (T_max < 1 || T_max > kMaxT) return moe::set_error(MOE_E_INVAL, "T_max out of range (1..1024)");
  int dev = 0, major = 0, minor = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (e == cudaSuccess && (major != 10 || minor != 3))
    return moe::set_error(MOE_E_INVAL, "this library is built for sm_103a (GB300) only");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (e == cudaSuccess && h->ws) {
    e = cudaStreamSynchronize(s);
    if (e == cudaSuccess) e = cudaFree(h->ws);
    h->ws = nullptr;
    h->T_max = 0;
  }
  if (e != cudaSuccess) return moe::set_cuda_error(e, "moe_w4_reserve");
  const size_t bytes = (size_t)workspace(h, T_max);
  if (cudaMalloc(&h->ws, bytes) != cudaSuccess) {
    h->ws = nullptr;
    cudaGetLastError();
    return moe::set_error(MOE_E_NOMEM, "workspace allocation failed");
  }
  e = cudaMemsetAsync(h->ws, 0, bytes, s);
  if (e != cudaSuccess) return moe::set_cuda_error(e, "cudaMemsetAsync");
  h->T_max = T_max;
  moe::clear_error();
  return MOE_OK;
}

int moe_w4_set_weights(moe_w4_t* h, const moe_w4_weight* gate, const moe_w4_weight* up,
                       const moe_w4_weight* down) {
  if (!h) return moe::set_error(MOE_E_INVAL, "null handle");
  const moe_w4_weight* m[3] = {gate, up, down};
  for (auto* p : m) {
    if (!p || !p->codes || !p->scales) return moe::set_error(MOE_E_INVAL, "null weights");
    if (!aligned(p->codes, 16) || !aligned(p->scales, 16) || !aligned(p->zeros, 16))
      return moe::set_error(MOE_E_INVAL, "codes, scales and zeros must be 16-byte aligned");
    if (!p->zeros != !gate->zeros) return moe::set_error(MOE_E_INVAL, "zero points: for all three matrices or for none");
  }
  auto take = [](const moe_w4_weight* p) {
    return Weight{static_cast<const uint8_t*>(p->codes), static_cast<const __nv_bfloat16*>(p->scales),
                  static_cast<const uint8_t*>(p->zeros)};
  };
  h->gate = take(gate);
  h->up = take(up);
  h->down = take(down);
  return MOE_OK;
}

int moe_w4_forward(moe_w4_t* h, int T, const void* x, const int32_t* idx, const float* w, void* out,
                   void* stream) {
  if (!h) return moe::set_error(MOE_E_INVAL, "null handle");
  if (!h->ws) return moe::set_error(MOE_E_STATE, "moe_w4_reserve was not called");
  if (!h->gate.codes) return moe::set_error(MOE_E_STATE, "moe_w4_set_weights was not called");
  if (T < 0 || T > h->T_max) return moe::set_error(MOE_E_INVAL, "T out of range (0..T_max)");
  if (T == 0) return MOE_OK;
  if (!x || !idx || !w || !out) return moe::set_error(MOE_E_INVAL, "null tensor pointer");
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(idx, 4) || !aligned(w, 4))
    return moe::set_error(MOE_E_INVAL, "x and out must be 16-byte aligned, idx and w 4-byte");
  Experts a{T, h->d, h->f, h->E, h->k, h->S, h->group, h->gate, h->up, h->down,
            static_cast<const __nv_bfloat16*>(x), idx, w, reinterpret_cast<__nv_bfloat16*>(h->ws),
            static_cast<__nv_bfloat16*>(out)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch(w4_gate_up, dim3(h->f / 8, T * (h->k + h->S)), 256, s, a);
  if (e == cudaSuccess) e = launch(w4_down, dim3(h->d / 8, T), 256, s, a);
  return e == cudaSuccess ? MOE_OK : moe::set_cuda_error(e, "w4_experts");
}

void moe_w4_destroy(moe_w4_t* h) {
  if (!h) return;
  if (h->ws) cudaFree(h->ws);
  delete h;
}

}  // extern "C"
