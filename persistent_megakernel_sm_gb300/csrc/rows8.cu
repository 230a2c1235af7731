// 8-bit rows: activations kept for the backward pass, and fetched back.
//
//   scale = bf16(max |v| / 127) of a group of 32, 64 or 128 consecutive columns
//           (the last one of a row may be short)
//   code  = clamp(round(v / scale), -127, 127), half to even
//
// Both directions are bound by HBM: 1 byte and 2 / group a value on one side, 2
// or 4 on the other, each once.  24576 x 1408 bf16 in groups of 128 there and back take
// 34 us, 6.1 TB/s of the 6.8 that a copy has; 1021 x 1411 fp32 in groups of 32, whose rows
// are not aligned, 8.8 (two launches; their bytes 2.2).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "error.h"
#include "moe.h"
#include "rows8.cuh"

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kUnroll = 4;
constexpr int kMaxCols = 1 << 30;  // a column and a warp's step stay in 32 bits

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_float(float v, float* o) { *o = v; }
__device__ __forceinline__ void from_float(float v, __nv_bfloat16* o) { *o = __float2bfloat16_rn(v); }

// 8 consecutive values, 16-byte aligned.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 q = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 q = __ldcs(reinterpret_cast<const float4*>(p) + i);
    v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  union {
    __nv_bfloat162 b[4];
    uint4 q;
  } u;
#pragma unroll
  for (int i = 0; i < 4; ++i) u.b[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  __stcs(reinterpret_cast<uint4*>(p), u.q);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    __stcs(reinterpret_cast<float4*>(p) + i, make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
}

// Rows of whole groups, aligned: the tensor is one run of groups, a lane takes 8
// consecutive values (kUnroll such, all loads first), and the G / 8 lanes of a
// group find its range by shuffles.
template <typename T, int G>
__global__ void __launch_bounds__(256)
    rows8_quantize_flat(long long n8, const T* __restrict__ v, uint2* __restrict__ codes, __nv_bfloat16* __restrict__ scales) {
  constexpr int kLanes = G / 8;
  const unsigned mask = ((1u << kLanes) - 1u) << (threadIdx.x & 31 & ~(kLanes - 1));
  const long long i0 = (long long)blockIdx.x * (256 * kUnroll) + threadIdx.x;
  float x[kUnroll][8];
#pragma unroll
  for (int n = 0; n < kUnroll; ++n)
    if (i0 + n * 256 < n8) load8(v + (i0 + n * 256) * 8, x[n]);
#pragma unroll
  for (int n = 0; n < kUnroll; ++n) {
    const long long i = i0 + n * 256;
    if (i >= n8) break;  // n8 is a multiple of kLanes: the lanes of a group go together
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) most = max(most, moe::abs_bits(x[n][j]));
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) most = max(most, __shfl_xor_sync(mask, most, o));
    const __nv_bfloat16 s = moe::rows8_scale<T>(most);
    const float2 two[4] = {make_float2(x[n][0], x[n][1]), make_float2(x[n][2], x[n][3]), make_float2(x[n][4], x[n][5]),
                           make_float2(x[n][6], x[n][7])};
    __stcs(codes + i, moe::rows8_codes<T>(two, s));
    if (i % kLanes == 0) scales[i / kLanes] = s;
  }
}

template <typename T, int G>
__global__ void __launch_bounds__(256)
    rows8_dequantize_flat(long long n8, const uint2* __restrict__ codes, const __nv_bfloat16* __restrict__ scales, T* __restrict__ v) {
  const long long i0 = (long long)blockIdx.x * (256 * kUnroll) + threadIdx.x;
  uint2 word[kUnroll];
  float s[kUnroll];
#pragma unroll
  for (int n = 0; n < kUnroll; ++n) {
    const long long i = i0 + n * 256;
    if (i >= n8) break;
    word[n] = __ldcs(codes + i);
    s[n] = __bfloat162float(scales[i / (G / 8)]);
  }
#pragma unroll
  for (int n = 0; n < kUnroll; ++n) {
    const long long i = i0 + n * 256;
    if (i >= n8) break;
    float2 lo[2], hi[2];
    moe::rows8_floats(word[n].x, lo);
    moe::rows8_floats(word[n].y, hi);
    const float x[8] = {lo[0].x * s[n], lo[0].y * s[n], lo[1].x * s[n], lo[1].y * s[n],
                        hi[0].x * s[n], hi[0].y * s[n], hi[1].x * s[n], hi[1].y * s[n]};
    store8(v + i * 8, x);
  }
}

// Any other rows: a warp takes 256 columns of a row, a lane every 32nd of them, so
// loads and stores run along the row whatever its alignment; 32 columns are one
// step of the warp, a group 1, 2 or 4 of them.
template <typename T, int G>
__global__ void __launch_bounds__(256)
    rows8_quantize_any(long long units, int cols, int segments, const T* __restrict__ v, int8_t* __restrict__ codes,
                       __nv_bfloat16* __restrict__ scales) {
  const long long unit = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (unit >= units) return;
  const long long row = unit / segments;
  const int lane = threadIdx.x & 31, c0 = (int)(unit % segments) * 256;
  const int groups = (cols + G - 1) / G;
  const T* from = v + row * cols;
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = c0 + i * 32 + lane < cols ? to_float(from[c0 + i * 32 + lane]) : 0.f;
  constexpr int kSteps = G / 32;
  uint32_t most[8 / kSteps];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t& m = most[i / kSteps];
    m = i % kSteps ? max(m, moe::abs_bits(x[i])) : moe::abs_bits(x[i]);
  }
#pragma unroll
  for (int g = 0; g < 8 / kSteps; ++g) most[g] = __reduce_max_sync(kAll, most[g]);
#pragma unroll
  for (int g = 0; g < 8 / kSteps; ++g) {
    const int c = c0 + g * G;
    if (c >= cols) break;
    const __nv_bfloat16 s = moe::rows8_scale<T>(most[g]);
    float in[8] = {};
#pragma unroll
    for (int i = 0; i < kSteps; ++i) in[i] = x[g * kSteps + i];
    const float2 two[4] = {make_float2(in[0], in[1]), make_float2(in[2], in[3]), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    const uint32_t word = moe::rows8_codes<T>(two, s).x;
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
      if (c + i * 32 + lane < cols) codes[row * cols + c + i * 32 + lane] = (int8_t)(word >> (8 * i));
    if (lane == 0) scales[row * groups + c / G] = s;
  }
}

template <typename T>
__global__ void __launch_bounds__(256)
    rows8_dequantize_any(long long units, int cols, int segments, int group_log, const int8_t* __restrict__ codes,
                         const __nv_bfloat16* __restrict__ scales, T* __restrict__ v) {
  const long long unit = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (unit >= units) return;
  const long long row = unit / segments;
  const int lane = threadIdx.x & 31, c0 = (int)(unit % segments) * 256;
  const int groups = ((cols - 1) >> group_log) + 1;
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = c0 + i * 32 + lane;
    x[i] = c < cols ? (float)codes[row * cols + c] * __bfloat162float(scales[row * groups + (c >> group_log)]) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = c0 + i * 32 + lane;
    if (c < cols) from_float(x[i], v + row * cols + c);
  }
}

template <typename... A, typename... B>
cudaError_t launch(void (*kernel)(A...), unsigned grid, cudaStream_t s, B... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<A>(args)...);
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int check_rows(long long rows, int cols, int type, int group, const void* v, const void* codes, const void* scales) {
  if (group != 32 && group != 64 && group != 128) return moe::set_error(MOE_E_INVAL, "group must be 32, 64 or 128");
  if (type != MOE_TYPE_F32 && type != MOE_TYPE_BF16)
    return moe::set_error(MOE_E_INVAL, "values are MOE_TYPE_F32 or MOE_TYPE_BF16");
  if (rows < 0 || cols < 0 || cols > kMaxCols) return moe::set_error(MOE_E_INVAL, "rows must not be negative, cols in 0..2^30");
  if (rows == 0 || cols == 0) return MOE_OK;
  if (rows > (1ll << 38) / cols) return moe::set_error(MOE_E_INVAL, "more than 2^38 values");
  if (!v || !codes || !scales) return moe::set_error(MOE_E_INVAL, "null tensor pointer");
  if (!aligned(v, type == MOE_TYPE_F32 ? 4 : 2) || !aligned(scales, 2))
    return moe::set_error(MOE_E_INVAL, "values and scales must be aligned to their types");
  return MOE_OK;
}

// The blocks of a kernel of `per` units a block; 0: more than a grid holds.
unsigned blocks_of(long long units, long long per) {
  const long long n = (units + per - 1) / per;
  return n > 0x7fffffffll ? 0 : (unsigned)n;
}

template <typename T>
int quantize(long long rows, int cols, int group, const void* v, void* codes, void* scales, cudaStream_t s) {
  cudaError_t e;
  const T* in = static_cast<const T*>(v);
  __nv_bfloat16* sc = static_cast<__nv_bfloat16*>(scales);
  if (cols % group == 0 && aligned(v, 16) && aligned(codes, 8)) {
    const long long n8 = rows * (cols / 8);
    const unsigned grid = blocks_of(n8, 256 * kUnroll);
    if (!grid) return moe::set_error(MOE_E_INVAL, "too many rows");
    auto kernel = group == 32 ? rows8_quantize_flat<T, 32> : group == 64 ? rows8_quantize_flat<T, 64> : rows8_quantize_flat<T, 128>;
    e = launch(kernel, grid, s, n8, in, static_cast<uint2*>(codes), sc);
  } else {
    const int segments = (cols + 255) / 256;
    const unsigned grid = blocks_of(rows * segments, 8);
    if (!grid) return moe::set_error(MOE_E_INVAL, "too many rows");
    auto kernel = group == 32 ? rows8_quantize_any<T, 32> : group == 64 ? rows8_quantize_any<T, 64> : rows8_quantize_any<T, 128>;
    e = launch(kernel, grid, s, rows * segments, cols, segments, in, static_cast<int8_t*>(codes), sc);
  }
  return e == cudaSuccess ? MOE_OK : moe::set_cuda_error(e, "rows8_quantize");
}

template <typename T>
int dequantize(long long rows, int cols, int group, const void* codes, const void* scales, void* v, cudaStream_t s) {
  cudaError_t e;
  T* out = static_cast<T*>(v);
  const __nv_bfloat16* sc = static_cast<const __nv_bfloat16*>(scales);
  if (cols % group == 0 && aligned(v, 16) && aligned(codes, 8)) {
    const long long n8 = rows * (cols / 8);
    const unsigned grid = blocks_of(n8, 256 * kUnroll);
    if (!grid) return moe::set_error(MOE_E_INVAL, "too many rows");
    auto kernel = group == 32 ? rows8_dequantize_flat<T, 32> : group == 64 ? rows8_dequantize_flat<T, 64> : rows8_dequantize_flat<T, 128>;
    e = launch(kernel, grid, s, n8, static_cast<const uint2*>(codes), sc, out);
  } else {
    const int segments = (cols + 255) / 256;
    const unsigned grid = blocks_of(rows * segments, 8);
    if (!grid) return moe::set_error(MOE_E_INVAL, "too many rows");
    e = launch(rows8_dequantize_any<T>, grid, s, rows * segments, cols, segments, group == 32 ? 5 : group == 64 ? 6 : 7,
                                                 static_cast<const int8_t*>(codes), sc, out);
  }
  return e == cudaSuccess ? MOE_OK : moe::set_cuda_error(e, "rows8_dequantize");
}

}  // namespace

extern "C" {

int moe_rows8_quantize(long long rows, int cols, int type, int group, const void* v, void* codes, void* scales,
                       void* stream) {
  if (int rc = check_rows(rows, cols, type, group, v, codes, scales)) return rc;
  if (rows == 0 || cols == 0) return MOE_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return type == MOE_TYPE_F32 ? quantize<float>(rows, cols, group, v, codes, scales, s)
                              : quantize<__nv_bfloat16>(rows, cols, group, v, codes, scales, s);
}

int moe_rows8_dequantize(long long rows, int cols, int type, int group, const void* codes, const void* scales, void* v,
                         void* stream) {
  if (int rc = check_rows(rows, cols, type, group, v, codes, scales)) return rc;
  if (rows == 0 || cols == 0) return MOE_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return type == MOE_TYPE_F32 ? dequantize<float>(rows, cols, group, codes, scales, v, s)
                              : dequantize<__nv_bfloat16>(rows, cols, group, codes, scales, v, s);
}

}  // extern "C"
