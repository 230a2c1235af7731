// Experts on 4-bit weights with group scales: the conversion of bf16 weights,
// the way back, and the experts' SwiGLU product for decode batches.
//
// A weight matrix [rows, cols] is held as codes (two 4-bit numbers to a byte,
// the even column in the low half), one bf16 scale for each group of 32, 64
// or 128 consecutive columns of a row and, optionally, one zero point (0..15,
// a byte) for each group: value = (code - zero) * scale, zero 8 where there
// are no zero points.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <new>

#include "error.h"
#include "moe.h"
#include "ptx.cuh"
#include "tmap.h"

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

// Both directions move 2.5 bytes a weight: a lane takes 8 consecutive weights (16
// bytes), four such a pass, all loads first.  There and back 32768 x 14336 take
// 363 us in groups of 128, 0.96 of the copy rate; 12288 x 2048 in groups of 32
// with zero points 24 us, where the quantisation's instructions count.
constexpr int kConvertUnroll = 4;

__device__ __forceinline__ float bf16_low(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float bf16_high(uint32_t pair) { return __uint_as_float(pair & 0xffff0000u); }

// The 8 codes of a lane's weights by the definition: divisions.
__device__ __noinline__ uint32_t codes_by_division(uint4 q, float div, float z) {
  const uint32_t p[4] = {q.x, q.y, q.z, q.w};
  uint32_t word = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float v = j & 1 ? bf16_high(p[j >> 1]) : bf16_low(p[j >> 1]);
    word |= (uint32_t)fminf(fmaxf(rintf(v / div) + z, 0.f), 15.f) << (4 * j);
  }
  return word;
}

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {  // NaN wins
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 1 / s within 2^-22, s normal and at most 2^126.
__device__ __forceinline__ float reciprocal(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

// v / s rounded to an integer (half to even), plus 1.5 2^23, |v / s| below 16.
// v and s have 8 bits each, so a quotient that is not halfway between two
// integers is at least 2^-9 from it: the first sum rounds it to a multiple of
// 2^-10, which makes those exact that are halfway (inv is off by less than
// 2^-18 of the quotient) and leaves the others on their side; the second rounds
// to the integer.
constexpr float kGrid = 12288.f, kInteger = 12582912.f;  // 1.5 2^13 and 2^23: steps of 2^-10 and 1

__device__ __forceinline__ float rounded_quotient(float v, float inv) {
  return fmaf(v, inv, kGrid) + (kInteger - kGrid);
}

// a / 7.5 by one correction of the quotient by its remainder (Markstein);
// small ones, whose remainder is not exact, by division.
__device__ __forceinline__ float over_7_5(float a) {
  if (a < 1e-30f) return a / 7.5f;
  const float q = a * (1.f / 7.5f);
  return fmaf(fmaf(-q, 7.5f, a), 1.f / 7.5f, q);
}

// The G / 8 lanes of a group share its range by shuffles: the largest value and
// the largest negated one, at least 0 each, packed.  A division a weight would
// bound the kernel; only scales that are zero, subnormal or not finite take it.
// The scale itself: max / 7 is never near halfway between two bf16 numbers (7
// times an odd number is odd), so a product does; (hi - lo) / 15 can be.
template <int G, bool Z>
__global__ void __launch_bounds__(256)
    w4_quantize(long long n8, const uint4* __restrict__ w, uint32_t* __restrict__ codes,
                __nv_bfloat16* __restrict__ scales, uint8_t* __restrict__ zeros) {
  constexpr int kLanes = G / 8;
  const unsigned mask = ((1u << kLanes) - 1u) << (threadIdx.x & 31 & ~(kLanes - 1));
  const long long i0 = (long long)blockIdx.x * (256 * kConvertUnroll) + threadIdx.x;
  uint4 q[kConvertUnroll];
#pragma unroll
  for (int n = 0; n < kConvertUnroll; ++n)
    if (i0 + n * 256 < n8) q[n] = __ldcs(w + i0 + n * 256);
#pragma unroll
  for (int n = 0; n < kConvertUnroll; ++n) {
    const long long i = i0 + n * 256;
    if (i >= n8) break;  // n8 is a multiple of kLanes: the lanes of a group go together
    const uint32_t p[4] = {q[n].x, q[n].y, q[n].z, q[n].w};
    const uint32_t above = max2(max2(p[0], p[1]), max2(p[2], p[3]));
    const uint32_t below = max2(max2(p[0] ^ 0x80008000u, p[1] ^ 0x80008000u), max2(p[2] ^ 0x80008000u, p[3] ^ 0x80008000u));
    uint32_t range = max2(max2(__byte_perm(above, below, 0x5410), __byte_perm(above, below, 0x7632)), 0u);
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) range = max2(range, __shfl_xor_sync(mask, range, o));
    const float hi = bf16_low(range), lo = bf16_high(range);  // lo: how far below zero
    // (hi + lo) / 15, halved first so that no range overflows
    const float step = Z ? over_7_5(hi * 0.5f + lo * 0.5f) : fmaxf(hi, lo) * (1.f / 7.f);
    const bool finite = hi + lo < INFINITY || (hi < INFINITY && lo < INFINITY);
    const __nv_bfloat16 sb = __float2bfloat16(finite ? step : __uint_as_float(0x7fffffffu));
    const float s = __bfloat162float(sb);
    const bool plain = finite && s >= 1.17549435e-38f;
    const float inv = reciprocal(s);
    float z = 8.f;
    if (Z) {
      z = fminf(rounded_quotient(lo, inv) - kInteger, 15.f);
      if (!plain) z = !finite ? 8.f : fminf(rintf(lo / (s == 0.f ? 1.f : s)), 15.f);
    }
    const int zero = (int)z - 0x4b400000;  // less the bits of 1.5 2^23
    uint32_t word = 0;
#pragma unroll
    for (int j = 7; j >= 0; --j) {
      const float v = j & 1 ? bf16_high(p[j >> 1]) : bf16_low(p[j >> 1]);
      int c = __float_as_int(rounded_quotient(v, inv)) + zero;
      if (Z) c = min(c, 15);  // hi / s and lo / s may both be rounded up
      word = word * 16u + (uint32_t)c;
    }
    if (!plain) word = finite ? codes_by_division(q[n], s == 0.f ? 1.f : s, z) : 0x88888888u;
    __stcs(codes + i, word);
    if (i % kLanes == 0) {
      scales[i / kLanes] = sb;
      if (Z) zeros[i / kLanes] = (uint8_t)z;
    }
  }
}

// A code as bf16: 128 + code sits in the mantissa of a number of that binade;
// less 128 + zero exactly; times the scale, the one rounding.
template <int G, bool Z>
__global__ void __launch_bounds__(256)
    w4_dequantize(long long n8, const uint32_t* __restrict__ codes,
                  const __nv_bfloat16* __restrict__ scales, const uint8_t* __restrict__ zeros,
                  uint4* __restrict__ w) {
  const long long i0 = (long long)blockIdx.x * (256 * kConvertUnroll) + threadIdx.x;
  uint32_t word[kConvertUnroll], s2[kConvertUnroll], z2[kConvertUnroll];
#pragma unroll
  for (int n = 0; n < kConvertUnroll; ++n) {
    const long long i = i0 + n * 256;
    if (i >= n8) break;
    word[n] = __ldcs(codes + i);
    s2[n] = __bfloat16_as_ushort(__ldg(scales + i / (G / 8)));
    z2[n] = Z ? __ldg(zeros + i / (G / 8)) : 8u;
  }
#pragma unroll
  for (int n = 0; n < kConvertUnroll; ++n) {
    const long long i = i0 + n * 256;
    if (i >= n8) break;
    const uint32_t s = s2[n] * 0x00010001u, base = 0x43004300u + (z2[n] & 15u) * 0x00010001u;
    uint32_t v[4];  // columns (j, j + 4)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t u = ((word[n] >> (4 * j)) & 0x000f000fu) | 0x43004300u;
      asm("{\n\t.reg .b32 t;\n\tsub.rn.bf16x2 t, %1, %2;\n\tmul.rn.bf16x2 %0, t, %3;\n\t}"
          : "=r"(v[j])
          : "r"(u), "r"(base), "r"(s));
    }
    __stcs(w + i, make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                             __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632)));
  }
}

// --------------------------------------------------------------------- experts
//
// Two kernels, gate/up then down, of the same shape, and a third that adds the
// slots of a token (with few of them the last item of a column tile does).  An
// item is 64 weight rows of one expert (gate/up: 32 of each) times up to 8 of the
// expert's token rows; a team of 1, 2, 4 or 8 warps works an item off, its warps
// taking the 128-column blocks of the product in turn, and its first warp adds the
// others' sums.  Blocks of eight warps stay
// resident, two to an SM, and teams take items by turns.
//
// A warp's unit is 64 rows x 128 columns: 4 KB of codes, loaded by TMA into the
// warp's own ring of two stages with the token rows' 128 columns and the scales
// beside them, across items; one barrier a stage.  ldmatrix hands each lane the
// word of 8 codes (one row, 8 columns) that it needs of a 32-column chunk.
//
// Codes to numbers: a bf16 whose bits are the integer n < 256 is n 2^-133
// (below 128 a subnormal, from there on the first binade, with the same
// spacing), and mma.sync takes subnormal operands as they are.  So the codes
// of columns (0, 4) and (2, 6) are an AND with 000f000f of the word and the
// word shifted by 8, those of (1, 5) and (3, 7) an AND with 00f000f0, 16 times
// larger: five instructions for 8 codes.  The tokens' columns are paired the
// same way and scaled by 2^64, the 16-fold ones by 2^60, both exact in bf16;
// with |x| below 2^64 nothing overflows, and what is below 2^-57 counts as
// zero.  A group's sum of q x comes out as an fp32 sum of exact products; the
// sum of x over the group, from one more mma whose weights are ones, takes the
// zero point off: scale * (sum q x - zero * sum x), with the scale kept 2^40
// times too large and the other 2^29 at the end, so that the product of a small
// scale and a small sum does not vanish.  No weight is rounded.
constexpr int kRows = 64;             // weight rows of an item
constexpr int kChunk = 8;             // token rows of an item
constexpr int kBlockK = 128;          // columns of a unit
constexpr int kCodeBytes = kRows * kBlockK / 2;
constexpr int kTokenBytes = kBlockK * 2;  // of one token row of a unit
constexpr int kStages = 2;
constexpr int kItemWarps = 8;
constexpr int kBlocksSm = 2;
constexpr int kSms = 152;
constexpr int kInline = 32;           // slots up to which every block lists the experts' rows itself
// Mean token rows of an expert from which the tile kernels run.  The small
// kernels take 8 rows at once; on 128 experts of 2048 x 768, 113 us (small)
// against 115 at 8 rows, 121 against 120 at 9; on 8 of 4096 x 14336, 186 against
// 189 at 8 and 228 against 190 at 9; both in groups of 128 without zero points,
// the other kinds take the same number.  The mean is that of the routed experts:
// a few experts with many rows among idle ones, or a shared expert's T rows, stay
// on the small kernels where the mean is below (1024 tokens on 8 of 256 experts of
// 2048 x 768, 256 rows each, 147 us; 256 tokens of 256 + 1 experts of 7168 x 2048,
// eight each, 1600 us, their bytes 862).
constexpr int kTileMinRows = 9;
// Partial sums of a pass (slots times K splits) up to which the last item of a
// column tile adds them: more are added sooner by a kernel of their own.
constexpr int kFewSums = 64;
constexpr int kMaxSplit = 16;         // K splits of the down product
constexpr uint32_t kScaleX = 0x5f805f80u, kScaleX16 = 0x5d805d80u;  // 2^64, 2^60 twice
constexpr float kScaleUp = 1099511627776.f;                         // 2^40, in the arranged scales
constexpr float kUnscale = 536870912.f;                             // 2^29

struct Experts {
  int T, d, f, E, k, S;
  int team[2];              // warps to an item, gate/up and down
  int splits;               // K splits of the down product
  int scale_groups[2];      // an expert's fours of row tiles, gate/up and down
  int tile_tokens;          // token rows of an item of the tile kernels
  // gate/up's and down's scales and zero points as the units take them:
  // [expert][4 row tiles][128-column block][row tile][8 lanes][128 / G groups][8
  // rows], the last four tiles of an expert filled up
  const uint4* scales[2];
  const uint2* zeros[2];
  // large batches: the scales in fp16, each row's divided by the power of two in
  // exps, of gate, up and down
  const uint4* tile_scales[2];
  const short* exps[3];
  const __nv_bfloat16* x;   // [T, d]
  const int* idx;           // [T, k]
  const float* w;           // [T, k]
  // [T k + T S, f], columns of each 8 in the order 0 4 1 5 2 6 3 7 and scaled as
  // the product takes them; as they are in large batches
  __nv_bfloat16* h;
  float* y;                 // [splits, T k + T S, d]
  int* arrived;             // [d / 64] items of a column tile done, zero between passes; null: w4_combine adds
  int* status;              // MOE_E_TIMEOUT if a wait ran out
  void* list;               // List and Rows of a batch of more than kInline slots
  uint16_t *list_slot, *list_row;
  // large batches: x [T k + T S, d] in the order of the list and h, in fp16, and
  // the powers of two that their rows were divided by
  __half *x16, *h16;
  int *x_exp, *h_exp;
  __nv_bfloat16* out;       // [T, d]
};

// The experts that have rows, in order (up to kInline slots: of appearance).
struct List {
  int n_active;
  uint16_t start[kMaxE + 2];     // first of each one's entries in slot and row
  uint16_t expert[kMaxE + 2];
};

// Per token row of an expert: its slot (t k + j, and T k + t for the shared
// expert) and the token.
struct Rows {
  uint16_t* slot;
  uint16_t* row;
};

using moe::bulk_load;
using moe::fence_proxy_async_shared;
using moe::mbar_init;
using moe::smem_u32;

// The codes of both products: [rows of all experts, bytes of a row], boxes of
// 64 bytes x 32 rows (gate, up) or 64 (down), 64-byte swizzle: a row's 16-byte
// chunk c lies at chunk c ^ (row / 2 % 4), so that ldmatrix meets no conflicts.
struct Maps {
  CUtensorMap gate, up, down;
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// c = A B + c, or A B alone for the first of a sum.
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1, bool first) {
  if (first)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ void mbar_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y)
      : "memory");
}

// Where column c of a row of h is stored, and 2^64 or 2^60.
__device__ __forceinline__ int h_place(int c) { return (c & ~7) | ((c & 3) << 1) | (c >> 2 & 1); }
__device__ __forceinline__ float h_scale(int c) { return c & 1 ? 1152921504606846976.f : 18446744073709551616.f; }

__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// The expert of slot p, or -1 if it has none.
__device__ __forceinline__ int expert_at(const Experts& a, int p) {
  const int e = p < a.T * a.k ? __ldg(a.idx + p) : -1;
  return (unsigned)e < (unsigned)a.E ? e : -1;
}

// The list of at most 32 slots, by the first warp alone.
__device__ void list_few(const Experts& a, List* l, const Rows& rows) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const int e = expert_at(a, lane);
    const unsigned same = __match_any_sync(0xffffffffu, e);
    const bool leads = e >= 0 && lane == __ffs(same) - 1;
    const unsigned leaders = __ballot_sync(0xffffffffu, leads);
    int sum = leads ? __popc(same) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    const int all = __shfl_sync(0xffffffffu, sum, 31);
    const int start = __shfl_sync(0xffffffffu, leads ? sum - __popc(same) : 0, __ffs(same) - 1);
    if (leads) {
      const int at = __popc(leaders & ((1u << lane) - 1u));
      l->expert[at] = (uint16_t)e;
      l->start[at] = (uint16_t)start;
    }
    if (e >= 0) {
      const int to = start + __popc(same & ((1u << lane) - 1u));
      rows.slot[to] = (uint16_t)lane;
      rows.row[to] = (uint16_t)(lane / a.k);
    }
    if (lane == 0) {
      int n = __popc(leaders);
      l->start[n] = (uint16_t)all;
      if (a.S) {
        l->expert[n++] = (uint16_t)a.E;
        l->start[n] = (uint16_t)(all + a.T);
      }
      l->n_active = n;
    }
    if (a.S && lane < a.T) {
      rows.slot[all + lane] = (uint16_t)(a.T * a.k + lane);
      rows.row[all + lane] = (uint16_t)lane;
    }
  }
  __syncthreads();
}

// The list of a larger batch, once for both products: one block.  Slots keep
// their order inside an expert.  1024 slots a round: what each warp's 32 have of
// each expert, then a prefix over the warps.  More than one round counts first
// (`before`: what the rounds before have), since an expert's first entry lies
// behind every earlier expert's last.
__global__ void __launch_bounds__(1024) w4_list(Experts a) {
  __shared__ int count[kMaxE], before[kMaxE];
  __shared__ uint16_t table[32][kMaxE];
  __shared__ List l;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.T * a.k;
  wait_for_previous_kernel();
  let_next_kernel_start();
  const int rounds = (n + 1023) / 1024;
  int e = -1;
  unsigned same = 0;
  // a round's table, and its prefix over the warps on top of `from`
  auto tabulate = [&](int round, int* from) {
    for (int i = tid; i < 32 * kMaxE / 2; i += 1024) reinterpret_cast<uint32_t*>(table)[i] = 0u;
    e = expert_at(a, round * 1024 + tid);
    same = __match_any_sync(0xffffffffu, e);
    __syncthreads();
    if (e >= 0 && lane == __ffs(same) - 1) table[warp][e] = (uint16_t)__popc(same);
    __syncthreads();
    if (tid < kMaxE) {
      int run = from[tid];
      const int warps = min(32, (n - round * 1024 + 31) / 32);
#pragma unroll 8
      for (int q = 0; q < warps; ++q) {
        const int v = table[q][tid];
        table[q][tid] = (uint16_t)run;
        run += v;
      }
      from[tid] = run;
    }
    __syncthreads();
  };
  if (tid < kMaxE) count[tid] = before[tid] = 0;
  for (int r = 0; r < rounds; ++r) tabulate(r, count);
  __shared__ int start[kMaxE];
  if (tid < 32) {  // one warp: 8 experts a lane
    int c[8], sum = 0, act = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = count[lane * 8 + i];
      sum += c[i];
      act += c[i] > 0;
    }
    int s0 = sum, a0 = act;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int s1 = __shfl_up_sync(0xffffffffu, s0, o), a1 = __shfl_up_sync(0xffffffffu, a0, o);
      if (lane >= o) s0 += s1, a0 += a1;
    }
    if (lane == 31) {
      int na = a0;
      l.start[na] = (uint16_t)s0;
      if (a.S) {
        l.expert[na++] = (uint16_t)a.E;
        l.start[na] = (uint16_t)(s0 + a.T);
      }
      l.n_active = na;
    }
    s0 -= sum, a0 -= act;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      start[lane * 8 + i] = s0;
      if (c[i] > 0) {
        l.expert[a0] = (uint16_t)(lane * 8 + i);
        l.start[a0++] = (uint16_t)s0;
        s0 += c[i];
      }
    }
  }
  __syncthreads();
  for (int r = 0; r < rounds; ++r) {
    if (rounds > 1) tabulate(r, before);
    if (e >= 0) {
      const int to = start[e] + table[warp][e] + __popc(same & ((1u << lane) - 1u));
      a.list_slot[to] = (uint16_t)(r * 1024 + tid);
      a.list_row[to] = (uint16_t)((r * 1024 + tid) / a.k);
    }
    __syncthreads();
  }
  if (a.S) {
    const int first = l.start[l.n_active - 1];
    for (int t = tid; t < a.T; t += 1024) {
      a.list_slot[first + t] = (uint16_t)(n + t);
      a.list_row[first + t] = (uint16_t)t;
    }
  }
  for (int i = tid; i < (int)sizeof(List) / 4; i += 1024)
    static_cast<int*>(a.list)[i] = reinterpret_cast<const int*>(&l)[i];
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

// Wait for a barrier, two seconds at most: then the error is noted and the pass
// goes on, its output undefined, every later wait lasting 10 ms at most (so that
// a block still waits for copies of its own before it ends).  The clock and the
// noted error are looked at only after many tries: a load from global memory
// between two tries makes a wait end most of a microsecond late.
__device__ __forceinline__ void wait_stage(uint64_t* bar, uint32_t parity, int* status) {
#pragma unroll 1
  for (int i = 0; i < 1 << 14; ++i)
    if (moe::mbar_try_wait(bar, parity)) return;
  const uint64_t limit = moe::ld_relaxed(status) != 0 ? 10000000ull : 2000000000ull;
  if (!moe::mbar_wait(bar, parity, moe::globaltimer() + limit)) *status = MOE_E_TIMEOUT;
}

// One item: an expert, 64 of its rows, a K range and a chunk of token rows.
struct Item {
  int e, tile, split, rows, first, kb0, kb1;
};

constexpr int kInlineRows = 2 * kInline;                   // slots, and the shared expert's tokens

// Shared memory of a block, every region [warp][stage].
template <int G, bool Z>
struct Smem {
  static constexpr int kG = kBlockK / G;  // groups of a unit's row
  static constexpr int kScaleBytes = kRows * kG * 2;
  static constexpr int kZeroBytes = Z ? kRows * kG : 0;
  static constexpr int kSlots = kItemWarps * kStages;
  static constexpr int kCodes = 0;
  static constexpr int kTokens = kCodes + kSlots * kCodeBytes;
  static constexpr int kScales = kTokens + kSlots * kChunk * kTokenBytes;
  static constexpr int kZeros = kScales + kSlots * kScaleBytes;
  static constexpr int kBars = kZeros + kSlots * kZeroBytes;
  static constexpr int kLast = kBars + kSlots * 8;             // the stage of each warp's sums
  static constexpr int kItemStart = kLast + kItemWarps * 4;
  static constexpr int kList = kItemStart + (kMaxE + 2) * 4;
  static constexpr int kFew = kList + (int)sizeof(List);
  static constexpr int kBytes = kFew + 2 * kInlineRows * 2 + 512;  // and the alignment of the codes
  static_assert(kBytes <= 113 * 1024 - 128, "two blocks to an SM");
};

__device__ __forceinline__ void add_to(float2& a, float2 b) { a.x += b.x, a.y += b.y; }
__device__ __forceinline__ void add_to(float4& a, float4 b) { a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w; }
__device__ __forceinline__ float2 times(float w, float2 a) { return make_float2(w * a.x, w * a.y); }
__device__ __forceinline__ float4 times(float w, float4 a) { return make_float4(w * a.x, w * a.y, w * a.z, w * a.w); }

// A token's output at some columns: the weighted sum of its slots, in slot
// order, each the sum of its K splits, in order.  The loads of four slots and
// splits go out together, whether the slot has an expert or not.
template <typename V>
__device__ __forceinline__ V combine_token(const Experts& a, int t, int col) {
  const int n = a.k + a.S;
  const size_t slots = (size_t)a.T * n;
  V o{};
  for (int j0 = 0; j0 < n; j0 += 4) {
    const float* from[4];
    float wj[4];
    bool live[4];
    V y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = min(j0 + i, n - 1), p = j < a.k ? t * a.k + j : a.T * a.k + t;
      live[i] = j0 + i < n && (j >= a.k || expert_at(a, p) >= 0);
      wj[i] = j < a.k ? __ldg(a.w + p) : 1.f;
      from[i] = a.y + (size_t)p * a.d + col;
      y[i] = __ldcg(reinterpret_cast<const V*>(from[i]));
    }
#pragma unroll 4
    for (int q = 1; q < a.splits; ++q) {
#pragma unroll
      for (int i = 0; i < 4; ++i) add_to(y[i], __ldcg(reinterpret_cast<const V*>(from[i] + q * slots * a.d)));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (live[i]) add_to(o, times(wj[i], y[i]));
  }
  return o;
}

// One pass over the items for one of the two products.
template <bool DOWN, int G, bool Z>
__global__ void __launch_bounds__(kItemWarps * 32, kBlocksSm)
    w4_experts(const Experts a, const __grid_constant__ Maps maps) {
  using Sm = Smem<G, Z>;
  constexpr int kG = Sm::kG;
  extern __shared__ char smem_raw[];
  const int lr8 = threadIdx.x >> 2 & 7, lc4 = threadIdx.x & 3;  // an mma fragment's row and column pair
  char* smem = smem_raw + (-smem_u32(smem_raw) & 511u);
  int* sums_stage = reinterpret_cast<int*>(smem + Sm::kLast);
  int* item_start = reinterpret_cast<int*>(smem + Sm::kItemStart);  // [n_active + 1]
  List* list = reinterpret_cast<List*>(smem + Sm::kList);
  uint16_t* few = reinterpret_cast<uint16_t*>(smem + Sm::kFew);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int team = a.team[DOWN], member = warp & (team - 1);
  const int team_id = warp / team * gridDim.x + blockIdx.x;  // an SM's teams are far apart
  const int teams = kItemWarps / team * gridDim.x;
  const int K = DOWN ? a.f : a.d;
  const int rows_of = DOWN ? a.d : a.f;                // weight rows of an expert
  const int row_tiles = DOWN ? a.d / kRows : a.f / 32;
  const int splits = DOWN ? a.splits : 1;
  const int blocks_k = K / kBlockK;
  Rows rows{few, few + kInlineRows};
  if (tid < Sm::kSlots) {
    mbar_init(reinterpret_cast<uint64_t*>(smem + Sm::kBars) + tid, 1);
    moe::fence_mbar_init();
  }
  // gate/up is a pass's first kernel (or follows the list's): it waits for what
  // came before the pass; down starts only after every block of it has, so that
  // down may read the routing, or the list, at once
  if (!DOWN) {
    wait_for_previous_kernel();
    let_next_kernel_start();
  }
  if (a.T * a.k <= kInline) {
    list_few(a, list, rows);
  } else {
    for (int i = tid; i < (int)sizeof(List) / 4; i += blockDim.x)
      reinterpret_cast<int*>(list)[i] = __ldcg(static_cast<const int*>(a.list) + i);
    rows = Rows{a.list_slot, a.list_row};
    __syncthreads();
  }
  const int n_active = list->n_active;
  if (tid < 32) {  // items of the experts before each one
    int base = 0;
    for (int i0 = 0; i0 < n_active; i0 += 32) {
      const int i = i0 + lane;
      const int mine =
          i < n_active ? (list->start[i + 1] - list->start[i] + kChunk - 1) / kChunk * row_tiles * splits : 0;
      int sum = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      if (i < n_active) item_start[i] = base + sum - mine;
      base += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) item_start[n_active] = base;
  }
  __syncthreads();
  const int n_items = item_start[n_active];

  if (DOWN && a.arrived && n_items == 0) {  // no slot has an expert, and no kernel follows
    wait_for_previous_kernel();
    for (int i = blockIdx.x * blockDim.x + tid; i < a.T * a.d / 2; i += gridDim.x * blockDim.x)
      reinterpret_cast<uint32_t*>(a.out)[i] = 0u;
    return;
  }

  auto item_of = [&](int i, int* at, Item* it) {  // `at` only moves forward
    while (i >= item_start[*at + 1]) ++*at;
    const int n = list->start[*at + 1] - list->start[*at];
    const int local = i - item_start[*at];
    int c = 0, rest = local;
    if (n > kChunk) {  // chunks of the same weights side by side
      const int chunks = (n + kChunk - 1) / kChunk;
      rest = local / chunks;
      c = local - rest * chunks;
    }
    it->e = list->expert[*at];
    it->split = 0;
    it->tile = rest;
    it->kb0 = 0;
    it->kb1 = blocks_k;
    if (DOWN && splits > 1) {
      it->tile = rest / splits;
      it->split = rest - it->tile * splits;
      it->kb0 = blocks_k * it->split / splits;
      it->kb1 = blocks_k * (it->split + 1) / splits;
    }
    it->rows = min(kChunk, n - c * kChunk);
    it->first = list->start[*at] + c * kChunk;
  };

  const uint32_t codes = smem_u32(smem + Sm::kCodes) + warp * kStages * kCodeBytes;
  char* tokens = smem + Sm::kTokens + warp * kStages * kChunk * kTokenBytes;
  char* scales = smem + Sm::kScales + warp * kStages * Sm::kScaleBytes;
  char* zeros = smem + Sm::kZeros + warp * kStages * Sm::kZeroBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sm::kBars) + warp * kStages;

  // ---- the cursor of the loads, kStages units ahead of the products
  int l_item, l_at = 0, l_kb = 0, l_row = 0;
  Item l_it{};
  long long l_unit = 0;          // of the item's first column block; the next is 4 on
  const char* l_token = nullptr;  // lane n: token row n
  bool l_more;
  auto l_seek = [&]() {  // the next item from l_item on of which this warp has a unit
    while (true) {
      l_more = l_item < n_items;
      if (!l_more) return;
      item_of(l_item, &l_at, &l_it);
      l_kb = l_it.kb0 + member;
      if (l_kb < l_it.kb1) break;
      l_item += teams;
    }
    l_row = l_it.e * rows_of + l_it.tile * (DOWN ? kRows : 32);
    l_unit = ((long long)l_it.e * a.scale_groups[DOWN] + (l_it.tile >> 2)) * blocks_k * 4 + (l_it.tile & 3);
    if (lane < l_it.rows)
      l_token = reinterpret_cast<const char*>((DOWN ? a.h : a.x) + (size_t)(DOWN ? rows.slot : rows.row)[l_it.first + lane] * K);
  };
  auto l_next = [&](int stage, bool weights, bool rest) {
    if (!l_more) return;
    uint64_t* bar = bars + stage;
    if (lane == 0) {
      uint32_t bytes = rest ? l_it.rows * kTokenBytes : 0;
      if (weights) bytes += kCodeBytes + Sm::kScaleBytes + Sm::kZeroBytes;
      if (rest) moe::mbar_arrive_expect_tx(bar, bytes);
      else mbar_expect(bar, bytes);
      if (weights) {
        const uint32_t dst = codes + stage * kCodeBytes;
        if (DOWN) {
          tma_load(dst, &maps.down, bar, l_kb * 64, l_row);
        } else {
          tma_load(dst, &maps.gate, bar, l_kb * 64, l_row);
          tma_load(dst + kCodeBytes / 2, &maps.up, bar, l_kb * 64, l_row);
        }
        bulk_load(scales + stage * Sm::kScaleBytes, a.scales[DOWN] + (l_unit + l_kb * 4) * (Sm::kScaleBytes / 16),
                  Sm::kScaleBytes, bar);
        if (Z)
          bulk_load(zeros + stage * Sm::kZeroBytes, a.zeros[DOWN] + (l_unit + l_kb * 4) * (Sm::kZeroBytes / 8),
                    Sm::kZeroBytes, bar);
      }
    }
    if (rest && lane < l_it.rows)
      bulk_load(tokens + (stage * kChunk + lane) * kTokenBytes, l_token + l_kb * kTokenBytes, kTokenBytes, bar);
    l_kb += team;
    if (l_kb >= l_it.kb1) {
      l_item += teams;
      l_seek();
    }
  };

  // the weights wait for nobody: down's first stages load while gate/up ends
  l_item = team_id;
  l_seek();
#pragma unroll 1
  for (int s = 0; s < kStages; ++s) l_next(s, true, false);
  if (DOWN) {
    let_next_kernel_start();
    wait_for_previous_kernel();
    moe::fence_proxy_async_global();
  }
  l_item = team_id;
  l_at = 0;
  l_seek();
#pragma unroll 1
  for (int s = 0; s < kStages; ++s) l_next(s, false, true);

  int at = 0, stage = 0;
  uint32_t phase = 0;  // bit s: the parity that stage s waits for
  for (int i = team_id; i < n_items; i += teams) {
    Item it;
    item_of(i, &at, &it);
    float acc[4][4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[m][q] = 0.f;

#pragma unroll 1
    for (int kb = it.kb0 + member; kb < it.kb1; kb += team) {
      wait_stage(bars + stage, phase >> stage & 1u, a.status);
      phase ^= 1u << stage;
      const uint32_t st = codes + stage * kCodeBytes;
      const uint32_t tk = smem_u32(tokens) + (stage * kChunk + lr8) * kTokenBytes + lc4 * 16;
      const uint32_t sc = smem_u32(scales) + stage * Sm::kScaleBytes + lr8 * kG * 16;
      const uint32_t zr = smem_u32(zeros) + stage * Sm::kZeroBytes + lr8 * kG * 8;
      float part[4][4], sx[4];
      const int lr = lane & 15, lc = lane >> 4;  // ldmatrix: rows 0-15, chunk of the pair
#pragma unroll
      for (int q = 0; q < 2; ++q) {  // 64 columns: two chunks of 32
        uint32_t code[4][4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
          ldmatrix4(st + (m * 16 + lr) * 64 + (((2 * q + lc) ^ (lr >> 1 & 3)) << 4), code[m]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int c = 2 * q + half;
          const bool first = c * 32 % G == 0;
          // the tokens' pairs of columns 32 c + 8 t .. + 7
          const uint4 v = lds128(tk + c * 64);
          uint4 b = v;
          if (!DOWN)
            b = make_uint4(mul2(__byte_perm(v.x, v.z, 0x5410), kScaleX), mul2(__byte_perm(v.x, v.z, 0x7632), kScaleX16),
                           mul2(__byte_perm(v.y, v.w, 0x5410), kScaleX), mul2(__byte_perm(v.y, v.w, 0x7632), kScaleX16));
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const uint32_t u = code[m][half * 2], w = code[m][half * 2 + 1];
            mma16816(part[m], u & 0x000f000fu, w & 0x000f000fu, u & 0x00f000f0u, w & 0x00f000f0u, b.x, b.y, first);
          }
          mma16816(sx, 0x00010001u, 0x00010001u, 0x00100010u, 0x00100010u, b.x, b.y, first);
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const uint32_t u = code[m][half * 2] >> 8, w = code[m][half * 2 + 1] >> 8;
            mma16816(part[m], u & 0x000f000fu, w & 0x000f000fu, u & 0x00f000f0u, w & 0x00f000f0u, b.z, b.w, false);
          }
          mma16816(sx, 0x00010001u, 0x00010001u, 0x00100010u, 0x00100010u, b.z, b.w, false);
          if ((c + 1) * 32 % G == 0) {  // the group ends
            const int grp = c * 32 / G;
            const uint4 s4 = lds128(sc + grp * 16);
            const uint2 z4 = Z ? lds64(zr + grp * 8) : make_uint2(0u, 0u);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const uint32_t s2 = m == 0 ? s4.x : m == 1 ? s4.y : m == 2 ? s4.z : s4.w;
              const float s0 = __uint_as_float(s2 << 16), s1 = __uint_as_float(s2 & 0xffff0000u);
              const uint32_t z2 = (m < 2 ? z4.x : z4.y) >> (m & 1) * 16;
              const float z0 = Z ? (float)(z2 & 15u) : 8.f, z1 = Z ? (float)(z2 >> 8 & 15u) : 8.f;
              acc[m][0] += s0 * (part[m][0] - z0 * sx[0]);
              acc[m][1] += s0 * (part[m][1] - z0 * sx[1]);
              acc[m][2] += s1 * (part[m][2] - z1 * sx[2]);
              acc[m][3] += s1 * (part[m][3] - z1 * sx[3]);
            }
          }
        }
      }
      __syncwarp();
      // a member's last stage of an item holds its sums until they are added
      if (team == 1 || kb + team < it.kb1) l_next(stage, true, true);
      stage ^= 1;
    }

    if (team > 1) {  // the first warp adds the others' sums
      const int bar = 1 + warp / team;
      const bool had = it.kb0 + member < it.kb1;  // this warp had a unit, whose stage is free
      const int free_stage = stage ^ 1;
      if (member > 0 && had) {
        float4* buf = reinterpret_cast<float4*>(smem + Sm::kCodes + (warp * kStages + free_stage) * kCodeBytes) + lane;
#pragma unroll
        for (int m = 0; m < 4; ++m) buf[m * 32] = make_float4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
      }
      if (lane == 0) sums_stage[warp] = had ? free_stage : -1;
      asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(team * 32) : "memory");
      if (member == 0) {
        for (int q = 1; q < team; ++q) {
          if (sums_stage[warp + q] < 0) continue;
          const float4* buf =
              reinterpret_cast<const float4*>(smem + Sm::kCodes + ((warp + q) * kStages + sums_stage[warp + q]) * kCodeBytes) + lane;
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const float4 v = buf[m * 32];
            acc[m][0] += v.x;
            acc[m][1] += v.y;
            acc[m][2] += v.z;
            acc[m][3] += v.w;
          }
        }
      }
      asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(team * 32) : "memory");
      if (had) {
        fence_proxy_async_shared();  // the sums were written by the threads, TMA writes next
        __syncwarp();
        l_next(free_stage, true, true);
      }
      if (member > 0) continue;
    }
    // a lane's values: rows g and g + 8 of each 16, token rows 2 t and 2 t + 1
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col = lc4 * 2 + j;
      if (col >= it.rows) break;
      const size_t slot = rows.slot[it.first + col];
      if constexpr (!DOWN) {
        __nv_bfloat16* h = a.h + slot * a.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int m = q >> 1, v = (q & 1) * 2 + j;
          const int c = it.tile * 32 + m * 16 + (q & 1) * 8 + lr8;
          const float g = acc[m][v] * kUnscale, u = acc[m + 2][v] * kUnscale;
          // the one rounding between the products, to what the next one multiplies:
          // the output is off by 2.4e-3 of its norm, its own rounding alone 1.7e-3
          h[h_place(c)] = __float2bfloat16(g / (1.f + expf(-g)) * u * h_scale(c));
        }
      } else {
        float* y = a.y + ((size_t)it.split * (a.T * (a.k + a.S)) + slot) * a.d + it.tile * kRows + lr8;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          y[m * 16] = acc[m][j] * kUnscale;
          y[m * 16 + 8] = acc[m][2 + j] * kUnscale;
        }
      }
    }
    if (DOWN && a.arrived) {  // the warp that completes a column tile adds its tokens' slots
      __threadfence();
      __syncwarp();
      int last = 0;
      if (lane == 0) {
        last = atomicAdd(a.arrived + it.tile, 1) + 1 == n_items / row_tiles;
        if (last) a.arrived[it.tile] = 0;
      }
      if (__shfl_sync(0xffffffffu, last, 0)) {
        __threadfence();
        for (int t = 0; t < a.T; ++t) {
          const float2 o = combine_token<float2>(a, t, it.tile * kRows + lane * 2);
          *reinterpret_cast<__nv_bfloat162*>(a.out + (size_t)t * a.d + it.tile * kRows + lane * 2) =
              __floats2bfloat162_rn(o.x, o.y);
        }
      }
    }
  }
}

#include "w4_tiles.cuh"

// Arrange scales and zero points once as the units take them: one thread per
// lane and group of a unit.  first, second: the matrices of a unit's first and
// last 32 rows (gate and up; down twice, both32 = 0).
__global__ void __launch_bounds__(256)
    w4_arrange(Weight first, Weight second, int both32, int experts, int row_tiles, int blocks_k, int kg,
               uint4* scales, uint2* zeros, uint4* tile_scales, const short* exps_first,
               const short* exps_second) {
  const int fours = (row_tiles + 3) / 4;
  const long long units = (long long)experts * fours * blocks_k * 4;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < units * 8 * kg; i += (long long)gridDim.x * 256) {
    const int grp = (int)(i % kg), g = (int)(i / kg % 8);
    const long long unit = i / kg / 8;
    const int kb = (int)(unit / 4 % blocks_k);
    const long long four = unit / 4 / blocks_k;  // over the experts
    const int tile = (int)(four % fours) * 4 + (int)(unit & 3);
    if (tile >= row_tiles) continue;
    union {
      uint4 q;
      __nv_bfloat16 b[8];
    } s;
    union {
      uint2 q;
      uint8_t b[8];
    } z;
    union {
      uint4 q;
      __half h[8];
    } t;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const Weight& m = r < 4 ? first : second;
      const long long row =
          (four / fours * row_tiles + tile) * (both32 ? 32 : kRows) + (both32 ? (r & 3) * 8 : r * 8) + g;
      const long long o = (row * blocks_k + kb) * kg + grp;
      const float v = __bfloat162float(m.scales[o]);
      s.b[r] = __float2bfloat16(v * kScaleUp);  // exact
      t.h[r] = __float2half_rn(times_two_to(v, kScaleTop - (r < 4 ? exps_first : exps_second)[row]));
      if (zeros) z.b[r] = m.zeros[o] & 15;
    }
    scales[i] = s.q;
    tile_scales[i] = t.q;
    if (zeros) zeros[i] = z.q;
  }
}

__global__ void __launch_bounds__(128) w4_combine(const Experts a) {
  const int t = blockIdx.y, col = (blockIdx.x * 128 + threadIdx.x) * 4;
  let_next_kernel_start();
  wait_for_previous_kernel();
  if (col >= a.d) return;
  const float4 o = combine_token<float4>(a, t, col);
  union {
    __nv_bfloat162 b[2];
    uint2 u;
  } r;
  r.b[0] = __floats2bfloat162_rn(o.x, o.y);
  r.b[1] = __floats2bfloat162_rn(o.z, o.w);
  *reinterpret_cast<uint2*>(a.out + (size_t)t * a.d + col) = r.u;
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int check_matrix(long long rows, int cols, int group, const void* codes, const void* scales, const void* w) {
  if (group != 32 && group != 64 && group != 128) return moe::set_error(MOE_E_INVAL, "group must be 32, 64 or 128");
  if (rows < 0 || cols < 0 || cols % group != 0)
    return moe::set_error(MOE_E_INVAL, "cols must be a multiple of the group, rows and cols not negative");
  if (rows == 0 || cols == 0) return MOE_OK;
  if (rows > (1ll << 40) / cols) return moe::set_error(MOE_E_INVAL, "more than 2^40 weights");
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

dim3 convert_grid(long long n8) {
  constexpr int per = 256 * kConvertUnroll;
  return dim3((unsigned)((n8 + per - 1) / per));
}

}  // namespace

namespace {

struct Split {
  int team, splits;
};

// How a batch of T tokens is run.
struct Run {
  int tokens;   // > 0: on the kernels of w4_tiles.cuh, so many token rows an item
  Split gate_up, down;
};

// The workspace's regions, offsets from its start; h is first.
struct Layout {
  size_t y, x16, h16, x_exp, h_exp, status, arrived, list, slot, row, bytes;
};

}  // namespace

struct moe_w4 {
  int d, f, E, k, S, group;
  int T_max = 0;
  bool weights = false, zeros = false;  // set, with zero points
  Layout l{};
  Run run{};                            // of batches of run_T tokens
  int run_T = 0;
  Maps maps;
  TileMaps tile_maps;                                              // x and h: of the pass
  CUtensorMap x_maps[kTileTokens / 32], h_maps[kTileTokens / 32];  // by an item's token rows
  char* ws = nullptr;
  char* arranged = nullptr;  // the scales' and zero points' copies
  int device = -1;           // where they are
};

namespace {

// Teams of warps and K splits.  Estimated time, in us, of one product with
// `team` warps to an item and `splits` K splits: with w of an SM's 16 warps at
// work each takes 0.28 + 0.125 w for a unit (fitted to 6, 12 and 16 warps);
// an SM's items come in rounds of 16 / team, and each round ends with the
// teams' sums and the results (a warp alone 0.5, eight together 1.4).  Long
// chains of units end at different times (0.15 a unit), and the splits' partial
// sums cost the combine about 0.4 each.  The numbers are fitted to two layers and
// not measured apart from them.  One token of the 4096 x 14336 eight-expert
// layer: 53 us with single warps and no split, 42 with teams of 4 and 4 splits;
// 64 tokens of 128 experts of 2048 x 768: 97 us with teams of 8 in both products,
// 85 with teams of 2 and single warps.
float estimate(long long items, int blocks, int team, int splits) {
  const long long per_sm = (items * splits + kSms - 1) / kSms;
  const int units = ((blocks + splits - 1) / splits + team - 1) / team;
  const int teams = kItemWarps * kBlocksSm / team;
  const long long full = per_sm / teams, rest = per_sm % teams;
  auto unit_us = [](long long warps) { return 0.28f + 0.125f * (float)warps; };
  const float round = team == 1 ? 0.5f : team == 8 ? 1.4f : 0.6f;
  return units * ((float)full * unit_us(teams * team) + (rest ? unit_us(rest * team) : 0.f)) +
         round * (float)(full + (rest > 0)) + 0.15f * units + 0.4f * (splits - 1);
}

Split best_split(long long items, int blocks, int most_splits) {
  Split best{1, 1};
  float least = INFINITY;
  for (int splits = 1; splits <= most_splits && splits <= blocks; ++splits)
    for (int team = 1; team <= kItemWarps; team *= 2) {
      const float t = estimate(items, blocks, team, splits);
      if (t < least * 0.999f) least = t, best = Split{team, splits};
    }
  return best;
}

// Experts that T tokens can reach, each with its chunks of token rows if they
// spread evenly.
long long chunks_of(const moe_w4* h, int T) {
  const long long experts = std::min<long long>(h->E, (long long)T * h->k);
  const long long rows = ((long long)T * h->k + experts - 1) / experts;
  return experts * ((rows + kChunk - 1) / kChunk) + (h->S ? (T + kChunk - 1) / kChunk : 0);
}

Run run_of(const moe_w4* h, int T) {
  const long long experts = std::min<long long>(h->E, (long long)T * h->k);
  Run r;
  r.tokens = 0;
  if (T * h->k <= kInline || (long long)T * h->k < kTileMinRows * experts) {
    r.gate_up = best_split(chunks_of(h, T) * (h->f / 32), h->d / kBlockK, 1);
    r.down = best_split(chunks_of(h, T) * (h->d / kRows), h->f / kBlockK, kMaxSplit);
    return r;
  }
  // a block to an SM: the K split whose fullest block has the fewest columns
  // to do, with about three column blocks' time at the end of each item
  const long long rows = ((long long)T * h->k + experts - 1) / experts;
  // room for an expert with three deviations more rows than the mean
  const int room = (int)(rows + 3.f * sqrtf((float)rows));
  r.tokens = std::min(kTileTokens, (room + 31) / 32 * 32);
  const long long items = (experts * ((rows + r.tokens - 1) / r.tokens) + (h->S ? (T + r.tokens - 1) / r.tokens : 0)) *
                          ((h->d + 2 * kTileRows - 1) / (2 * kTileRows));
  const int blocks = h->f / kBlockK;
  r.gate_up = Split{1, 1};
  r.down = Split{1, 1};
  long long least = 0;
  for (int s = 1; s <= kMaxSplit && s <= blocks; ++s) {
    const long long cost = (items * s + kSms - 1) / kSms * ((blocks + s - 1) / s + 3) + s;
    if (s == 1 || cost < least) least = cost, r.down.splits = s;
  }
  return r;
}

Layout layout(const moe_w4* h, int T_max) {
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  const size_t slots = (size_t)T_max * (h->k + h->S);
  size_t y = 0;  // shorter batches may split more
  for (int T = 1; T <= T_max; ++T) y = std::max(y, (size_t)T * (h->k + h->S) * h->d * 4 * run_of(h, T).down.splits);
  Layout l;
  l.y = up(slots * h->f * 2);
  l.x16 = l.y + up(y);
  l.h16 = l.x16 + up(slots * h->d * 2);
  l.x_exp = l.h16 + up(slots * h->f * 2);
  l.h_exp = l.x_exp + up(slots * 4);
  l.status = l.h_exp + up(slots * 4);
  l.arrived = l.status + 256;
  l.list = l.arrived + up((size_t)h->d / kRows * 4);
  l.slot = l.list + up(sizeof(List));
  l.row = l.slot + up(slots * 2);
  l.bytes = l.row + up(slots * 2);
  return l;
}

// The copies that moe_w4_set_weights makes: gate/up's scales and down's, the same
// for the tile kernels with the rows' exponents, and the zero points of both.
struct Arranged {
  size_t down, tile, tile_down, exps[3], zeros, zeros_down, bytes;
};

// Fours of row tiles of an expert: 128 rows of gate and up, 256 of down.
int fours(const moe_w4* h, bool down) { return down ? (h->d + 255) / 256 : h->f / 128; }

Arranged arranged(const moe_w4* h) {
  const size_t n = (size_t)(h->E + h->S) * 256 / h->group;  // scales of a four and a column
  const size_t gate_up = n * fours(h, false) * h->d, down = n * fours(h, true) * h->f;
  Arranged at;  // every size is a multiple of 256 bytes
  at.down = 2 * gate_up;
  at.tile = at.down + 2 * down;
  at.tile_down = at.tile + 2 * gate_up;
  at.exps[0] = at.tile_down + 2 * down;
  at.exps[1] = at.exps[0] + (size_t)(h->E + h->S) * h->f * sizeof(short);
  at.exps[2] = at.exps[1] + (size_t)(h->E + h->S) * h->f * sizeof(short);
  at.zeros = at.exps[2] + (size_t)(h->E + h->S) * h->d * sizeof(short);
  at.zeros_down = at.zeros + gate_up;
  at.bytes = at.zeros_down + down;
  return at;
}

// Every kernel of a pass may be launched before the one in front of it has
// ended, and waits for it itself (wait_for_previous_kernel) before it touches
// anything that is written on the stream; so may the first of the next pass.
template <typename... A>
cudaError_t launch_after(void (*kernel)(A...), dim3 grid, int threads, int smem, cudaStream_t s,
                         const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Codes [rows, bytes]: boxes of 64 bytes x box_rows, 64-byte swizzle.
bool encode_codes(CUtensorMap* m, const void* base, uint64_t rows, uint64_t bytes, uint32_t box_rows) {
  cuuint64_t dims[2] = {bytes, rows};
  cuuint64_t strides[1] = {bytes};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t es[2] = {1, 1};
  return moe::encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 16-bit rows [rows, cols]: boxes of 64 columns x box_rows, 128-byte swizzle.
bool encode_rows(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t es[2] = {1, 1};
  return moe::encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Kernels {
  void (*gate_up)(Experts, Maps);
  void (*down)(Experts, Maps);
  void (*tiles_gate_up)(Experts, TileMaps);
  void (*tiles_down)(Experts, TileMaps);
  int smem;
};

template <int G, bool Z>
Kernels kernels_of() {
  return Kernels{w4_experts<false, G, Z>, w4_experts<true, G, Z>, w4_tiles<false, G, Z>, w4_tiles<true, G, Z>,
                 Smem<G, Z>::kBytes};
}

Kernels kernels(int group, bool zeros) {
  if (group == 32) return zeros ? kernels_of<32, true>() : kernels_of<32, false>();
  if (group == 64) return zeros ? kernels_of<64, true>() : kernels_of<64, false>();
  return zeros ? kernels_of<128, true>() : kernels_of<128, false>();
}

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
  return !h || T_max < 0 || T_max > kMaxT ? -1 : (long long)(layout(h, T_max).bytes + arranged(h).bytes);
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
  if (!moe::encode_fn()) return moe::set_error(MOE_E_CUDA, "cuTensorMapEncodeTiled is not available");
  if (e == cudaSuccess && h->arranged && h->device != dev)
    return moe::set_error(MOE_E_STATE, "the handle was reserved on another device");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (e == cudaSuccess && h->ws) {
    e = cudaStreamSynchronize(s);
    if (e == cudaSuccess) e = cudaFree(h->ws);
    h->ws = nullptr;
    h->T_max = 0;
  }
  if (e != cudaSuccess) return moe::set_cuda_error(e, "moe_w4_reserve");
  const Layout l = layout(h, T_max);
  const size_t bytes = l.bytes;
  if (!h->arranged && cudaMalloc(&h->arranged, arranged(h).bytes) != cudaSuccess) h->arranged = nullptr;
  h->device = dev;
  if (!h->arranged || cudaMalloc(&h->ws, bytes) != cudaSuccess) {
    h->ws = nullptr;
    cudaGetLastError();
    return moe::set_error(MOE_E_NOMEM, "workspace allocation failed");
  }
  e = cudaMemsetAsync(h->ws, 0, bytes, s);
  for (int z = 0; z < 2 && e == cudaSuccess; ++z) {
    const Kernels kn = kernels(h->group, z);
    const struct {
      const void* f;
      int smem;
    } all[] = {{(const void*)kn.gate_up, kn.smem},
               {(const void*)kn.down, kn.smem},
               {(const void*)kn.tiles_gate_up, 227 * 1024},
               {(const void*)kn.tiles_down, 227 * 1024}};
    for (const auto& k : all)
      if (e == cudaSuccess) e = cudaFuncSetAttribute(k.f, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
  }
  if (e != cudaSuccess) return moe::set_cuda_error(e, "moe_w4_reserve");
  const uint64_t slots = (uint64_t)T_max * (h->k + h->S);
  for (uint32_t n = 0; n < kTileTokens / 32; ++n)
    if (!encode_rows(&h->x_maps[n], h->ws + l.x16, slots, h->d, 32 * n + 32) ||
        !encode_rows(&h->h_maps[n], h->ws + l.h16, slots, h->f, 32 * n + 32))
      return moe::set_error(MOE_E_INVAL, "tensor map encoding failed");
  h->l = l;
  h->T_max = T_max;
  moe::clear_error();
  return MOE_OK;
}

int moe_w4_set_weights(moe_w4_t* h, const moe_w4_weight* gate, const moe_w4_weight* up,
                       const moe_w4_weight* down, void* stream) {
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
  if (!h->arranged) return moe::set_error(MOE_E_STATE, "moe_w4_reserve was not called");
  const Arranged at = arranged(h);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int kg = kBlockK / h->group;
  const bool z = gate->zeros != nullptr;
  cudaError_t e = cudaSuccess;
  short* exps[3];
  for (int i = 0; i < 3; ++i) {
    exps[i] = reinterpret_cast<short*>(h->arranged + at.exps[i]);
    const long long rows = (long long)(h->E + h->S) * (i < 2 ? h->f : h->d);
    if (e == cudaSuccess)
      e = launch(w4_row_exponents, dim3((unsigned)((rows + 7) / 8)), 256, s, take(m[i]).scales, rows,
                 (i < 2 ? h->d : h->f) / h->group, exps[i]);
  }
  for (int d = 0; d < 2 && e == cudaSuccess; ++d) {
    const int row_tiles = d ? h->d / kRows : h->f / 32, blocks_k = (d ? h->f : h->d) / kBlockK;
    const long long units = (long long)(h->E + h->S) * fours(h, d) * blocks_k * 4;
    e = launch(w4_arrange, dim3((unsigned)std::min<long long>((units * 8 * kg + 255) / 256, kSms * 8)), 256, s, take(d ? down : gate), take(d ? down : up), 1 - d,
               h->E + h->S, row_tiles, blocks_k, kg, reinterpret_cast<uint4*>(h->arranged + (d ? at.down : 0)),
               z ? reinterpret_cast<uint2*>(h->arranged + (d ? at.zeros_down : at.zeros)) : nullptr,
               reinterpret_cast<uint4*>(h->arranged + (d ? at.tile_down : at.tile)),
               static_cast<const short*>(exps[d ? 2 : 0]), static_cast<const short*>(exps[d ? 2 : 1]));
  }
  if (e != cudaSuccess) return moe::set_cuda_error(e, "w4_arrange");
  const uint64_t n = h->E + h->S;
  if (!encode_codes(&h->maps.gate, gate->codes, n * h->f, h->d / 2, 32) ||
      !encode_codes(&h->maps.up, up->codes, n * h->f, h->d / 2, 32) ||
      !encode_codes(&h->maps.down, down->codes, n * h->d, h->f / 2, kRows) ||
      !encode_codes(&h->tile_maps.gate, gate->codes, n * h->f, h->d / 2, kTileRows) ||
      !encode_codes(&h->tile_maps.up, up->codes, n * h->f, h->d / 2, kTileRows) ||
      !encode_codes(&h->tile_maps.down, down->codes, n * h->d, h->f / 2, kTileRows))
    return moe::set_error(MOE_E_INVAL, "tensor map encoding failed");
  h->weights = true;
  h->zeros = z;
  return MOE_OK;
}

int moe_w4_forward(moe_w4_t* h, int T, const void* x, const int32_t* idx, const float* w, void* out,
                   void* stream) {
  if (!h) return moe::set_error(MOE_E_INVAL, "null handle");
  if (!h->ws) return moe::set_error(MOE_E_STATE, "moe_w4_reserve was not called");
  if (!h->weights) return moe::set_error(MOE_E_STATE, "moe_w4_set_weights was not called");
  if (T < 0 || T > h->T_max) return moe::set_error(MOE_E_INVAL, "T out of range (0..T_max)");
  if (T == 0) return MOE_OK;
  if (!x || !idx || !w || !out) return moe::set_error(MOE_E_INVAL, "null tensor pointer");
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(idx, 4) || !aligned(w, 4))
    return moe::set_error(MOE_E_INVAL, "x and out must be 16-byte aligned, idx and w 4-byte");
  const Layout& l = h->l;
  if (h->run_T != T) h->run = run_of(h, T), h->run_T = T;
  const Run& r = h->run;
  Experts a;
  a.T = T;
  a.d = h->d;
  a.f = h->f;
  a.E = h->E;
  a.k = h->k;
  a.S = h->S;
  a.team[0] = r.gate_up.team;
  a.team[1] = r.down.team;
  a.splits = r.down.splits;
  a.tile_tokens = r.tokens;
  a.scale_groups[0] = fours(h, false);
  a.scale_groups[1] = fours(h, true);
  const Arranged at = arranged(h);
  a.scales[0] = reinterpret_cast<const uint4*>(h->arranged);
  a.scales[1] = reinterpret_cast<const uint4*>(h->arranged + at.down);
  a.zeros[0] = reinterpret_cast<const uint2*>(h->arranged + at.zeros);
  a.zeros[1] = reinterpret_cast<const uint2*>(h->arranged + at.zeros_down);
  a.tile_scales[0] = reinterpret_cast<const uint4*>(h->arranged + at.tile);
  a.tile_scales[1] = reinterpret_cast<const uint4*>(h->arranged + at.tile_down);
  for (int i = 0; i < 3; ++i) a.exps[i] = reinterpret_cast<const short*>(h->arranged + at.exps[i]);
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.idx = idx;
  a.w = w;
  a.h = reinterpret_cast<__nv_bfloat16*>(h->ws);
  a.y = reinterpret_cast<float*>(h->ws + l.y);
  a.x16 = reinterpret_cast<__half*>(h->ws + l.x16);
  a.h16 = reinterpret_cast<__half*>(h->ws + l.h16);
  a.x_exp = reinterpret_cast<int*>(h->ws + l.x_exp);
  a.h_exp = reinterpret_cast<int*>(h->ws + l.h_exp);
  // few partial sums: the last item of a column tile adds them, and no third
  // kernel follows (one token of the eight-expert layer 44.1 -> 42.9 us)
  const bool few = !r.tokens && T * (h->k + h->S) * r.down.splits <= kFewSums;
  a.arrived = few ? reinterpret_cast<int*>(h->ws + l.arrived) : nullptr;
  a.status = reinterpret_cast<int*>(h->ws + l.status);
  a.list = h->ws + l.list;
  a.list_slot = reinterpret_cast<uint16_t*>(h->ws + l.slot);
  a.list_row = reinterpret_cast<uint16_t*>(h->ws + l.row);
  a.out = static_cast<__nv_bfloat16*>(out);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Kernels kn = kernels(h->group, h->zeros);
  const bool listed = T * h->k > kInline;
  cudaError_t e = cudaSuccess;
  if (listed) e = launch_after(w4_list, dim3(1), 1024, 0, s, a);
  if (r.tokens) {
    const int smem = tile_smem(r.tokens, h->group, h->zeros).bytes;
    h->tile_maps.x = h->x_maps[r.tokens / 32 - 1];
    h->tile_maps.h = h->h_maps[r.tokens / 32 - 1];
    if (e == cudaSuccess) e = launch_after(w4_rows<false>, dim3(T * (h->k + h->S)), 256, 0, s, a);
    if (e == cudaSuccess) e = launch_after(kn.tiles_gate_up, dim3(kSms), kTileThreads, smem, s, a, h->tile_maps);
    if (e == cudaSuccess) e = launch_after(w4_rows<true>, dim3(T * (h->k + h->S)), 256, 0, s, a);
    if (e == cudaSuccess) e = launch_after(kn.tiles_down, dim3(kSms), kTileThreads, smem, s, a, h->tile_maps);
  } else {
    const dim3 grid(kSms * kBlocksSm);
    if (e == cudaSuccess) e = launch_after(kn.gate_up, grid, kItemWarps * 32, kn.smem, s, a, h->maps);
    if (e == cudaSuccess) e = launch_after(kn.down, grid, kItemWarps * 32, kn.smem, s, a, h->maps);
  }
  if (e == cudaSuccess && !a.arrived) e = launch_after(w4_combine, dim3((h->d / 4 + 127) / 128, T), 128, 0, s, a);
  return e == cudaSuccess ? MOE_OK : moe::set_cuda_error(e, "w4_experts");
}

int moe_w4_status(moe_w4_t* h, void* stream) {
  if (!h) return moe::set_error(MOE_E_INVAL, "null handle");
  if (!h->ws) return moe::set_error(MOE_E_STATE, "moe_w4_reserve was not called");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int* at = reinterpret_cast<int*>(h->ws + h->l.status);
  int status = 0;
  cudaError_t e = cudaMemcpyAsync(&status, at, sizeof(int), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  // with the arrivals that the pass may have left
  if (e == cudaSuccess && status) e = cudaMemsetAsync(at, 0, h->l.list - h->l.status, s);
  if (e != cudaSuccess) return moe::set_cuda_error(e, "moe_w4_status");
  return status ? moe::set_error(status, "device wait timed out") : MOE_OK;
}

void moe_w4_destroy(moe_w4_t* h) {
  if (!h) return;
  if (h->ws) cudaFree(h->ws);
  if (h->arranged) cudaFree(h->arranged);
  delete h;
}

}  // extern "C"
