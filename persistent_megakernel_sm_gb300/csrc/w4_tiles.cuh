// Experts on 4-bit weights for batches that give an expert many token rows:
// the products on the fifth-generation tensor cores (part of w4.cu).
//
// An item is 256 weight rows of one expert (gate/up: 128 of each, down: 256)
// times up to 128 of its token rows.  Codes come in by TMA; eight warps, a
// warpgroup for each 128 rows, turn them into 16-bit numbers, 64 columns at a
// time, and store them as an MMA operand in tensor memory (lane = weight row);
// a warp for each 128 rows issues the MMAs: A from tensor memory, the tokens
// from shared memory, fp32 sums in tensor memory over all of K; eight warps
// take an item's sums out.  Operands have four buffers of 64 columns for each
// 128 rows; with up to 64 tokens an item there is room for two sets of sums, so
// that one is taken out while the other comes in.  As many stages as fit (8 for
// 32 tokens an item, 4 for 128) cover a stage's way from its loads' start to
// its MMAs' end.
//
// What bounds it is the way from warp to warp: a look at a barrier takes 100 to
// 200 cycles even when it is ready, an MMA of any width 30 to 60 to issue.  So
// the loops look one step ahead and convert before they wait.
//
// A code q as an operand: the bits 0x6400 + q (0x5400 + 16 q, for every other
// pair) are the fp16 number 1024 + q (64 + q), so a subtraction gives q - zero,
// exact, and a multiply (q - zero) scale, rounded to 11 bits.  (Scaling the sums
// instead, which rounds nothing, would cost one fp32 operation per row, token and
// group, as many as the conversion itself at 64 tokens; in bf16 a conversion is
// 5 + 4 instructions and 256 tokens of the eight-expert layer took 189 us in place
// of 224, but the output was off by 3.4e-3 of its norm in place of 2.4e-3, of
// which 1.7e-3 are its own rounding to bf16 and as much h's.)  For fp16's range,
// each weight row's scales are divided by a power of two, the largest one's, and
// each row of x and of h too, by kernels of their own (w4_row_exponents once,
// w4_rows in every pass); the sums are multiplied back.  Scales under 2^-24 of
// their row's largest, and values under 2^-29 of theirs, lose bits.
//
// A conversion is 5 + 8 instructions for 8 codes.  The tokens' rows are read
// again for every 256 weight rows, which is why both matrices (or twice the
// rows) share them.
#pragma once

constexpr int kTileTokens = 128;     // at most
constexpr int kTileRows = 128;       // of one MMA; two of them share the tokens
constexpr int kTileStages = 8;       // at most
constexpr int kConvertWarps = 8;
constexpr int kFirstConvert = 4;     // warps 0 and 3 load, 1 and 2 issue the MMAs
constexpr int kFirstOut = kFirstConvert + kConvertWarps;  // eight warps take the sums out
constexpr int kOutWarps = 8;
constexpr int kTileThreads = (kFirstOut + kOutWarps) * 32;
// tensor memory: sums [set][tile], operands [tile][buffer][half][32 columns]
constexpr uint32_t kAColumn = 256;

// x gathered by expert, and h: [T k + T S, columns], columns of each 8 in the
// order 0 4 1 5 2 6 3 7, in the order of the list.
struct TileMaps {
  CUtensorMap gate, up, down;  // codes, boxes of 64 bytes x 128 rows, 64-byte swizzle
  CUtensorMap x, h;            // boxes of 64 columns x an item's token rows, 128-byte swizzle
};

// Shared memory: `stages` stages, then the barriers and the list.  In a stage,
// tokens [2 halves of 64 columns][token][128 bytes], codes [2 tiles][128
// rows][64 bytes], 4 blocks of 64 rows' scales and zero points.
struct TileSmem {
  int half, codes, scales, zeros, stage, stages, bars, bytes;
};

constexpr int kTileBars = 4 * 64 + 64;  // full, empty, operands stored and read; sums
constexpr int kTileTail = kTileBars + (kMaxE + 2) * 4 + (int)sizeof(List);

__host__ __device__ constexpr TileSmem tile_smem(int tokens, int group, bool zeros) {
  TileSmem m{};
  const int kg = kBlockK / group;
  m.half = tokens * 128;
  m.codes = 2 * m.half;
  m.scales = m.codes + 2 * kTileRows * 64;
  m.zeros = m.scales + 4 * kRows * kg * 2;
  m.stage = (m.zeros + (zeros ? 4 * kRows * kg : 0) + 1023) / 1024 * 1024;
  const int fit = (227 * 1024 - 1024 - kTileTail) / m.stage;
  m.stages = fit < kTileStages ? fit : kTileStages;
  m.bars = m.stages * m.stage;
  m.bytes = m.bars + kTileTail + 1024;
  return m;
}

struct TileItem {
  int e, tile, split, rows, first, kb0, kb1;
};

__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D (+)= A B^T, A [128 x 16] fp16 in tensor memory (lane = row, 8 columns), B
// in shared memory, K-major.
__device__ __forceinline__ void mma_tmem_a(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}

// Whether a barrier's phase is over, without waiting.  A look takes most of
// 200 cycles even at a barrier that is ready, so the loops look one step ahead.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

// Arrive on the barrier at `bar` when the MMAs issued so far are done.
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ uint32_t sub2h(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// (a & b) | c, c a constant: one instruction where b is in a register.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// Volatile, so that a conversion stays in front of the wait that follows it.
__device__ __forceinline__ uint32_t mul2hv(uint32_t a, uint32_t b) {
  uint32_t r;
  asm volatile("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126 to 127

// v 2^e, |e| up to 252; exact where the result is.
__device__ __forceinline__ float times_two_to(float v, int e) { return v * two_to(e >> 1) * two_to(e - (e >> 1)); }

// The magnitude of a bf16 number, as bits; 0 if it is not finite.
__device__ __forceinline__ uint32_t finite_bits(uint32_t b) {
  b &= 0x7fffu;
  return b < 0x7f80u ? b : 0u;
}

// The power of two at or below it, 2^-126 at least.
__device__ __forceinline__ int exponent_of(uint32_t bits) { return max((int)(bits >> 7), 1) - 127; }

constexpr int kScaleTop = 10, kTokenTop = 14;  // a row's largest scale is 2^10 to 2^11, 15 times that in fp16's range

// Per weight row the power of two of its largest scale: a warp a row.
__global__ void __launch_bounds__(256)
    w4_row_exponents(const __nv_bfloat16* scales, long long rows, int groups, short* exps) {
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  uint32_t m = 0u;
  for (int g = threadIdx.x & 31; g < groups; g += 32)
    m = max(m, finite_bits(__bfloat16_as_ushort(scales[row * groups + g])));
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) exps[row] = (short)exponent_of(m);
}

// The rows of x in the order of the list, or of h (H), as the tiles take them: in
// fp16 with their largest value at 2^14 to 2^15 (below that if it is under
// 2^-113).  One block a row; bound by its chain of loads (512 rows of 14336
// columns 9 us alone).
template <bool H>
__global__ void __launch_bounds__(256) w4_rows(Experts a) {
  constexpr int kKeep = H ? 8 : 4;  // loads a thread keeps until the factor is known; more are read again
  __shared__ uint32_t most[8];
  if (H) let_next_kernel_start();  // it has the list already
  wait_for_previous_kernel();
  if (!H) let_next_kernel_start();
  const int pos = blockIdx.x, tid = threadIdx.x, cols = H ? a.f : a.d;
  const List* list = static_cast<const List*>(a.list);
  const int row = H ? pos : __ldcg(a.list_row + pos);  // whatever it is behind the list's end
  if (pos >= __ldcg(&list->start[__ldcg(&list->n_active)])) return;
  const uint4* from = reinterpret_cast<const uint4*>((H ? a.h : a.x) + (size_t)row * cols);
  uint4* to = reinterpret_cast<uint4*>((H ? a.h16 : a.x16) + (size_t)pos * cols);
  const int n = cols / 8;
  auto words = [](const uint4& v, auto&& f) { f(v.x), f(v.y), f(v.z), f(v.w); };
  uint4 keep[kKeep];
#pragma unroll
  for (int q = 0; q < kKeep; ++q) keep[q] = tid + q * 256 < n ? __ldcg(from + tid + q * 256) : make_uint4(0u, 0u, 0u, 0u);
  uint32_t two = 0u;  // the largest magnitudes of even and of odd columns
  auto look = [&](uint32_t w) { two = __vmaxu2(two, w & 0x7fff7fffu); };
#pragma unroll
  for (int q = 0; q < kKeep; ++q) words(keep[q], look);
  for (int i = tid + kKeep * 256; i < n; i += 256) words(__ldcg(from + i), look);
  uint32_t m = __reduce_max_sync(0xffffffffu, max(two & 0xffffu, two >> 16));
  if (m >= 0x7f80u) {  // of the finite ones alone
    m = 0u;
    auto finite = [&](uint32_t w) { m = max(m, max(finite_bits(w), finite_bits(w >> 16))); };
    for (int i = tid; i < n; i += 256) words(__ldcg(from + i), finite);
    m = __reduce_max_sync(0xffffffffu, m);
  }
  if ((tid & 31) == 0) most[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 8; ++q) m = max(m, most[q]);
  const int e = max(exponent_of(m), kTokenTop - 127);
  if (tid == 0) (H ? a.h_exp : a.x_exp)[pos] = e;
  const float factor = two_to(kTokenTop - e);
  auto put = [&](int i, const uint4& v) {
    auto pair = [&](uint32_t lo, uint32_t hi) {  // two numbers' bits in the upper halves
      const __half2 h = __floats2half2_rn(__uint_as_float(lo) * factor, __uint_as_float(hi) * factor);
      return *reinterpret_cast<const uint32_t*>(&h);
    };
    to[i] = make_uint4(pair(v.x << 16, v.z << 16), pair(v.x & 0xffff0000u, v.z & 0xffff0000u), pair(v.y << 16, v.w << 16),
                       pair(v.y & 0xffff0000u, v.w & 0xffff0000u));
  };
#pragma unroll
  for (int q = 0; q < kKeep; ++q)
    if (tid + q * 256 < n) put(tid + q * 256, keep[q]);
  for (int i = tid + kKeep * 256; i < n; i += 256) put(i, __ldcg(from + i));
}

template <bool DOWN, int G, bool Z>
__global__ void __launch_bounds__(kTileThreads, 1)
    w4_tiles(const Experts a, const __grid_constant__ TileMaps maps) {
  constexpr int kG = kBlockK / G;
  const int most = a.tile_tokens;  // token rows of an item
  const TileSmem sm = tile_smem(most, G, Z);
  extern __shared__ char smem_raw[];
  char* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + sm.bars);  // a stage's loads, the weights' and the tokens'
  uint64_t* empty = full + kTileStages;                            // 16 warps and the MMAs are done with it
  uint64_t* a_full = empty + kTileStages;                          // [tile][buffer][half] the operand is stored (4 warps)
  uint64_t* a_free = a_full + 8;                                   // [tile][buffer][half] read by the MMAs
  uint64_t* d_full = a_free + 8;                                   // [set] an item's sums, both tiles'
  uint64_t* d_free = d_full + 2;                                   // [set] read by 8 warps
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(d_free + 2);
  int* item_start = reinterpret_cast<int*>(smem + sm.bars + kTileBars);
  List* list = reinterpret_cast<List*>(item_start + kMaxE + 2);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int K = DOWN ? a.f : a.d;
  const int rows_of = DOWN ? a.d : a.f;
  const int tile_rows = DOWN ? 2 * kTileRows : kTileRows;  // of one matrix
  const int row_tiles = (rows_of + tile_rows - 1) / tile_rows;
  const int splits = DOWN ? a.splits : 1;
  const int blocks_k = K / kBlockK;
  const int sets = most <= 64 ? 2 : 1, sum_columns = sets == 2 ? 64 : 128;

  if (tid == 0) {
    for (int s = 0; s < sm.stages; ++s) {
      mbar_init(full + s, 2);
      mbar_init(empty + s, kConvertWarps + 2);
    }
    for (int b = 0; b < 8; ++b) {
      mbar_init(a_full + b, 4);
      mbar_init(a_free + b, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(d_full + b, 2);
      mbar_init(d_free + b, kOutWarps);
    }
    moe::fence_mbar_init();
  }
  if (warp == 0) {
    moe::tmem_alloc<1>(tmem_at, 512);
    moe::tmem_relinquish<1>();
  }
  // the list is complete before the kernel before this one lets it start
  if (DOWN) let_next_kernel_start();
  for (int i = tid; i < (int)sizeof(List) / 4; i += kTileThreads)
    reinterpret_cast<int*>(list)[i] = __ldcg(static_cast<const int*>(a.list) + i);
  __syncthreads();
  const int n_active = list->n_active;
  if (tid < 32) {  // items of the experts before each one
    int base = 0;
    for (int i0 = 0; i0 < n_active; i0 += 32) {
      const int i = i0 + lane;
      const int mine = i < n_active ? (list->start[i + 1] - list->start[i] + most - 1) / most * row_tiles *
                                          splits : 0;
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
  moe::tc_fence_before();
  __syncthreads();
  moe::tc_fence_after();
  if (!DOWN) let_next_kernel_start();
  const uint32_t tmem = *tmem_at;
  const int n_items = item_start[n_active];

  auto item_of = [&](int i, int* at, TileItem* it) {  // `at` only moves forward
    while (i >= item_start[*at + 1]) ++*at;
    const int n = list->start[*at + 1] - list->start[*at];
    const int chunks = (n + most - 1) / most;
    const int local = i - item_start[*at], rest = local / chunks, c = local - rest * chunks;
    it->e = list->expert[*at];
    it->tile = rest / splits;
    it->split = rest - it->tile * splits;
    it->kb0 = blocks_k * it->split / splits;
    it->kb1 = blocks_k * (it->split + 1) / splits;
    // chunks of nearly the same size
    const int per = (n + chunks - 1) / chunks;
    it->rows = min(per, n - c * per);
    it->first = list->start[*at] + c * per;
  };

  if (warp == 0 || warp == 3) {  // ------------------- loads: weights, tokens
    if (elect_one()) {
      const bool weights = warp == 0;
      int at = 0, s = 0;
      uint32_t phase = 1;  // a fresh barrier's preceding phase has passed
      if (!weights) {      // the tokens (h) are the kernel's before; the weights wait for nobody
        wait_for_previous_kernel();
        moe::fence_proxy_async_global();
      }
      for (int i = blockIdx.x; i < n_items; i += gridDim.x) {
        TileItem it;
        item_of(i, &at, &it);
        const int row = it.e * rows_of + it.tile * tile_rows;
        // scale blocks of 64 rows (gate/up: 32 of each), four to a group
        const long long unit = ((long long)it.e * a.scale_groups[DOWN] + it.tile) * blocks_k;
        constexpr uint32_t kScaleBytes = 4 * kRows * kG * 2, kZeroBytes = Z ? 4 * kRows * kG : 0;
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
          wait_stage(empty + s, phase, a.status);
          const uint32_t st = smem_u32(smem) + s * sm.stage;
          if (weights) {
            moe::mbar_arrive_expect_tx(full + s, 2 * kTileRows * 64 + kScaleBytes + kZeroBytes);
            tma_load(st + sm.codes, DOWN ? &maps.down : &maps.gate, full + s, kb * 64, row);
            tma_load(st + sm.codes + kTileRows * 64, DOWN ? &maps.down : &maps.up, full + s, kb * 64,
                     DOWN ? row + kTileRows : row);
            bulk_load(smem + s * sm.stage + sm.scales, a.tile_scales[DOWN] + (unit + kb) * (kScaleBytes / 16), kScaleBytes,
                      full + s);
            if (Z)
              bulk_load(smem + s * sm.stage + sm.zeros, a.zeros[DOWN] + (unit + kb) * (kZeroBytes / 8), kZeroBytes,
                        full + s);
          } else {
            // rows past the expert's belong to the next one (or are zero): never stored
            moe::mbar_arrive_expect_tx(full + s, 2 * sm.half);
            tma_load(st, DOWN ? &maps.h : &maps.x, full + s, kb * kBlockK, it.first);
            tma_load(st + sm.half, DOWN ? &maps.h : &maps.x, full + s, kb * kBlockK + 64, it.first);
          }
          if (++s == sm.stages) s = 0, phase ^= 1;
        }
      }
    }
  } else if (warp < kFirstConvert) {  // ---------------------------------- MMAs
    // the whole warp loops, on values the compiler can see are the same in all
    // lanes (they then stay in uniform registers), and one lane issues
    const int t = __shfl_sync(0xffffffffu, warp, 0) - 1;
    const uint32_t smem0 = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t full0 = smem0 + sm.bars, a_free0 = full0 + (2 * kTileStages + 8 + t * 4) * 8;
    const uint64_t half = sm.half >> 4;
    int at = 0, s = 0, buf = 0, set = 0;
    uint32_t phase = 0, a_phase = 0, d_phase = 1;
    bool full_ready = false, a_ready = false;
    for (int i = blockIdx.x; i < n_items; i += gridDim.x) {
      TileItem it;
      item_of(i, &at, &it);
      const uint32_t idesc = moe::idesc_bf16(kTileRows, max(16, (__shfl_sync(0xffffffffu, it.rows, 0) + 15) & ~15)) &
                             ~(1u << 7 | 1u << 10);  // both operands fp16
      const int blocks = __shfl_sync(0xffffffffu, it.kb1 - it.kb0, 0);
      const uint32_t d = tm + (set * 2 + t) * sum_columns;
      wait_stage(d_free + set, d_phase, a.status);
      moe::tc_fence_after();
      for (int kb = 0; kb < blocks; ++kb) {
        const uint64_t b = moe::sw128_desc(smem0 + s * sm.stage);
        const uint32_t from = tm + kAColumn + (t * 2 + buf) * 64;
        const uint32_t done = full0 + (kTileStages + s) * 8, read = a_free0 + buf * 16;
        uint64_t* const a_bar = a_full + (t * 2 + buf) * 2;
        if (!full_ready) wait_stage(full + s, phase, a.status);
        if (!a_ready) wait_stage(a_bar, a_phase, a.status);
        moe::tc_fence_after();
        a_ready = mbar_test(a_bar + 1, a_phase);
        if (elect_one()) {
          mma_tmem_a(d, from, b, idesc, kb > 0);
#pragma unroll
          for (int j = 1; j < 4; ++j) mma_tmem_a(d, from + j * 8, b + j * 2, idesc, true);
          commit(read);
        }
        __syncwarp();
        if (!a_ready) wait_stage(a_bar + 1, a_phase, a.status);
        moe::tc_fence_after();
        if (++s == sm.stages) s = 0, phase ^= 1;
        buf ^= 1;
        if (buf == 0) a_phase ^= 1;
        full_ready = mbar_test(full + s, phase);
        a_ready = mbar_test(a_full + (t * 2 + buf) * 2, a_phase);
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_tmem_a(d, from + 32 + j * 8, b + half + j * 2, idesc, true);
          commit(read + 8);
          commit(done);
        }
        __syncwarp();
      }
      if (elect_one()) commit(full0 + (2 * kTileStages + 16 + set) * 8);  // d_full
      __syncwarp();
      if (++set == sets) set = 0, d_phase ^= 1;
    }
  } else if (warp < kFirstOut) {  // ------------------------------- conversion
    // the tile, and the row = the tensor memory's lane
    const int t = (warp - kFirstConvert) >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t to = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kAColumn + t * 128;
    // where this row's scales are in a stage: block, then [8 lanes][groups][8 rows]
    const int in_tile = DOWN ? t * kTileRows + row : row;  // of the item's rows of one matrix
    const int in_block = in_tile % (DOWN ? 64 : 32);
    const int scale_at =
        in_tile / (DOWN ? 64 : 32) * kRows * kG + (in_block & 7) * kG * 8 + (in_block >> 3) + (DOWN ? 0 : t * 4);
    const int swizzle = row >> 1 & 3;
    const uint32_t code_at = smem_u32(smem) + sm.codes + (t * kTileRows + row) * 64;
    uint32_t m1, m16;  // the codes' masks, in registers
    asm volatile("mov.b32 %0, 0x000f000f;\n\tmov.b32 %1, 0x00f000f0;" : "=r"(m1), "=r"(m16));
    int at = 0, s = 0, buf = 0;
    uint32_t phase = 0, a_phase = 1;
    bool full_ready = false;
    for (int i = blockIdx.x; i < n_items; i += gridDim.x) {
      TileItem it;
      item_of(i, &at, &it);
      for (int kb = it.kb0; kb < it.kb1; ++kb) {
        if (!full_ready) wait_stage(full + s, phase, a.status);
        const char* st = smem + s * sm.stage;
        uint4 w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] = lds128(code_at + s * sm.stage + ((c ^ swizzle) << 4));
        uint32_t sc[kG], zr[kG];
#pragma unroll
        for (int q = 0; q < kG; ++q) {
          sc[q] = reinterpret_cast<const uint16_t*>(st + sm.scales)[scale_at + q * 8];
          zr[q] = Z ? reinterpret_cast<const uint8_t*>(st + sm.zeros)[scale_at + q * 8] : 8u;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + s);
        if (++s == sm.stages) s = 0, phase ^= 1;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int at_buf = (t * 2 + buf) * 2 + half;
          const bool a_ready = mbar_test(a_free + at_buf, a_phase);
          if (half == 1) full_ready = mbar_test(full + s, phase);
          uint32_t r[32];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int q = (half * 2 + c) * 32 / G;
            const uint32_t s1 = sc[q] * 0x00010001u;
            const uint32_t z1 = zr[q] * 0x00010001u, z16 = zr[q] * 0x00100010u;
            const uint4 v = w[half * 2 + c];
            const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t u = words[k], u8 = u >> 8;
              uint32_t* o = r + c * 16 + k * 4;
              o[0] = mul2hv(sub2h(and_or(u, m1, 0x64006400u), z1 + 0x64006400u), s1);
              o[1] = mul2hv(sub2h(and_or(u, m16, 0x54005400u), z16 + 0x54005400u), s1);
              o[2] = mul2hv(sub2h(and_or(u8, m1, 0x64006400u), z1 + 0x64006400u), s1);
              o[3] = mul2hv(sub2h(and_or(u8, m16, 0x54005400u), z16 + 0x54005400u), s1);
            }
          }
          // everything but the stores comes before the wait for the MMAs of two
          // blocks ago
          if (!a_ready) wait_stage(a_free + at_buf, a_phase, a.status);
          moe::tc_fence_after();
          tmem_st32(to + buf * 64 + half * 32, r);
          tmem_st_wait();
          moe::tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(a_full + at_buf);
        }
        buf ^= 1;
        if (buf == 0) a_phase ^= 1;
      }
    }
  } else {  // ------------------------------------------------ the sums' way out
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_at = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const size_t slots = (size_t)a.T * (a.k + a.S);
    int at = 0, set = 0;
    uint32_t d_phase = 0;
    wait_for_previous_kernel();  // the tokens' exponents
    for (int i = blockIdx.x; i < n_items; i += gridDim.x) {
      TileItem it;
      item_of(i, &at, &it);
      const int col = it.tile * tile_rows + row;
      // the powers of two in halves, so that no partial product leaves the range
      const size_t at_row = (size_t)it.e * rows_of + col;
      const int e0 = __ldg(a.exps[DOWN ? 2 : 0] + at_row);
      const int e1 = !DOWN ? __ldg(a.exps[1] + at_row) : col + kTileRows < a.d ? __ldg(a.exps[2] + at_row + kTileRows) : 0;
      const float g1 = two_to(e0 >> 1), g2 = two_to(e0 - (e0 >> 1)), u1 = two_to(e1 >> 1), u2 = two_to(e1 - (e1 >> 1));
      wait_stage(d_full + set, d_phase, a.status);
      moe::tc_fence_after();
      const uint32_t from = lane_at + set * 2 * sum_columns;
      for (int c0 = (warp - kFirstOut) / 4 * 16; c0 < it.rows; c0 += 32) {  // two warps to a row, in turn
        float g[16], u[16];  // gate and up, or rows and rows + 128
        const int* exps = (DOWN ? a.h_exp : a.x_exp) + it.first + c0;
        const int x_e = (c0 + (lane & 15) < it.rows ? __ldcg(exps + (lane & 15)) : 0) - kScaleTop - kTokenTop;
        const float x_half = two_to(lane < 16 ? x_e >> 1 : x_e - (x_e >> 1));
        moe::tmem_ld2x16(from + c0, from + sum_columns + c0, g, u);
        const int n = min(16, it.rows - c0);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          if (c >= n) break;
          const float x1 = __shfl_sync(0xffffffffu, x_half, c), x2 = __shfl_sync(0xffffffffu, x_half, 16 + c);
          const float z = g[c] * g1 * x1 * g2 * x2, v = u[c] * u1 * x1 * u2 * x2;
          if constexpr (!DOWN) {  // bf16, the h that the header defines, though fp16 operands could hold more
            a.h[(size_t)(it.first + c0 + c) * a.f + col] = __float2bfloat16(__fdividef(z, 1.f + __expf(-z)) * v);
          } else {
            float* y = a.y + (it.split * slots + __ldg(a.list_slot + it.first + c0 + c)) * a.d + col;
            if (col < a.d) y[0] = z;
            if (col + kTileRows < a.d) y[kTileRows] = v;
          }
        }
      }
      moe::tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(d_free + set);
      if (++set == sets) set = 0, d_phase ^= 1;
    }
  }
  __syncthreads();
  if (warp == 0) {
    moe::tc_fence_after();
    moe::tmem_dealloc<1>(tmem, 512);
  }
}
