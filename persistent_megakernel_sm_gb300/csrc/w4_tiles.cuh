// Experts on 4-bit weights for batches that give an expert many token rows:
// the products on the fifth-generation tensor cores (part of w4.cu).
//
// An item is 256 weight rows of one expert (gate/up: 128 of each, down: 256)
// times up to 128 of its token rows.  Codes come in by TMA; eight warps, a
// warpgroup for each 128 rows, turn a block of 128 columns into bf16 numbers
// and store them as an MMA operand in tensor memory (lane = weight row), and
// one thread issues the MMAs: A from tensor memory, the tokens from shared
// memory, fp32 sums in tensor memory over all of K.  Two operand buffers per
// warpgroup and four stages keep loads, conversion and MMAs apart.
//
// A code q as an operand: the bits n = q (or 16 q, for every other pair) of the
// word are the bf16 number n 2^-133, and one bf16 fused multiply-add with
// scale * 2^96 (2^92) and -8 scale 2^-37 gives (q - 8) scale 2^-37, rounded
// once (8 scale is exact); with zero points the subtraction comes first, exact,
// and the multiply rounds.  So a weight is its 4-bit value rounded to bf16 --
// what moe_w4_dequantize gives -- where the small-batch kernels round none:
// scaling the sums instead would cost one fp32 operation per row, token and
// group, as many as the conversion itself at 64 tokens.
//
// Per 128 columns and warp the conversion is 16 words x (5 + 4) instructions;
// the tokens' rows are read again for every 256 weight rows, which is why both
// matrices (or twice the rows) share them.
#pragma once

constexpr int kTileTokens = 128;
constexpr int kTileRows = 128;       // of one MMA; two of them share the tokens
constexpr int kTileStages = 4;
constexpr int kTileThreads = 320;    // 8 conversion warps, the loads' and the MMAs'
constexpr uint32_t kAColumn = 256;   // operand buffers: [tile][buffer][64 columns]
constexpr float kTileUnscale = 137438953472.f;  // 2^37

// x gathered by expert, and h: [T k + T S, columns], columns of each 8 in the
// order 0 4 1 5 2 6 3 7, in the order of the list.
struct TileMaps {
  CUtensorMap gate, up, down;  // codes, boxes of 64 bytes x 128 rows, 64-byte swizzle
  CUtensorMap x, h;            // boxes of 64 columns x 32 rows, 128-byte swizzle
};

template <int G, bool Z>
struct TileSmem {
  static constexpr int kG = kBlockK / G;
  static constexpr int kTokens = 0;                                  // [2 halves of 64 columns][128 rows][128 bytes]
  static constexpr int kHalf = kTileTokens * 128;
  static constexpr int kCodes = kTokens + 2 * kHalf;                 // [2 tiles][128 rows][64 bytes]
  static constexpr int kScales = kCodes + 2 * kTileRows * 64;        // 4 blocks of 64 rows
  static constexpr int kZeros = kScales + 4 * kRows * kG * 2;
  static constexpr int kStage = (kZeros + (Z ? 4 * kRows * kG : 0) + 1023) / 1024 * 1024;
  static constexpr int kWeightBytes = 2 * kTileRows * 64 + 4 * kRows * kG * (Z ? 3 : 2);
  static constexpr int kBars = kTileStages * kStage;
  static constexpr int kItemStart = kBars + 128;
  static constexpr int kList = kItemStart + (kMaxE + 2) * 4;
  static constexpr int kBytes = kList + (int)sizeof(List) + 1024;
  static_assert(kBytes <= 227 * 1024, "one block to an SM");
};

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

// D (+)= A B^T, A [128 x 16] bf16 in tensor memory (lane = row, 8 columns), B
// in shared memory, K-major.
__device__ __forceinline__ void mma_tmem_a(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t bf16_twice(float v) {
  const uint32_t b = __bfloat16_as_ushort(__float2bfloat16(v));
  return b | b << 16;
}

// Token rows in the order of the list: one block a row.
__global__ void __launch_bounds__(128) w4_gather(Experts a) {
  wait_for_previous_kernel();
  let_next_kernel_start();
  const int pos = blockIdx.x;
  const List* list = static_cast<const List*>(a.list);
  if (pos >= __ldcg(&list->start[__ldcg(&list->n_active)])) return;
  const uint4* from = reinterpret_cast<const uint4*>(a.x + (size_t)__ldcg(a.list_row + pos) * a.d);
  uint4* to = reinterpret_cast<uint4*>(a.xg + (size_t)pos * a.d);
  for (int i = threadIdx.x; i < a.d / 8; i += 128) {
    const uint4 v = __ldg(from + i);
    to[i] = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                       __byte_perm(v.y, v.w, 0x7632));
  }
}

template <bool DOWN, int G, bool Z>
__global__ void __launch_bounds__(kTileThreads, 1)
    w4_tiles(const Experts a, const __grid_constant__ TileMaps maps) {
  using Sm = TileSmem<G, Z>;
  constexpr int kG = Sm::kG;
  extern __shared__ char smem_raw[];
  char* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Sm::kBars);  // a stage's loads
  uint64_t* empty = full + kTileStages;                            // 8 warps and the MMAs are done with it
  uint64_t* a_full = empty + kTileStages;                          // [buffer] both tiles' operands stored
  uint64_t* a_free = a_full + 2;                                   // [buffer] read by the MMAs
  uint64_t* d_full = a_free + 2;                                   // an item's sums
  uint64_t* d_free = d_full + 1;                                   // read by the 8 warps
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(d_free + 1);
  int* item_start = reinterpret_cast<int*>(smem + Sm::kItemStart);
  List* list = reinterpret_cast<List*>(smem + Sm::kList);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int K = DOWN ? a.f : a.d;
  const int rows_of = DOWN ? a.d : a.f;
  const int tile_rows = DOWN ? 2 * kTileRows : kTileRows;  // of one matrix
  const int row_tiles = (rows_of + tile_rows - 1) / tile_rows;
  const int splits = DOWN ? a.splits : 1;
  const int blocks_k = K / kBlockK;

  if (tid == 0) {
    for (int s = 0; s < kTileStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 9);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(a_full + b, 8);
      mbar_init(a_free + b, 1);
    }
    mbar_init(d_full, 1);
    mbar_init(d_free, 8);
    moe::fence_mbar_init();
  }
  if (warp == 9) {
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
      const int mine = i < n_active ? (list->start[i + 1] - list->start[i] + kTileTokens - 1) / kTileTokens * row_tiles *
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
    const int chunks = (n + kTileTokens - 1) / kTileTokens;
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

  if (warp == 8) {
    if (lane == 0) {  // ---------------------------------------------- loads
      int at = 0, s = 0;
      uint32_t phase = 1;  // a fresh barrier's preceding phase has passed
      bool waited = false;
      for (int i = blockIdx.x; i < n_items; i += gridDim.x) {
        TileItem it;
        item_of(i, &at, &it);
        const int row0 = it.e * rows_of + it.tile * tile_rows;
        // rows past the expert's belong to the next one (or are zero): never stored
        const int boxes = (it.rows + 31) / 32;
        // scale blocks of 64 rows (gate/up: 32 of each) that follow one another
        const int blocks = min(4, (rows_of - it.tile * tile_rows + (DOWN ? 63 : 31)) / (DOWN ? 64 : 32));
        const long long unit0 =
            ((long long)it.e * (rows_of / (DOWN ? 64 : 32)) + (long long)it.tile * 4) * blocks_k;
        const uint32_t weights = 2 * kTileRows * 64 + blocks * kRows * kG * (Z ? 3 : 2);
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
          wait_stage(empty + s, phase, a.status);
          char* st = smem + s * Sm::kStage;
          moe::mbar_arrive_expect_tx(full + s, weights + boxes * 2 * 32 * 128);
          const uint32_t codes = smem_u32(st + Sm::kCodes);
          tma_load(codes, DOWN ? &maps.down : &maps.gate, full + s, kb * 64, row0);
          tma_load(codes + kTileRows * 64, DOWN ? &maps.down : &maps.up, full + s, kb * 64, DOWN ? row0 + kTileRows : row0);
          for (int q = 0; q < blocks; ++q) {
            const long long unit = unit0 + (long long)q * blocks_k + kb;
            bulk_load(st + Sm::kScales + q * kRows * kG * 2, a.scales[DOWN] + unit * (kRows * kG * 2 / 16),
                      kRows * kG * 2, full + s);
            if (Z)
              bulk_load(st + Sm::kZeros + q * kRows * kG, a.zeros[DOWN] + unit * (kRows * kG / 8), kRows * kG, full + s);
          }
          if (!waited) {  // the tokens (h) are the kernel's before; the weights wait for nobody
            wait_for_previous_kernel();
            moe::fence_proxy_async_global();
            waited = true;
          }
          for (int half = 0; half < 2; ++half)
            for (int b = 0; b < boxes; ++b)
              tma_load(smem_u32(st + Sm::kTokens + half * Sm::kHalf + b * 32 * 128), DOWN ? &maps.h : &maps.x, full + s,
                       kb * kBlockK + half * 64, it.first + b * 32);
          if (++s == kTileStages) s = 0, phase ^= 1;
        }
      }
    }
  } else if (warp == 9) {
    if (lane == 0) {  // ----------------------------------------------- MMAs
      int at = 0, s = 0, buf = 0, items = 0;
      uint32_t phase = 0, a_phase = 0;
      for (int i = blockIdx.x; i < n_items; i += gridDim.x, ++items) {
        TileItem it;
        item_of(i, &at, &it);
        const int n = max(16, (it.rows + 15) & ~15);
        const uint32_t idesc = moe::idesc_bf16(kTileRows, n);
        wait_stage(d_free, (items & 1) ^ 1, a.status);
        moe::tc_fence_after();
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
          wait_stage(full + s, phase, a.status);
          wait_stage(a_full + buf, a_phase, a.status);
          moe::tc_fence_after();
          const uint32_t tokens = smem_u32(smem + s * Sm::kStage + Sm::kTokens);
#pragma unroll
          for (int j = 0; j < kBlockK / 16; ++j) {
            const uint64_t b = moe::sw128_desc(tokens + (j >> 2) * Sm::kHalf + (j & 3) * 32);
#pragma unroll
            for (int t = 0; t < 2; ++t)
              mma_tmem_a(tmem + t * kTileTokens, tmem + kAColumn + (t * 2 + buf) * 64 + j * 8, b, idesc,
                         kb > it.kb0 || j > 0);
          }
          moe::mma_commit_all<1>(a_free + buf);
          moe::mma_commit_all<1>(empty + s);
          if (++s == kTileStages) s = 0, phase ^= 1;
          buf ^= 1;
          if (buf == 0) a_phase ^= 1;
        }
        moe::mma_commit_all<1>(d_full);
      }
    }
  } else {  // ------------------------------- conversion, and the sums' way out
    const int t = warp >> 2, row = (warp & 3) * 32 + lane;  // the tile, its row = the tensor memory's lane
    const uint32_t lane_at = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    // where this row's scales are in a stage: block, then [8 lanes][groups][8 rows]
    const int in_tile = DOWN ? t * kTileRows + row : row;  // of the item's rows of one matrix
    const int block = in_tile / (DOWN ? 64 : 32), in_block = in_tile % (DOWN ? 64 : 32);
    const int scale_at = block * kRows * kG + (in_block & 7) * kG * 8 + (in_block >> 3) + (DOWN ? 0 : t * 4);
    const int swizzle = row >> 1 & 3;
    int at = 0, s = 0, buf = 0, items = 0;
    uint32_t phase = 0, a_phase = 1;
    for (int i = blockIdx.x; i < n_items; i += gridDim.x, ++items) {
      TileItem it;
      item_of(i, &at, &it);
      for (int kb = it.kb0; kb < it.kb1; ++kb) {
        wait_stage(full + s, phase, a.status);
        char* st = smem + s * Sm::kStage;
        const uint32_t codes = smem_u32(st + Sm::kCodes) + (t * kTileRows + row) * 64;
        uint4 w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] = lds128(codes + ((c ^ swizzle) << 4));
        uint32_t sc[kG], zr[kG];
#pragma unroll
        for (int q = 0; q < kG; ++q) {
          sc[q] = reinterpret_cast<const uint16_t*>(st + Sm::kScales)[scale_at + q * 8];
          zr[q] = Z ? reinterpret_cast<const uint8_t*>(st + Sm::kZeros)[scale_at + q * 8] : 8u;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + s);
        wait_stage(a_free + buf, a_phase, a.status);
        moe::tc_fence_after();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t r[32];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int chunk = half * 2 + c;  // 32 columns
            const int q = chunk * 32 / G;
            // scale * 2^96 and 2^92, -8 scale 2^-37, each twice: the exponent
            // field of a bf16 is bits 7 to 14; a scale of 0 stays 0
            const float sf = __uint_as_float(sc[q] << 16);
            const uint32_t s1 = bf16_twice(sf * 79228162514264337593543950336.f), s16 = bf16_twice(sf * 4951760157141521099596496896.f);
            const uint32_t c8 = bf16_twice(sf * -5.820766091346741e-11f);
            const uint32_t z1 = zr[q] * 0x00010001u, z16 = zr[q] * 0x00100010u;
            const uint4 v = w[chunk];
            const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t u = words[k], u8 = u >> 8;
              uint32_t* o = r + c * 16 + k * 4;
              if (Z) {
                o[0] = mul2(sub2(u & 0x000f000fu, z1), s1);
                o[1] = mul2(sub2(u & 0x00f000f0u, z16), s16);
                o[2] = mul2(sub2(u8 & 0x000f000fu, z1), s1);
                o[3] = mul2(sub2(u8 & 0x00f000f0u, z16), s16);
              } else {
                o[0] = fma2(u & 0x000f000fu, s1, c8);
                o[1] = fma2(u & 0x00f000f0u, s16, c8);
                o[2] = fma2(u8 & 0x000f000fu, s1, c8);
                o[3] = fma2(u8 & 0x00f000f0u, s16, c8);
              }
            }
          }
          tmem_st32(lane_at + kAColumn + (t * 2 + buf) * 64 + half * 32, r);
        }
        tmem_st_wait();
        moe::tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(a_full + buf);
        if (++s == kTileStages) s = 0, phase ^= 1;
        buf ^= 1;
        if (buf == 0) a_phase ^= 1;
      }
      wait_stage(d_full, items & 1, a.status);
      moe::tc_fence_after();
      if constexpr (!DOWN) {
        // the warpgroups share the item's tokens, 16 at a time in turn
        for (int c0 = t * 16; c0 < it.rows; c0 += 32) {
          float g[16], u[16];
          moe::tmem_ld2x16(lane_at + c0, lane_at + kTileTokens + c0, g, u);
          const int col = it.tile * kTileRows + row;
          __nv_bfloat16* h = a.h + (size_t)(it.first + c0) * a.f + h_place(col);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            if (c0 + c >= it.rows) break;
            const float z = g[c] * kTileUnscale;
            h[(size_t)c * a.f] = __float2bfloat16(z / (1.f + expf(-z)) * (u[c] * kTileUnscale));
          }
        }
      } else {
        const int col = it.tile * tile_rows + in_tile;
        const size_t slots = (size_t)a.T * (a.k + a.S);
        for (int c0 = 0; c0 < it.rows; c0 += 16) {
          float y[16];
          moe::tmem_ld16(lane_at + t * kTileTokens + c0, y);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            if (c0 + c >= it.rows) break;
            const size_t slot = it.split * slots + __ldg(a.list_slot + it.first + c0 + c);
            if (col < a.d) a.y[slot * a.d + col] = y[c] * kTileUnscale;
          }
        }
      }
      moe::tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(d_free);
    }
  }
  __syncthreads();
  if (warp == 9) {
    moe::tc_fence_after();
    moe::tmem_dealloc<1>(tmem, 512);
  }
}
