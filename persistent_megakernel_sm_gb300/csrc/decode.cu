// The whole MoE layer for a few tokens (1 to 16) in one kernel: router, choice,
// the chosen experts' SwiGLU and their weighted sum.
//
// With so few rows every product is a stream of weights past a handful of vectors,
// so the kernel is laid out by the weights alone: each expert that some token chose
// is read once, in bf16, and the grid's blocks (one an SM) share the weight rows
// evenly, whatever the choice was.
//   1  logits: the router's rows                              grid-wide wait
//   2  every block chooses for itself (a warp a token) and lists the experts;
//      h' = w silu(Wg x) (Wu x) for its share of the experts' f rows   grid-wide wait
//   3  out = sum over the listed experts of Wd h' for its share of the d rows: no
//      block needs another's sums, so there is no combine
// A product's tile is 16 weight rows times 8 or 16 token columns (gate and up: 8 rows
// of each, so that a lane has both for its values) on mma.sync m16n8k16.  The tensor
// cores are nearly idle here; they are used because a multiply-add for every weight
// and token would not keep up with HBM.  Weights go from HBM straight to the
// registers that the mma takes: a lane loads 16 bytes of a row, which the mma sees
// as another order of the same columns, the same for tokens.  A block's 16 warps
// split the columns; each loads a step ahead, and their sums meet in shared memory.
//
// Columns are the tokens themselves.  A token that did not choose an expert has a
// zero column there and takes nothing from its sums, which are kept apart expert by
// expert, so an infinity or a NaN in weights that a token did not choose does not
// reach it.  Sums are fp32, over at most 128 columns in the tensor cores and from
// there on rounded to nearest.  h' is held as the sum of two bf16 numbers, 16 bits
// in all: its rounding does not show in the output's, and costs one more mma on
// weights that are there anyway.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <new>

#include "error.h"
#include "moe.h"
#include "ptx.cuh"

namespace {

using bf16 = __nv_bfloat16;

constexpr int kMaxT = 16, kMaxK = 16, kMaxE = 256, kMaxD = 32768;
constexpr int kWarps = 16, kThreads = kWarps * 32;
constexpr int kBlock = 32;     // columns of a step's block: two mma
constexpr int kColumn = 20;    // floats of a token's column of a tile: 16, and 4 so that its lanes miss each other's banks
constexpr unsigned kAll = 0xffffffffu;
constexpr uint64_t kLimitNs = 2000000000ull;

struct Sched {
  int count, gen, status;
};

struct Decode {
  int T, d, f, E, k, S;
  const bf16 *x, *router_w, *gate, *up, *down;
  const float* bias;
  const int* idx_in;   // routed: the caller's choice, else null
  const float* w_in;
  int* idx_out;        // may be null
  float* w_out;
  bf16* out;
  float* logits;       // [T, E]
  bf16 *h_hi, *h_lo;   // [slots, f], slots expert by expert
  Sched* sched;
};

// What the choice is for a block: the experts in it, in order, the shared one last.
struct List {
  int n;
  int expert[kMaxE + 1];
  int start[kMaxE + 1];           // of its slots
  uint32_t tokens[kMaxE + 1];     // that chose it
  float w[kMaxE + 1][kMaxT];      // their weights
  int place[kMaxE];               // of an expert in the list, -1
  int idx[kMaxT][kMaxK];
  float idx_w[kMaxT][kMaxK];
  int ok;                         // of the last grid-wide wait
};

__device__ __forceinline__ uint4 load_weights(const bf16* p) {
  uint4 v;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Rows g and g + 8 of a tile, 32 columns, times a column block.
__device__ __forceinline__ void mma_block(float (&c)[4], const uint4 (&a)[2], uint4 b) {
  mma(c, a[0].x, a[1].x, a[0].y, a[1].y, b.x, b.y);
  mma(c, a[0].z, a[1].z, a[0].w, a[1].w, b.z, b.w);
}

// Every block arrives; false if the wait ran out somewhere.
__device__ bool grid_wait(Sched* s, int gen, uint64_t deadline, int* ok) {
  __syncthreads();
  if (threadIdx.x == 0) {
    *ok = 1;
    __threadfence();
    if (moe::atom_add_acq_rel(&s->count, 1) == (int)gridDim.x - 1) {
      s->count = 0;
      moe::st_release(&s->gen, gen + 1);
    } else {
      while (moe::ld_acquire(&s->gen) == gen) {
        if (moe::ld_relaxed(&s->status) != 0 || moe::globaltimer() > deadline) {
          if (moe::ld_acquire(&s->gen) != gen) break;
          s->status = MOE_E_TIMEOUT;
          *ok = 0;
          break;
        }
      }
    }
    __threadfence();
  }
  __syncthreads();
  return *ok != 0;
}

// Unsigned order of floats: NaN above everything, both zeros equal; kDead and below: -inf, never chosen.
constexpr uint32_t kDead = 0x007fffffu;
__device__ __forceinline__ uint32_t key_of(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t u = __float_as_uint(v + 0.f);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}

// A warp chooses for token t from its logits: the k largest, the lower expert on
// ties, their weights exp(l - max) over the kept ones' sum.
__device__ void choose(const Decode& p, List* list, int t) {
  const int lane = threadIdx.x & 31;
  uint32_t key[kMaxE / 32];
  float l[kMaxE / 32];
#pragma unroll
  for (int i = 0; i < kMaxE / 32; ++i) {
    const int e = lane + 32 * i;
    l[i] = e < p.E ? __ldcg(p.logits + t * p.E + e) : -INFINITY;
    key[i] = key_of(l[i]);
  }
  float mine = -INFINITY;  // the logit of slot `lane`
  int my_e = -1;
  for (int j = 0; j < p.k; ++j) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < kMaxE / 32; ++i) best = max(best, key[i]);
    best = __reduce_max_sync(kAll, best);
    if (best <= kDead) break;
    int at = kMaxE;
#pragma unroll
    for (int i = kMaxE / 32 - 1; i >= 0; --i)
      if (key[i] == best) at = lane + 32 * i;
    at = __reduce_min_sync(kAll, at);
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxE / 32; ++i)
      if (lane + 32 * i == at) v = l[i], key[i] = 0;
    v = __shfl_sync(kAll, v, at & 31);
    if (lane == j) mine = v, my_e = at;
  }
  float top = mine, sum;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float v = __shfl_xor_sync(kAll, top, o);
    top = (v > top || v != v) ? v : top;  // NaN stays
  }
  // equal logits weigh the same, infinities too
  const float e = my_e < 0 ? 0.f : mine == top ? 1.f : expf(mine - top);
  sum = e;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  if (lane < p.k) {
    list->idx[t][lane] = my_e;
    list->idx_w[t][lane] = my_e < 0 ? 0.f : e / sum;
  }
}

// The experts that the tokens chose, in order, with their tokens and weights.
__device__ void make_list(const Decode& p, List* list) {
  const int tid = threadIdx.x, lane = tid & 31;
  for (int e = tid; e < p.E; e += kThreads) list->place[e] = -1;
  __syncthreads();
  for (int i = tid; i < p.T * p.k; i += kThreads) {
    const int e = list->idx[i / p.k][i % p.k];
    if ((unsigned)e < (unsigned)p.E) list->place[e] = 0;
  }
  __syncthreads();
  if (tid < 32) {
    int n = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const bool live = e0 + lane < p.E && list->place[e0 + lane] == 0;
      const unsigned m = __ballot_sync(kAll, live);
      const int at = n + __popc(m & ((1u << lane) - 1u));
      if (live) list->place[e0 + lane] = at, list->expert[at] = e0 + lane;
      n += __popc(m);
    }
    if (lane == 0) {
      if (p.S) list->expert[n] = p.E;
      list->n = n + p.S;
    }
  }
  __syncthreads();
  const int n = list->n;
  for (int i = tid; i < n * kMaxT; i += kThreads) list->w[i / kMaxT][i % kMaxT] = 0.f;
  for (int i = tid; i < n; i += kThreads) list->tokens[i] = p.S && i == n - 1 ? (1u << p.T) - 1u : 0u;
  __syncthreads();
  if (tid < p.T) {  // a token's slots in order: an expert named twice has both weights
    for (int j = 0; j < p.k; ++j) {
      const int e = list->idx[tid][j];
      if ((unsigned)e >= (unsigned)p.E) continue;
      const int at = list->place[e];
      list->w[at][tid] += list->idx_w[tid][j];
      atomicOr(&list->tokens[at], 1u << tid);
    }
    if (p.S) list->w[n - 1][tid] = 1.f;
  }
  __syncthreads();
  if (tid < 32) {
    int base = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int mine = i0 + lane < n ? __popc(list->tokens[i0 + lane]) : 0;
      int sum = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kAll, sum, o);
        if (lane >= o) sum += v;
      }
      if (i0 + lane < n) list->start[i0 + lane] = base + sum - mine;
      base += __shfl_sync(kAll, sum, 31);
    }
  }
  __syncthreads();
}

// A tile's place: its two row blocks' first rows and how many of them there are.
struct Tile {
  const bf16 *lo, *hi;   // row 0 of rows 0..7 and of rows 8..15
  int n_lo, n_hi;        // rows that are there
  int at, first;         // list entry (phase 2), first row of the matrix
};

// Warps' sums of the tiles of a batch; two batches, so that one wait a batch is enough.
template <int NT>
struct Sums {
  static constexpr int kTiles = 4 / NT, kTile = NT * 8 * kColumn;
  float v[2][kTiles][kWarps][kTile];
};

template <int NT>
__device__ __forceinline__ void put_sums(float* to, const float (&acc)[NT][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float* c = to + (n * 8 + 2 * t) * kColumn + g;
    c[0] = acc[n][0], c[kColumn] = acc[n][1], c[8] = acc[n][2], c[kColumn + 8] = acc[n][3];
  }
}

// The tiles [0, n) of a block's share.  Each warp goes over its column blocks
// [b0, b1) of every tile, U at a time, the next step's loads under way while this
// one's mma run.  tile(i) gives a tile, load_b(tile, block, b) the token columns of a
// block, row(block) its offset from a row block's first row, change(block) whether a
// block begins another expert's columns, whose sums `keep` adds up, and end(i, row,
// token, sum) takes a finished sum, all threads of the block together.
template <int NT, int NB, int U, typename TileOf, typename RowPtr, typename LoadB, typename Close, typename End>
__device__ __forceinline__ void run_tiles(int n, int b0, int b1, int stride, Sums<NT>* sums, TileOf&& tile_of, RowPtr&& at,
                                          LoadB&& load_b, Close&& close, End&& end) {
  using S = Sums<NT>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c8 = (lane & 3) * 8;
  uint4 a[2][U][2], b[2][U][NB];
  Tile now, next;
  auto load = [&](int buf, const Tile& tile, int block) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool there = block + u < b1;
      const long long o = there ? at(block + u) + (long long)g * stride + c8 : 0;
      a[buf][u][0] = there && g < tile.n_lo ? load_weights(tile.lo + o) : make_uint4(0, 0, 0, 0);
      a[buf][u][1] = there && g < tile.n_hi ? load_weights(tile.hi + o) : make_uint4(0, 0, 0, 0);
      if (there) {
        load_b(tile, block + u, b[buf][u]);
      } else {
#pragma unroll
        for (int i = 0; i < NB; ++i) b[buf][u][i] = make_uint4(0, 0, 0, 0);
      }
    }
  };
  if (n == 0) return;
  float total[NT][4] = {};
  int i = 0, block = b0;
  now = tile_of(0);
  load(0, now, block);
  auto step = [&](auto which) {
    constexpr int buf = decltype(which)::value;
    const bool last = block + U >= b1;
    int i2 = i, block2 = block + U;
    if (last) {
      i2 = i + 1, block2 = b0;
      if (i2 < n) next = tile_of(i2);
    } else {
      next = now;
    }
    if (i2 < n) load(buf ^ 1, next, block2);
    float part[NT][4] = {};
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int q = 0; q < NB; ++q) mma_block(part[q % NT], a[buf][u], b[buf][u][q]);
      // the sums so far are one expert's, or the step's end
      if (u == U - 1 || close(block + u)) {
        const uint32_t tokens = close.tokens(now, block + u);
#pragma unroll
        for (int q = 0; q < NT; ++q) {
          const int t0 = q * 8 + (lane & 3) * 2;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (tokens >> (t0 + (j & 1)) & 1u) total[q][j] += part[q][j];
            part[q][j] = 0.f;
          }
        }
      }
    }
    if (last) {
      const int in = i % S::kTiles, batch = i / S::kTiles & 1;
      put_sums<NT>(sums->v[batch][in][warp], total);
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) total[q][j] = 0.f;
      if (in == S::kTiles - 1 || i == n - 1) {
        __syncthreads();
        const int tid = threadIdx.x, first = i - in;  // 16 rows x 8 NT tokens x kTiles: a thread each
        const int mine = tid / (NT * 128), token = tid / 16 % (NT * 8), row = tid & 15;
        float s = 0.f;
        if (mine <= in) {
          const float* c = &sums->v[batch][mine][0][token * kColumn + row];
#pragma unroll
          for (int w = 0; w < kWarps; ++w) s += c[w * S::kTile];
        }
        end(first + mine, mine <= in, row, token, s);
      }
    }
    i = i2, block = block2, now = next;
  };
  while (true) {
    step(std::integral_constant<int, 0>{});
    if (i >= n) break;
    step(std::integral_constant<int, 1>{});
    if (i >= n) break;
  }
  __syncthreads();  // the sums' memory is free again
}

// run_tiles' `close` where all columns are one product's.
struct OneProduct {
  uint32_t all;
  __device__ __forceinline__ bool operator()(int) const { return false; }
  __device__ __forceinline__ uint32_t tokens(const Tile&, int) const { return all; }
};

// Columns run through the listed experts' f, one after another.
struct ByExpert {
  const List* list;
  int blocks;  // of an expert
  __device__ __forceinline__ bool operator()(int block) const { return (block + 1) % blocks == 0; }
  __device__ __forceinline__ uint32_t tokens(const Tile&, int block) const {
    const int at = block / blocks;
    return at < list->n ? list->tokens[at] : 0u;
  }
};

__device__ __forceinline__ int share(long long total, int part, int parts) { return (int)(total * part / parts); }

template <int NT>
__global__ void __launch_bounds__(kThreads, 1) decode_layer(const __grid_constant__ Decode p) {
  extern __shared__ __align__(16) char smem[];
  Sums<NT>* sums = reinterpret_cast<Sums<NT>*>(smem);
  List* list = reinterpret_cast<List*>(smem + sizeof(Sums<NT>));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c8 = (lane & 3) * 8;
  const int block = blockIdx.x, blocks = gridDim.x;
  const uint64_t deadline = moe::globaltimer() + kLimitNs;
  int gen = tid == 0 ? moe::ld_acquire(&p.sched->gen) : 0;
  const int nkb = p.d / kBlock;

  auto load_x = [&](uint32_t tokens, int kb, uint4 (&b)[NT]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int t = n * 8 + g;
      b[n] = tokens >> t & 1u ? __ldg(reinterpret_cast<const uint4*>(p.x + (size_t)t * p.d + kb * kBlock + c8))
                              : make_uint4(0, 0, 0, 0);
    }
  };
  const uint32_t all = (1u << p.T) - 1u;

  // 1: logits
  if (p.router_w) {
    const int e0 = share(p.E, block, blocks), e1 = share(p.E, block + 1, blocks);
    auto tile_of = [&](int i) {
      const int e = e0 + 16 * i;
      const bf16* row = p.router_w + (size_t)e * p.d;
      return Tile{row, row + 8 * p.d, min(8, e1 - e), min(8, max(0, e1 - e - 8)), 0, e};
    };
    run_tiles<NT, NT, 2>((e1 - e0 + 15) / 16, share(nkb, warp, kWarps), share(nkb, warp + 1, kWarps), p.d, sums, tile_of,
                         [](int kb) { return kb * kBlock; },
                         [&](const Tile&, int kb, uint4 (&b)[NT]) { load_x(all, kb, b); }, OneProduct{all},
                         [&](int i, bool there, int row, int token, float s) {
                           const int e = e0 + 16 * i + row;
                           if (there && e < e1 && token < p.T) p.logits[token * p.E + e] = s + (p.bias ? p.bias[e] : 0.f);
                         });
    if (!grid_wait(p.sched, gen++, deadline, &list->ok)) return;
    if (warp < p.T) choose(p, list, warp);
  } else {
    for (int i = tid; i < p.T * p.k; i += kThreads) {
      list->idx[i / p.k][i % p.k] = p.idx_in[i];
      list->idx_w[i / p.k][i % p.k] = p.w_in[i];
    }
  }
  __syncthreads();
  if (block == 0 && p.router_w)
    for (int i = tid; i < p.T * p.k; i += kThreads) {
      if (p.idx_out) p.idx_out[i] = list->idx[i / p.k][i % p.k];
      if (p.w_out) p.w_out[i] = list->idx_w[i / p.k][i % p.k];
    }
  make_list(p, list);

  // 2: gate and up
  {
    const long long rows = (long long)list->n * p.f;
    const int r0 = share(rows, block, blocks), r1 = share(rows, block + 1, blocks);
    // tiles of 8 rows from r0 on, none over an expert's end
    const int a0 = r0 / p.f, lead = min(r1, (a0 + 1) * p.f) - r0;  // rows of the first expert
    const int lead_tiles = (lead + 7) / 8, per = p.f / 8;
    const int rest = r1 - r0 - lead;
    auto tile_of = [&](int i) {
      int row, end;
      if (i < lead_tiles) {
        row = r0 + 8 * i, end = r0 + lead;
      } else {
        const int q = (i - lead_tiles) / per;
        row = (a0 + 1 + q) * p.f + (i - lead_tiles) % per * 8;
        end = min(r1, (a0 + 2 + q) * p.f);
      }
      const int at = row / p.f, n = min(8, end - row);
      const size_t o = ((size_t)list->expert[at] * p.f + row % p.f) * p.d;
      return Tile{p.gate + o, p.up + o, n, n, at, row % p.f};
    };
    const int tiles = r1 > r0 ? lead_tiles + rest / p.f * per + (rest % p.f + 7) / 8 : 0;
    struct ByTile {
      const List* list;
      __device__ __forceinline__ bool operator()(int) const { return false; }
      __device__ __forceinline__ uint32_t tokens(const Tile& t, int) const { return list->tokens[t.at]; }
    };
    run_tiles<NT, NT, NT == 1 ? 4 : 2>(
        tiles, share(nkb, warp, kWarps), share(nkb, warp + 1, kWarps), p.d, sums, tile_of,
        [](int kb) { return kb * kBlock; },
        [&](const Tile& t, int kb, uint4 (&b)[NT]) { load_x(list->tokens[t.at], kb, b); }, ByTile{list},
        [&](int i, bool there, int row, int token, float s) {
          const float up = __shfl_xor_sync(kAll, s, 8);  // rows 8 to 15 are up's
          if (!there || row >= 8) return;
          const Tile t = tile_of(i);
          const uint32_t tokens = list->tokens[t.at];
          if (row >= t.n_lo || !(tokens >> token & 1u)) return;
          const float h = s / (1.f + expf(-s)) * up * list->w[t.at][token];
          const size_t slot = list->start[t.at] + __popc(tokens & ((1u << token) - 1u));
          const bf16 hi = __float2bfloat16_rn(h);
          p.h_hi[slot * p.f + t.first + row] = hi;
          // an infinity or a NaN is all in the first part
          const float rest = h - __bfloat162float(hi);
          p.h_lo[slot * p.f + t.first + row] = __float2bfloat16_rn(isfinite(rest) ? rest : 0.f);
        });
  }
  if (!grid_wait(p.sched, gen++, deadline, &list->ok)) return;

  // 3: down
  {
    const int r0 = share(p.d, block, blocks), r1 = share(p.d, block + 1, blocks);
    const int per = p.f / kBlock;
    const long long nb = (long long)list->n * per;
    auto tile_of = [&](int i) {
      const int row = r0 + 16 * i;
      const bf16* at = p.down + (size_t)row * p.f;
      return Tile{at, at + 8 * (size_t)p.f, min(8, r1 - row), min(8, max(0, r1 - row - 8)), 0, row};
    };
    run_tiles<NT, 2 * NT, 2>(
        (r1 - r0 + 15) / 16, share(nb, warp, kWarps), share(nb, warp + 1, kWarps), p.f, sums, tile_of,
        [&](int b) { return (long long)list->expert[b / per] * p.d * p.f + b % per * kBlock; },
        [&](const Tile&, int b, uint4 (&v)[2 * NT]) {
          const int at = b / per;
          const uint32_t tokens = list->tokens[at];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const int t = n * 8 + g;
            const bool on = tokens >> t & 1u;
            const size_t o = (size_t)(list->start[at] + __popc(tokens & ((1u << t) - 1u))) * p.f + b % per * kBlock + c8;
            v[n] = on ? __ldcg(reinterpret_cast<const uint4*>(p.h_hi + o)) : make_uint4(0, 0, 0, 0);
            v[NT + n] = on ? __ldcg(reinterpret_cast<const uint4*>(p.h_lo + o)) : make_uint4(0, 0, 0, 0);
          }
        },
        ByExpert{list, per},
        [&](int i, bool there, int row, int token, float s) {
          const int r = r0 + 16 * i + row;
          if (there && r < r1 && token < p.T) p.out[(size_t)token * p.d + r] = __float2bfloat16_rn(s);
        });
  }
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

struct Layout {
  size_t logits, h_hi, h_lo, bytes;
};

}  // namespace

struct moe_decode {
  int d, f, E, k, S;
  int T_max = 0, blocks = 0, device = -1;
  char* ws = nullptr;
  Layout l{};
};

namespace {

Layout layout(const moe_decode* h, int T_max) {
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  const size_t slots = (size_t)T_max * (h->k + h->S);
  Layout l;
  l.logits = 256;
  l.h_hi = l.logits + up((size_t)T_max * h->E * 4);
  l.h_lo = l.h_hi + up(slots * h->f * 2);
  l.bytes = l.h_lo + up(slots * h->f * 2);
  return l;
}

template <int NT>
constexpr int smem_bytes() {
  return (int)(sizeof(Sums<NT>) + sizeof(List));
}

int check_call(moe_decode* h, int T, const void* x, const void* gate, const void* up, const void* down, const void* out) {
  if (!h) return moe::set_error(MOE_E_INVAL, "null handle");
  if (!h->ws) return moe::set_error(MOE_E_STATE, "moe_decode_reserve was not called");
  if (T < 0 || T > h->T_max) return moe::set_error(MOE_E_INVAL, "T out of range (0..T_max)");
  if (T == 0) return MOE_OK;
  if (!x || !gate || !up || !down || !out) return moe::set_error(MOE_E_INVAL, "null tensor pointer");
  if (!aligned(x, 16) || !aligned(gate, 16) || !aligned(up, 16) || !aligned(down, 16) || !aligned(out, 16))
    return moe::set_error(MOE_E_INVAL, "tensors must be 16-byte aligned");
  return MOE_OK;
}

int run(moe_decode* h, Decode& p, cudaStream_t s) {
  p.d = h->d, p.f = h->f, p.E = h->E, p.k = h->k, p.S = h->S;
  p.sched = reinterpret_cast<Sched*>(h->ws);
  p.logits = reinterpret_cast<float*>(h->ws + h->l.logits);
  p.h_hi = reinterpret_cast<bf16*>(h->ws + h->l.h_hi);
  p.h_lo = reinterpret_cast<bf16*>(h->ws + h->l.h_lo);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)h->blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)(p.T <= 8 ? smem_bytes<1>() : smem_bytes<2>());
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeCooperative;  // the grid waits for itself
  at.val.cooperative = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, p.T <= 8 ? decode_layer<1> : decode_layer<2>, p);
  return e == cudaSuccess ? MOE_OK : moe::set_cuda_error(e, "decode_layer");
}

}  // namespace

extern "C" {

moe_decode_t* moe_decode_create(int d, int f, int E, int k, int shared_experts) {
  const char* bad = nullptr;
  if (d <= 0 || d % 128 != 0 || d > kMaxD) bad = "d must be a positive multiple of 128, at most 32768";
  else if (f <= 0 || f % 128 != 0 || f > kMaxD) bad = "f must be a positive multiple of 128, at most 32768";
  else if (E < 1 || E > kMaxE || k < 1 || k > E || k > kMaxK) bad = "need 1 <= k <= E <= 256 and k <= 16";
  else if (shared_experts < 0 || shared_experts > 1) bad = "shared_experts must be 0 or 1";
  if (bad) {
    moe::set_error(MOE_E_INVAL, bad);
    return nullptr;
  }
  moe_decode_t* h = new (std::nothrow) moe_decode_t();
  if (!h) {
    moe::set_error(MOE_E_NOMEM, "out of host memory");
    return nullptr;
  }
  h->d = d, h->f = f, h->E = E, h->k = k, h->S = shared_experts;
  moe::clear_error();
  return h;
}

long long moe_decode_workspace_bytes(const moe_decode_t* h, int T_max) {
  return !h || T_max < 0 || T_max > kMaxT ? -1 : (long long)layout(h, T_max).bytes;
}

int moe_decode_reserve(moe_decode_t* h, int T_max, void* stream) {
  if (!h) return moe::set_error(MOE_E_INVAL, "null handle");
  if (T_max < 1 || T_max > kMaxT) return moe::set_error(MOE_E_INVAL, "T_max out of range (1..16)");
  int dev = 0, major = 0, minor = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && (major != 10 || minor != 3))
    return moe::set_error(MOE_E_INVAL, "this library is built for sm_103a (GB300) only");
  if (e == cudaSuccess && h->ws && h->device != dev)
    return moe::set_error(MOE_E_STATE, "the handle was reserved on another device");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (e == cudaSuccess && h->ws) {
    e = cudaStreamSynchronize(s);
    if (e == cudaSuccess) e = cudaFree(h->ws);
    h->ws = nullptr;
    h->T_max = 0;
  }
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute((const void*)decode_layer<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<1>());
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute((const void*)decode_layer<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<2>());
  if (e != cudaSuccess) return moe::set_cuda_error(e, "moe_decode_reserve");
  const Layout l = layout(h, T_max);
  if (cudaMalloc(&h->ws, l.bytes) != cudaSuccess) {
    h->ws = nullptr;
    cudaGetLastError();
    return moe::set_error(MOE_E_NOMEM, "workspace allocation failed");
  }
  e = cudaMemsetAsync(h->ws, 0, 256, s);
  if (e != cudaSuccess) return moe::set_cuda_error(e, "moe_decode_reserve");
  h->device = dev;
  h->blocks = sms;
  h->l = l;
  h->T_max = T_max;
  moe::clear_error();
  return MOE_OK;
}

int moe_decode_forward(moe_decode_t* h, int T, const void* x, const void* router_w, const float* bias, const void* w_gate,
                       const void* w_up, const void* w_down, void* out, int32_t* idx, float* w, void* stream) {
  if (int rc = check_call(h, T, x, w_gate, w_up, w_down, out)) return rc;
  if (T == 0) return MOE_OK;
  if (!router_w) return moe::set_error(MOE_E_INVAL, "null tensor pointer");
  if (!aligned(router_w, 16) || !aligned(bias, 4) || !aligned(idx, 4) || !aligned(w, 4))
    return moe::set_error(MOE_E_INVAL, "router_w must be 16-byte aligned, bias, idx and w 4-byte");
  Decode p = {};
  p.T = T;
  p.x = static_cast<const bf16*>(x), p.router_w = static_cast<const bf16*>(router_w), p.bias = bias;
  p.gate = static_cast<const bf16*>(w_gate), p.up = static_cast<const bf16*>(w_up), p.down = static_cast<const bf16*>(w_down);
  p.out = static_cast<bf16*>(out), p.idx_out = idx, p.w_out = w;
  return run(h, p, static_cast<cudaStream_t>(stream));
}

int moe_decode_forward_routed(moe_decode_t* h, int T, const void* x, const int32_t* idx, const float* w, const void* w_gate,
                              const void* w_up, const void* w_down, void* out, void* stream) {
  if (int rc = check_call(h, T, x, w_gate, w_up, w_down, out)) return rc;
  if (T == 0) return MOE_OK;
  if (!idx || !w) return moe::set_error(MOE_E_INVAL, "null idx or w");
  if (!aligned(idx, 4) || !aligned(w, 4)) return moe::set_error(MOE_E_INVAL, "idx and w must be 4-byte aligned");
  Decode p = {};
  p.T = T;
  p.x = static_cast<const bf16*>(x), p.idx_in = idx, p.w_in = w;
  p.gate = static_cast<const bf16*>(w_gate), p.up = static_cast<const bf16*>(w_up), p.down = static_cast<const bf16*>(w_down);
  p.out = static_cast<bf16*>(out);
  return run(h, p, static_cast<cudaStream_t>(stream));
}

int moe_decode_status(moe_decode_t* h, void* stream) {
  if (!h) return moe::set_error(MOE_E_INVAL, "null handle");
  if (!h->ws) return moe::set_error(MOE_E_STATE, "moe_decode_reserve was not called");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Sched* at = reinterpret_cast<Sched*>(h->ws);
  int status = 0;
  cudaError_t e = cudaMemcpyAsync(&status, &at->status, sizeof(int), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  // with the arrivals that the pass may have left
  if (e == cudaSuccess && status) e = cudaMemsetAsync(at, 0, sizeof(Sched), s);
  if (e != cudaSuccess) return moe::set_cuda_error(e, "moe_decode_status");
  return status ? moe::set_error(status, "device wait timed out") : MOE_OK;
}

void moe_decode_destroy(moe_decode_t* h) {
  if (!h) return;
  if (h->ws) cudaFree(h->ws);
  delete h;
}

}  // extern "C"
