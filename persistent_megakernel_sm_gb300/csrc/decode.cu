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
// A product's tile is 32 weight rows (16 of gate and 16 of up) times 8 or 16 token
// columns on mma.sync m16n8k16.  The tensor cores are nearly idle here; they are used
// because a multiply-add for every weight and token would not keep up with HBM.  A
// stage is 512 columns of a tile and of the tokens that its expert has.  Four warps of
// a block bring its weights by bulk copies, four more the tokens' columns, into a ring of
// single rows (160 to 180 KB an SM on their way, whatever a stage has of them); the
// weights do not wait for the grid, so the ring is full of down's first ones when h' is
// complete.  Eight warps, in teams that take stages by turns, multiply, and their sums
// meet in shared memory once a tile.  A lane reads 16 bytes of a row at once, which the
// mma sees as another order of the same columns, the same for the tokens'.
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
#include <new>
#include <type_traits>

#include "error.h"
#include "moe.h"
#include "ptx.cuh"

namespace {

using bf16 = __nv_bfloat16;

constexpr int kMaxT = 16, kMaxK = 16, kMaxE = 256, kMaxD = 32768;
constexpr int kWarps = 8, kConsumers = kWarps * 32;
constexpr int kTeams = 2, kTeam = kWarps / kTeams;
constexpr int kBringers = 4;     // warps that bring weights, and as many that bring tokens
constexpr int kThreads = kConsumers + 2 * kBringers * 32;
constexpr int kBlock = 32;       // columns of two mma
constexpr int kRows = 32;        // of a tile: gate and up 16 each
constexpr int kChunk = 512;      // columns of a stage
constexpr int kBlocks = kChunk / kBlock / kTeam;  // of a warp
constexpr int kPitch = kChunk * 2 + 64;  // bytes of a row: two rows next to each other use all banks
constexpr int kColumn = 36;      // floats of a token's column of sums: 32, and 4 so that its lanes miss each other's banks
constexpr int kStages = 16;      // on their way, at most
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
  uint8_t order[kMaxE + 1][kMaxT];  // the same, one after another
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

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(moe::smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void sync_consumers() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory"); }

// Every block's consumers arrive; false if the wait ran out somewhere.
__device__ bool grid_wait(Sched* s, int gen, uint64_t deadline, int* ok) {
  sync_consumers();
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
  sync_consumers();
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
  for (int e = tid; e < p.E; e += kConsumers) list->place[e] = -1;
  sync_consumers();
  for (int i = tid; i < p.T * p.k; i += kConsumers) {
    const int e = list->idx[i / p.k][i % p.k];
    if ((unsigned)e < (unsigned)p.E) list->place[e] = 0;
  }
  sync_consumers();
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
  sync_consumers();
  const int n = list->n;
  for (int i = tid; i < n * kMaxT; i += kConsumers) list->w[i / kMaxT][i % kMaxT] = 0.f;
  for (int i = tid; i < n; i += kConsumers) list->tokens[i] = p.S && i == n - 1 ? (1u << p.T) - 1u : 0u;
  sync_consumers();
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
  sync_consumers();
  if (tid < 32) {
    int base = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int mine = i0 + lane < n ? __popc(list->tokens[i0 + lane]) : 0;
      for (int j = 0, left = mine ? (int)list->tokens[i0 + lane] : 0; left; ++j, left &= left - 1)
        list->order[i0 + lane][j] = (uint8_t)(__ffs(left) - 1);
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
  sync_consumers();
}

// Warps' sums of a tile; two tiles' worth, so that one wait a tile is enough.
template <int NT>
struct Sums {
  static constexpr int kTile = NT * 8 * kColumn;
  float v[2][kWarps][kTile];
};

template <int NT>
struct Smem {
  static constexpr int kRing = NT == 1 ? 168 : 152;  // rows; a stage has 64 at most
  char ring[kRing][kPitch];
  Sums<NT> sums;
  List list;
  uint64_t full[kStages], empty[kStages], h_ready;
  int abort;  // a wait ran out: nothing more is brought
};

// Where one side of the ring stands: the stage's barriers and its first row.
template <int RING>
struct At {
  int stage = 0, row = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int rows) {
    if (++stage == kStages) stage = 0, parity ^= 1;
    row += rows;
    if (row >= RING) row -= RING;
  }
  __device__ __forceinline__ int at(int i) const { return row + i >= RING ? row + i - RING : row + i; }
};

// A bringing warp's view of what is free: a stage's rows are the consumers' until its
// `empty` completes.
template <int NT>
struct Room {
  Smem<NT>* sm;
  uint64_t deadline;
  At<Smem<NT>::kRing> at;        // of the next stage
  int oldest = 0, out = 0, used = 0;
  uint32_t oldest_parity = 0;
  int rows_of = 0;               // lane i: rows of the stage on barriers i

  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
    bool done = false;
    while (!done && !*static_cast<volatile int*>(&sm->abort)) {
      for (int i = 0; i < 32 && !done; ++i) done = moe::mbar_try_wait(bar, parity);
      if (!done && moe::globaltimer() > deadline) break;
    }
    return __all_sync(kAll, done);
  }
  // room for a stage of `rows`; false if the wait ran out
  __device__ __forceinline__ bool make(int rows) {
    while (used + rows > Smem<NT>::kRing || out == kStages) {
      if (!wait(&sm->empty[oldest], oldest_parity)) return false;
      used -= __shfl_sync(kAll, rows_of, oldest);
      --out;
      if (++oldest == kStages) oldest = 0, oldest_parity ^= 1;
    }
    return true;
  }
  __device__ __forceinline__ void take(int rows) {
    if ((threadIdx.x & 31) == at.stage) rows_of = rows;
    used += rows, ++out;
    at.next(rows);
  }
};

// A block's share of the experts' f rows, tile by tile: at most 16 (of gate and of
// up), none over an expert's end.  Stepped along: a division a tile in every warp, a
// stage even, is what the kernel then waits for.
struct GateUpTiles {
  int f, left;      // rows still to come, with this tile's
  int entry, first; // of the list, first row there
  __device__ __forceinline__ GateUpTiles(int f_, int r0, int r1) : f(f_), left(r1 - r0), entry(r0 / f_), first(r0 % f_) {}
  __device__ __forceinline__ int rows() const { return min(min(16, left), f - first); }
  __device__ __forceinline__ void next() {
    const int n = rows();
    left -= n, first += n;
    if (first == f) ++entry, first = 0;
  }
};

__device__ __forceinline__ int share(long long total, int part, int parts) { return (int)(total * part / parts); }

// What a stage is: weight rows (and how many of them are there), the tokens that it is
// for, and how many rows each of them has (h': two).
struct Stage {
  int rows, tokens, parts, columns;
  __device__ __forceinline__ int all() const { return rows + parts * __popc(tokens); }
};

// A consumer warp's way through the stages.  A wait that runs out leaves its mark in
// `abort`; no barrier of the block is left out.
template <int NT>
struct Consumer {
  Smem<NT>* sm;
  uint64_t deadline;
  int* status;
  At<Smem<NT>::kRing> at;
  int turn = 0, tile = 0;   // the team whose stage is next; tiles so far
  bool fine = true;
  float total[2][NT][4];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) total[m][q][j] = 0.f;
  }

  // One stage; the mma's rows 8 to 15 are those from `hi` on.
  template <int PARTS>
  __device__ __forceinline__ void stage(const Stage& st, int hi) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int team = warp / kTeam, member = warp % kTeam;
    const int n = __popc(st.tokens);
    if (turn == team) {
      const char* a_rows[2][2];
      const char* b_rows[PARTS * NT];
      const int in_row = t * 16 + member * (kBlocks * kBlock * 2);
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        a_rows[m][0] = sm->ring[at.at(8 * m + g)] + in_row;
        a_rows[m][1] = sm->ring[at.at(hi + 8 * m + g)] + in_row;
      }
#pragma unroll
      for (int q = 0; q < PARTS * NT; ++q) {
        const int token = q % NT * 8 + g;
        b_rows[q] = st.tokens >> token & 1
                        ? sm->ring[at.at(st.rows + q / NT * n + __popc(st.tokens & ((1 << token) - 1)))] + in_row : nullptr;
      }
      fine = fine && moe::mbar_wait(&sm->full[at.stage], at.parity, deadline);
      float part[2][NT][4] = {};
#pragma unroll
      for (int u = 0; u < kBlocks; ++u) {
        if ((member * kBlocks + u) * kBlock >= st.columns) break;
        uint4 b[PARTS * NT];
#pragma unroll
        for (int q = 0; q < PARTS * NT; ++q)
          b[q] = b_rows[q] ? *reinterpret_cast<const uint4*>(b_rows[q] + u * kBlock * 2) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const uint4 a[2] = {*reinterpret_cast<const uint4*>(a_rows[m][0] + u * kBlock * 2),
                              *reinterpret_cast<const uint4*>(a_rows[m][1] + u * kBlock * 2)};
#pragma unroll
          for (int q = 0; q < PARTS * NT; ++q) mma_block(part[m][q % NT], a, b[q]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->empty[at.stage]);
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (st.tokens >> (q * 8 + t * 2 + (j & 1)) & 1) total[m][q][j] += part[m][q][j];
    }
    at.next(st.rows + PARTS * n);
    if (++turn == kTeams) turn = 0;
  }

  // The warps' sums together: end(row, token, sum), all threads at once.
  template <typename End>
  __device__ __forceinline__ void finish(End&& end) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    float(*sums)[Sums<NT>::kTile] = sm->sums.v[tile++ & 1];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        float* to = sums[warp] + (q * 8 + 2 * t) * kColumn + 8 * m + g;
        to[0] = total[m][q][0], to[kColumn] = total[m][q][1], to[16] = total[m][q][2], to[kColumn + 16] = total[m][q][3];
      }
    sync_consumers();
#pragma unroll
    for (int q = 0; q < NT; ++q) {  // 32 rows of 8 tokens: a thread each
      const int row = lane, token = q * 8 + warp;
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += sums[w][token * kColumn + row];
      end(row, token, s);
    }
    clear();
  }

  __device__ __forceinline__ void tell() {
    if (fine) return;
    *status = MOE_E_TIMEOUT;
    *static_cast<volatile int*>(&sm->abort) = 1;
  }
};

// The router's logits: a block's share of its rows, each lane 8 columns at a time.
template <int NT>
__device__ __forceinline__ void logits(const Decode& p, Smem<NT>* sm, int e0, int e1) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int nkb = p.d / kBlock, b0 = share(nkb, warp, kWarps), b1 = share(nkb, warp + 1, kWarps);
  for (int e = e0; e < e1; e += 8) {  // rows 8 to 15 of the mma are not used
    float total[NT][4] = {};
    constexpr int U = 4;
    for (int kb = b0; kb < b1; kb += U) {
      uint4 a[U][2], b[U][NT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int col = (kb + u) * kBlock + t * 8;
        const bool there = kb + u < b1;
        a[u][1] = make_uint4(0, 0, 0, 0);
        a[u][0] = there && e + g < e1 ? load_weights(p.router_w + (size_t)(e + g) * p.d + col) : a[u][1];
#pragma unroll
        for (int n = 0; n < NT; ++n)
          b[u][n] = there && n * 8 + g < p.T ? __ldg(reinterpret_cast<const uint4*>(p.x + (size_t)(n * 8 + g) * p.d + col)) : a[u][1];
      }
      float part[NT][4] = {};
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_block(part[n], a[u], b[u][n]);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) total[n][j] += part[n][j];
    }
    float* mine = sm->sums.v[0][warp];
    sync_consumers();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) mine[(n * 8 + 2 * t + j) * kColumn + g] = total[n][j];
    sync_consumers();
    const int row = tid & 7, token = tid >> 3;
    if (token < p.T && e + row < e1) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += sm->sums.v[0][w][token * kColumn + row];
      p.logits[token * p.E + e + row] = s + (p.bias ? p.bias[e + row] : 0.f);
    }
  }
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 1) decode_layer(const __grid_constant__ Decode p) {
  extern __shared__ __align__(128) char smem_raw[];
  Smem<NT>* sm = reinterpret_cast<Smem<NT>*>(smem_raw);
  List* list = &sm->list;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int block = blockIdx.x, blocks = gridDim.x;
  const uint64_t deadline = moe::globaltimer() + kLimitNs;
  const bool producer = warp >= kWarps;
  if (tid < kStages) {
    moe::mbar_init(&sm->full[tid], kBringers + kBringers * 32);
    moe::mbar_init(&sm->empty[tid], kTeam);
    if (tid == 0) moe::mbar_init(&sm->h_ready, 1);
    moe::fence_mbar_init();
  }
  if (tid == 0) sm->abort = 0;
  bool fine = true;
  int gen = 0;
  if (!producer) {
    gen = tid == 0 ? moe::ld_acquire(&p.sched->gen) : 0;
    if (p.router_w) {  // 1: logits, and the choice
      logits<NT>(p, sm, share(p.E, block, blocks), share(p.E, block + 1, blocks));
      fine = grid_wait(p.sched, gen++, deadline, &list->ok);
      if (fine)
        for (int t = warp; t < p.T; t += kWarps) choose(p, list, t);
    } else {
      for (int i = tid; i < p.T * p.k; i += kConsumers) {
        list->idx[i / p.k][i % p.k] = p.idx_in[i];
        list->idx_w[i / p.k][i % p.k] = p.w_in[i];
      }
    }
    sync_consumers();
    if (fine) {
      if (block == 0 && p.router_w)
        for (int i = tid; i < p.T * p.k; i += kConsumers) {
          if (p.idx_out) p.idx_out[i] = list->idx[i / p.k][i % p.k];
          if (p.w_out) p.w_out[i] = list->idx_w[i / p.k][i % p.k];
        }
      make_list(p, list);
    }
    if (tid == 0 && !fine) sm->abort = 1;
  }
  __syncthreads();
  if (sm->abort) return;  // nothing is on its way yet

  const long long rows = (long long)list->n * p.f;
  GateUpTiles gate_up(p.f, share(rows, block, blocks), share(rows, block + 1, blocks));
  const int d0 = share(p.d, block, blocks), d1 = share(p.d, block + 1, blocks);
  const int down_tiles = (d1 - d0 + kRows - 1) / kRows;
  const int x_chunks = (p.d + kChunk - 1) / kChunk, f_chunks = (p.f + kChunk - 1) / kChunk;
  volatile int* abort = &sm->abort;
  const int n_list = list->n;

  if (producer) {
    Room<NT> room{sm, deadline};
    const int bringer = warp - kWarps;
    bool go = true;
    if (bringer < kBringers) {
      const int mine = lane * kBringers + bringer;  // the lane's row of a tile
      int issued = 0;
      // a stage: `row` is the lane's weight row at the chunk
      auto bring = [&](const Stage& st, const bf16* row) {
        const int rows = st.all();
        if (!room.make(rows)) return false;
        const bool there = mine < st.rows;
        const unsigned all = __ballot_sync(kAll, there);
        uint64_t* full = &sm->full[room.at.stage];
        moe::fence_proxy_async_shared();  // tokens' copies may have been in these rows before
        if (lane == 0) moe::mbar_arrive_expect_tx(full, (uint32_t)__popc(all) * st.columns * 2);
        __syncwarp();
        if (there) moe::bulk_load(sm->ring[room.at.at(mine)], row, (uint32_t)st.columns * 2, full);
        room.take(rows);
        ++issued;
        return true;
      };
      for (; go && gate_up.left > 0; gate_up.next()) {
        const int a = gate_up.entry, first = gate_up.first, n = gate_up.rows();
        const bf16* base = (mine < n ? p.gate : p.up) + ((size_t)list->expert[a] * p.f + first + (mine < n ? mine : mine - n)) * p.d;
        const int tokens = (int)list->tokens[a];
        for (int c = 0; go && c < x_chunks; ++c)
          go = bring(Stage{2 * n, tokens, 1, min(kChunk, p.d - c * kChunk)}, base + c * kChunk);
      }
      for (int i = 0; go && i < down_tiles; ++i) {
        const int first = d0 + i * kRows, n = min(kRows, d1 - first);
        for (int a = 0; go && a < n_list; ++a) {
          const bf16* base = p.down + ((size_t)list->expert[a] * p.d + first + mine) * p.f;
          const int tokens = (int)list->tokens[a];
          for (int c = 0; go && c < f_chunks; ++c)
            go = bring(Stage{n, tokens, 2, min(kChunk, p.f - c * kChunk)}, base + c * kChunk);
        }
      }
      // what is on its way arrives before the block ends, whatever became of the others
      const uint64_t last = moe::globaltimer() + kLimitNs;
      for (int i = max(0, issued - kStages); i < issued; ++i)
        moe::mbar_wait(&sm->full[i % kStages], (uint32_t)(i / kStages) & 1u, last);
      return;
    }
    // the tokens' columns: a warp brings a quarter of them, 16 bytes a lane, two rows at once
    constexpr int kPart = kChunk / kBringers, kLanes = kPart / 8;
    const int part = (bringer - kBringers) * kPart, sub = lane / kLanes, in_part = lane % kLanes * 8;
    // x's rows are the entry's tokens, h's its slots
    auto bring = [&](const Stage& st, const bf16* base, const bf16* base2, size_t stride, const uint8_t* order) {
      const int rows = st.all();
      if (!room.make(rows)) return false;
      const int n = __popc(st.tokens), all = rows - st.rows;
      if (part + in_part < st.columns) {
#pragma unroll 4
        for (int j = sub; j < all; j += 32 / kLanes) {
          const int slot = j < n ? j : j - n;
          const bf16* row = (j < n ? base : base2) + (size_t)(order ? order[slot] : slot) * stride;
          moe::cp_async16(sm->ring[room.at.at(st.rows + j)] + (part + in_part) * 2, row + part + in_part);
        }
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(moe::smem_u32(&sm->full[room.at.stage])) : "memory");
      room.take(rows);
      return true;
    };
    for (; go && gate_up.left > 0; gate_up.next()) {
      const int a = gate_up.entry, n = gate_up.rows();
      const int tokens = (int)list->tokens[a];
      for (int c = 0; go && c < x_chunks; ++c)
        go = bring(Stage{2 * n, tokens, 1, min(kChunk, p.d - c * kChunk)}, p.x + c * kChunk, nullptr, p.d, list->order[a]);
    }
    go = go && room.wait(&sm->h_ready, 0);
    for (int i = 0; go && i < down_tiles; ++i) {
      const int n = min(kRows, d1 - d0 - i * kRows);
      for (int a = 0; go && a < n_list; ++a) {
        const int tokens = (int)list->tokens[a];
        const size_t at = (size_t)list->start[a] * p.f;
        for (int c = 0; go && c < f_chunks; ++c)
          go = bring(Stage{n, tokens, 2, min(kChunk, p.f - c * kChunk)}, p.h_hi + at + c * kChunk, p.h_lo + at + c * kChunk,
                     p.f, nullptr);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }

  Consumer<NT> me{sm, deadline, &p.sched->status};
  me.clear();
  // 2: gate and up
  for (; gate_up.left > 0; gate_up.next()) {
    const int a = gate_up.entry, first = gate_up.first, n = gate_up.rows();
    const uint32_t tokens = list->tokens[a];
    for (int c = 0; c < x_chunks; ++c) me.template stage<1>(Stage{2 * n, (int)tokens, 1, min(kChunk, p.d - c * kChunk)}, n);
    me.finish([&](int row, int token, float s) {
      const float up = __shfl_xor_sync(kAll, s, 16);  // rows 16 to 31 are up's
      if (row >= n || !(tokens >> token & 1u)) return;
      const float h = s / (1.f + expf(-s)) * up * list->w[a][token];
      const size_t slot = list->start[a] + __popc(tokens & ((1u << token) - 1u));
      const bf16 hi = __float2bfloat16_rn(h);
      p.h_hi[slot * p.f + first + row] = hi;
      // an infinity or a NaN is all in the first part
      const float rest = h - __bfloat162float(hi);
      p.h_lo[slot * p.f + first + row] = __float2bfloat16_rn(isfinite(rest) ? rest : 0.f);
    });
  }
  me.tell();
  if (!grid_wait(p.sched, gen++, deadline, &list->ok) || *abort) {
    if (tid == 0) *abort = 1;
    return;
  }
  if (tid == 0) mbar_arrive(&sm->h_ready);

  // 3: down
  for (int r0 = d0; r0 < d1; r0 += kRows) {
    const int n = min(kRows, d1 - r0);
    for (int a = 0; a < n_list; ++a) {
      const int tokens = (int)list->tokens[a];
      for (int c = 0; c < f_chunks; ++c) me.template stage<2>(Stage{n, tokens, 2, min(kChunk, p.f - c * kChunk)}, 16);
    }
    me.finish([&](int row, int token, float s) {
      if (r0 + row < d1 && token < p.T) p.out[(size_t)token * p.d + r0 + row] = __float2bfloat16_rn(s);
    });
  }
  me.tell();
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
  return (int)sizeof(Smem<NT>);
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
