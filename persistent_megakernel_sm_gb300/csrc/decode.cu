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
// A product's tile is up to 32 weight rows (16 of gate and 16 of up) times 8 or 16
// token columns on mma.sync m16n8k16.  The tensor cores are nearly idle here; they are
// used because a multiply-add for every weight and token would not keep up with HBM.  A
// stage is 1024 columns of a tile and of the tokens that its expert has.  Four warps of
// a block bring its weights by bulk copies, four more the tokens' columns, into a ring
// of 86 single rows (182 KB an SM): two of gate and up's stages at least, of down's, with
// two rows for each token, one where many tokens meet a wide layer (16 tokens of width 7168:
// 24 + 32 rows).  The weights do not wait for the grid, so the ring is full of down's first
// ones when h' is complete.
// Eight warps multiply, each an eighth of a stage's columns, and their sums meet in
// shared memory once a tile.  A lane reads 16 bytes of a row at once, which the mma sees
// as another order of the same columns, the same for the tokens'.
//
// HBM bounds it: 4 tokens of 32 + 1 experts of 7168 x 2048 take 306 us (6.7 TB/s; a
// copy has 6.8), 4 of eight experts of 4096 x 14336 6.7 TB/s, 13 to 16 tokens 6.0 to 6.3.
// One token of 128 experts of 2048 x 768 (76 MB, 11 us) takes 25: the two waits of the
// grid 1.1 each, logits and choice 5, and streams that end before they are at speed.
//
// Down's columns are the tokens themselves.  A token that did not choose an expert has
// a zero column there and takes nothing from its sums, which are kept apart expert by
// expert, so an infinity or a NaN in weights that a token did not choose does not
// reach it.  Gate and up's, whose tile has one expert, are that expert's tokens.  Sums are fp32, over at most 128 columns in the tensor cores and from
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
constexpr int kBringers = 4;     // warps that bring weights, and as many that bring tokens
constexpr int kThreads = kConsumers + 2 * kBringers * 32;
constexpr int kBlock = 32;       // columns of two mma
constexpr int kRows = 32;        // of a tile: gate and up 16 each
constexpr int kColumn = 36;      // floats of a token's column of sums: 32, and 4 so that its lanes miss each other's banks
// Columns of a stage.  A stage costs the warps that bring and use it several hundred
// cycles whatever it holds, so longer is better: 4 tokens of 128 experts of 2048 x 768
// 76 us with 512, 65 with 1024, 16 tokens 196 and 159.
constexpr int kChunk = 1024;
constexpr int kBlocks = kChunk / kBlock / kWarps;  // of a warp
constexpr int kPitch = kChunk * 2 + 64;  // bytes of a row: two rows next to each other use all banks
constexpr int kRing = 86;        // rows of the ring: 182 KB
constexpr int kStages = 16;      // on their way, at most
constexpr unsigned kAll = 0xffffffffu;
constexpr uint64_t kLimitNs = 2000000000ull;  // of a pass's waits, where no option says otherwise
constexpr uint64_t kDrainNs = 2000000000ull;  // for copies on their way to arrive

// A wait that runs out leaves `arrived` off a whole number of grids, and the next wait
// would be let through early: so a pass that finds a status does nothing, until
// moe_decode_status clears both.
struct Sched {
  unsigned long long arrived;  // blocks, at all waits since it was cleared
  int status;
};

struct Decode {
  int T, d, f, E, k, S;
  int drop;            // test only: the wait (0: for the logits, 1: for h) at which block 0 does not arrive; -1: none
  uint64_t limit_ns;   // of the waits
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
  int start[kMaxE + 1];             // of its slots
  uint32_t tokens[kMaxE + 1];       // that chose it
  uint8_t order[kMaxE + 1][kMaxT];  // the same, one after another
  uint32_t by_expert[kMaxE];        // tokens, of every routed expert
  float w[kMaxE + 1][kMaxT];        // their weights, of every expert
  int warp_experts[kWarps], warp_slots[kWarps];
  int chosen[kWarps][kMaxK];
  float logit[kWarps][kMaxK];
  int ok;                           // of the last grid-wide wait
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

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(moe::smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void sync_consumers() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory"); }

// Every block's consumers arrive; false if the wait ran out somewhere, or if an earlier
// pass left a `status`.  `target` (of thread 0, as the status): the arrivals that make it
// complete.
__device__ bool grid_wait(Sched* s, unsigned long long target, uint64_t deadline, bool arrive, int status, int* ok) {
  sync_consumers();
  if (threadIdx.x == 0) {
    int fine = status == 0;
    if (fine && arrive) asm volatile("red.release.gpu.global.add.u64 [%0], 1;" ::"l"(&s->arrived) : "memory");
    unsigned long long now;
    for (int i = 0; fine; ++i) {
      asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(now) : "l"(&s->arrived) : "memory");
      if (now >= target) break;
      if (i % 16 == 15 && (moe::ld_relaxed(&s->status) != 0 || moe::globaltimer() > deadline)) {
        s->status = MOE_E_TIMEOUT;
        fine = 0;
        break;
      }
    }
    *ok = fine;
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
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}

// The larger first.
__device__ __forceinline__ void order_two(uint64_t& a, uint64_t& b) {
  const bool swap = a < b;
  const uint64_t hi = swap ? b : a;
  b = swap ? a : b;
  a = hi;
}

// A warp chooses for token t from its logits: the k largest, the lower expert on
// ties, their weights exp(l - max) over the kept ones' sum.  Lane j gets slot j.  A
// lane puts its PER experts in order once, so that each choice waits for no more than
// the lanes' first ones' largest and who has it.
template <int PER>
__device__ __forceinline__ void choose(const Decode& p, List* list, int t, int* expert, float* weight) {
  const int lane = threadIdx.x & 31;
  int* chosen = list->chosen[threadIdx.x >> 5];
  float* logit = list->logit[threadIdx.x >> 5];
  uint64_t key[PER + 1];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t k = lane * PER + i < p.E ? key_of(__ldcg(p.logits + t * p.E + lane * PER + i)) : 0u;
    key[i] = (uint64_t)k << 32 | (uint32_t)(PER - 1 - i);
  }
  key[PER] = 0;
#pragma unroll
  for (int round = 0; round < PER; ++round)  // neighbours, PER rounds
#pragma unroll
    for (int i = round & 1; i + 1 < PER; i += 2) order_two(key[i], key[i + 1]);
  if (lane < p.k) chosen[lane] = -1;
  __syncwarp();
  for (int j = 0; j < p.k; ++j) {
    const uint32_t best = (uint32_t)(key[0] >> 32);
    const uint32_t most = __reduce_max_sync(kAll, best);
    if (most <= kDead) break;
    if (lane == __ffs(__ballot_sync(kAll, best == most)) - 1) {
      chosen[j] = lane * PER + PER - 1 - (int)(uint32_t)key[0];
      logit[j] = value_of(most);
#pragma unroll
      for (int i = 0; i < PER; ++i) key[i] = key[i + 1];
    }
  }
  __syncwarp();
  const int my_e = lane < p.k ? chosen[lane] : -1;
  const float mine = my_e < 0 ? -INFINITY : logit[lane];
  // the first is the largest (a NaN, if there is one); equal logits weigh the same, infinities too
  const float top = __shfl_sync(kAll, mine, 0);
  const float e = my_e < 0 ? 0.f : mine == top ? 1.f : expf(mine - top);
  float sum = e;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  *expert = my_e;
  *weight = my_e < 0 ? 0.f : e / sum;
  __syncwarp();
}

// Lane j's slot of token t into the lists by expert.
__device__ __forceinline__ void enter(const Decode& p, List* list, int t, int e, float w) {
  const bool live = (threadIdx.x & 31) < p.k && (unsigned)e < (unsigned)p.E;
  if (!p.router_w) {  // an expert that the caller named twice has both weights, in slot order
    const int mine = live ? e : -1 - (int)(threadIdx.x & 31);
    float sum = 0.f;
    for (int j = 0; j < p.k; ++j) {
      const float v = __shfl_sync(kAll, w, j);
      if (__shfl_sync(kAll, mine, j) == mine) sum += v;
    }
    w = sum;
  }
  if (live) {
    atomicOr(&list->by_expert[e], 1u << t);
    list->w[e][t] = w;
  }
}

// The experts that the tokens chose, in order, from the lists by expert: a thread each.
__device__ __forceinline__ void make_list(const Decode& p, List* list) {
  static_assert(kMaxE <= kConsumers, "a thread an expert");
  const int e = threadIdx.x, lane = e & 31, warp = e >> 5;
  const uint32_t tokens = e < p.E ? list->by_expert[e] : 0u;
  const unsigned live = __ballot_sync(kAll, tokens != 0);
  const int mine = __popc(tokens);
  int sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kAll, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) list->warp_experts[warp] = __popc(live), list->warp_slots[warp] = sum;
  sync_consumers();
  int n = 0, slots = 0, n_all = 0, slots_all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int a = list->warp_experts[w], b = list->warp_slots[w];
    if (w < warp) n += a, slots += b;
    n_all += a, slots_all += b;
  }
  auto put = [&](int at, int expert, int start, uint32_t of) {
    list->expert[at] = expert, list->start[at] = start, list->tokens[at] = of;
    int j = 0;
    for (uint32_t left = of; left; left &= left - 1) list->order[at][j++] = (uint8_t)(__ffs(left) - 1);
  };
  if (tokens) put(n + __popc(live & ((1u << lane) - 1u)), e, slots + sum - mine, tokens);
  if (e == 0) {
    list->n = n_all + p.S;
    if (p.S) put(n_all, p.E, slots_all, (1u << p.T) - 1u);
  }
}

// Warps' sums of a tile; with 8 tokens two tiles' worth, so that one wait a tile is
// enough.
template <int NT>
struct Sums {
  static constexpr int kTile = NT * 8 * kColumn, kTiles = NT == 1 ? 2 : 1;
  float v[kTiles][kWarps][kTile];
};

template <int NT>
struct Smem {
  char ring[kRing][kPitch];
  Sums<NT> sums;
  List list;
  uint64_t full[kStages], empty[kStages], h_ready;
  int abort;  // a wait ran out: nothing more is brought
};

// Where one side of the ring stands: the stage's barriers and its first row.
struct At {
  int stage = 0, row = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int rows) {
    if (++stage == kStages) stage = 0, parity ^= 1;
    row += rows;
    if (row >= kRing) row -= kRing;
  }
  __device__ __forceinline__ int at(int i) const { return row + i >= kRing ? row + i - kRing : row + i; }
};

// A bringing warp's view of what is free: a stage's rows are the consumers' until its
// `empty` completes.
template <int NT>
struct Room {
  Smem<NT>* sm;
  uint64_t deadline;
  At at;        // of the next stage
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
    while (used + rows > kRing || out == kStages) {
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

__device__ __forceinline__ int share(long long total, int part, int parts) { return (int)(total * part / parts); }

// A block's share of the experts' f rows, tile by tile: at most 16 (of gate and of
// up), none over an expert's end.  Every block has its part of the shared expert's
// rows, first, and of the others' together: the shared expert's stages hold all
// tokens, and blocks that had nothing else would keep the grid waiting.  Stepped along:
// a division a tile in every warp, a stage even, is what the kernel then waits for.
struct GateUpTiles {
  const List* list;
  int f, left, later;  // rows still to come, with this tile's; of the other experts behind the shared one's
  int entry, first;    // of the list, first row there
  int later_entry, later_first;
  __device__ __forceinline__ GateUpTiles(const List* l, int f_, int shared, int block, int blocks) : list(l), f(f_) {
    const int routed = l->n - shared;
    const int r0 = share((long long)routed * f, block, blocks), r1 = share((long long)routed * f, block + 1, blocks);
    left = r1 - r0, entry = r0 / f, first = r0 % f;
    later = 0;
    if (shared) {
      later = left, later_entry = entry, later_first = first;
      first = share(f, block, blocks), left = share(f, block + 1, blocks) - first, entry = routed;
      if (left == 0) other();
    }
  }
  __device__ __forceinline__ void other() { left = later, entry = later_entry, first = later_first, later = 0; }
  // with more tokens fewer rows, so that two stages still fit into the ring
  __device__ __forceinline__ int rows() const { return min(min(__popc(list->tokens[entry]) > 11 ? 12 : 16, left), f - first); }
  __device__ __forceinline__ void next() {
    const int n = rows();
    left -= n, first += n;
    if (left == 0 && later > 0) other();
    else if (first == f) ++entry, first = 0;
  }
};


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
  At at;
  int tile = 0;  // tiles so far
  bool fine = true;
  float total[NT][2][4];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) total[q][m][j] = 0.f;
  }

  // 8 tokens' columns of a stage times M times 16 of its rows: 0 to 7 and 8 to 15 more
  // of the mma are rows 8 m and hi + 8 m on.  Sums of their own for both mma of a block
  // and both parts: one after another they would wait for each other.
  template <int PARTS, int M>
  __device__ __forceinline__ void multiply(const Stage& st, int hi, int tokens_before, uint32_t tokens, int n, float (&sum)[2][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int in_row = t * 16 + threadIdx.x / 32 * (kBlocks * kBlock * 2);
    const char* b_rows[PARTS];
    const bool on = tokens >> g & 1;
#pragma unroll
    for (int q = 0; q < PARTS; ++q)
      b_rows[q] = sm->ring[at.at(st.rows + q * n + tokens_before + (on ? __popc(tokens & ((1u << g) - 1u)) : 0))] + in_row;
    float part[M][PARTS][2][4] = {};
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
      uint4 b[PARTS];
#pragma unroll
      for (int q = 0; q < PARTS; ++q) {
        b[q] = *reinterpret_cast<const uint4*>(b_rows[q] + u * kBlock * 2);
        if (!on) b[q] = make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const uint4 a0 = *reinterpret_cast<const uint4*>(sm->ring[at.at(8 * m + g)] + in_row + u * kBlock * 2);
        const uint4 a1 = *reinterpret_cast<const uint4*>(sm->ring[at.at(hi + 8 * m + g)] + in_row + u * kBlock * 2);
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
          mma(part[m][q][0], a0.x, a1.x, a0.y, a1.y, b[q].x, b[q].y);
          mma(part[m][q][1], a0.z, a1.z, a0.w, a1.w, b[q].z, b[q].w);
        }
      }
    }
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float s = part[m][0][0][j] + part[m][0][1][j];
        if (PARTS == 2) s += part[m][PARTS - 1][0][j] + part[m][PARTS - 1][1][j];
        if (tokens >> (t * 2 + (j & 1)) & 1) sum[m][j] += s;
      }
  }

  // One stage, M as in multiply.  Columns are the tokens, or (a product of one part, whose
  // tile has one expert) those of them that are there, one after another.
  template <int PARTS, int M>
  __device__ __forceinline__ void stage(const Stage& st, int hi) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = __popc(st.tokens);
    fine = fine && moe::mbar_wait(&sm->full[at.stage], at.parity, deadline);
    if (warp * (kBlocks * kBlock) < st.columns) {  // a warp's 128 columns are all there or none
      int before = 0;
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        const uint32_t tokens = (PARTS == 1 ? (1u << n) - 1u : (uint32_t)st.tokens) >> (8 * q) & 0xffu;
        if (NT == 1 || tokens) multiply<PARTS, M>(st, hi, before, tokens, n, total[q]);
        before += __popc(tokens);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm->empty[at.stage]);
    at.next(st.rows + PARTS * n);
  }

  // The warps' sums together: end(row, column, sum), all threads at once.
  template <typename End>
  __device__ __forceinline__ void finish(End&& end) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    float(*sums)[Sums<NT>::kTile] = sm->sums.v[tile++ % Sums<NT>::kTiles];
    if (Sums<NT>::kTiles == 1) sync_consumers();  // the last tile's have been read
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        float* to = sums[warp] + (q * 8 + 2 * t) * kColumn + 8 * m + g;
        to[0] = total[q][m][0], to[kColumn] = total[q][m][1], to[16] = total[q][m][2], to[kColumn + 16] = total[q][m][3];
      }
    sync_consumers();
#pragma unroll
    for (int q = 0; q < NT; ++q) {  // 32 rows of 8 tokens: a thread each
      const int row = lane, column = q * 8 + warp;
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += sums[w][column * kColumn + row];
      end(row, column, s);
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
  const int nkb = p.d / kBlock, b0 = share(nkb, warp, kThreads / 32), b1 = share(nkb, warp + 1, kThreads / 32);
  for (int e = e0; e < e1; e += 8) {  // rows 8 to 15 of the mma are not used
    float total[NT][4] = {};
    constexpr int U = NT == 1 ? 8 : 4;
    for (int kb = b0; kb < b1; kb += U) {
      uint4 a[U], b[U][NT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int col = (kb + u) * kBlock + t * 8;
        const bool there = kb + u < b1;
        a[u] = there && e + g < e1 ? load_weights(p.router_w + (size_t)(e + g) * p.d + col) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          b[u][n] = there && n * 8 + g < p.T ? __ldg(reinterpret_cast<const uint4*>(p.x + (size_t)(n * 8 + g) * p.d + col)) : make_uint4(0, 0, 0, 0);
      }
      float part[NT][2][4] = {};
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma(part[n][0], a[u].x, 0, a[u].y, 0, b[u][n].x, b[u][n].y);
          mma(part[n][1], a[u].z, 0, a[u].w, 0, b[u][n].z, b[u][n].w);
        }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) total[n][j] += part[n][0][j] + part[n][1][j];
    }
    float* all = reinterpret_cast<float*>(sm->ring);  // nothing is on its way yet
    float* mine = all + warp * Sums<NT>::kTile;
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) mine[(n * 8 + 2 * t + j) * kColumn + g] = total[n][j];
    __syncthreads();
    const int row = tid & 7, token = tid >> 3;
    if (token < p.T && e + row < e1) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) s += all[w * Sums<NT>::kTile + token * kColumn + row];
      const float b = p.bias ? p.bias[e + row] : 0.f;
      p.logits[token * p.E + e + row] = b == -INFINITY ? b : s + b;  // masked beside a NaN or an infinity too
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
  const uint64_t deadline = moe::globaltimer() + p.limit_ns;
  const bool producer = warp >= kWarps;
  if (tid < kStages) {
    moe::mbar_init(&sm->full[tid], kBringers + kBringers * 32);
    moe::mbar_init(&sm->empty[tid], kWarps);
    if (tid == 0) moe::mbar_init(&sm->h_ready, 1);
    moe::fence_mbar_init();
  }
  if (tid == 0) sm->abort = 0;
  if (tid < p.E) list->by_expert[tid] = 0;
  if (tid < p.T) list->w[p.E][tid] = 1.f;  // the shared expert's
  // arrivals before this pass: a whole number of grids, and maybe others' first ones of this pass
  unsigned long long target = 0;
  int status = 0;  // that an earlier pass left
  if (tid == 0) {
    target = *static_cast<volatile unsigned long long*>(&p.sched->arrived);
    status = *static_cast<volatile int*>(&p.sched->status);
    target = target / blocks * blocks;
  }
  // 1: logits, and the choice
  if (p.router_w) logits<NT>(p, sm, share(p.E, block, blocks), share(p.E, block + 1, blocks));
  if (!producer) {
    bool fine;
    if (p.router_w) {
      fine = grid_wait(p.sched, target += blocks, deadline, block != 0 || p.drop != 0, status, &list->ok);
    } else {
      if (tid == 0) list->ok = status == 0;
      sync_consumers();
      fine = list->ok != 0;
    }
    if (fine) {
      for (int t = warp; t < p.T; t += kWarps) {
        int e = -1;
        float w = 0.f;
        if (p.router_w) {
          if (p.E <= 128) choose<4>(p, list, t, &e, &w);
          else choose<8>(p, list, t, &e, &w);
        } else if (lane < p.k) e = p.idx_in[t * p.k + lane], w = p.w_in[t * p.k + lane];
        enter(p, list, t, e, w);
        if (block == 0 && lane < p.k && p.router_w) {
          if (p.idx_out) p.idx_out[t * p.k + lane] = e;
          if (p.w_out) p.w_out[t * p.k + lane] = w;
        }
      }
      sync_consumers();
      make_list(p, list);
    }
    if (tid == 0 && !fine) sm->abort = 1;
  }
  __syncthreads();
  if (sm->abort) return;  // nothing is on its way yet

  GateUpTiles gate_up(list, p.f, p.S, block, blocks);
  const int d0 = share(p.d, block, blocks), d1 = share(p.d, block + 1, blocks);
  const int down_tiles = (d1 - d0 + kRows - 1) / kRows, down_rows = (d1 - d0 + down_tiles - 1) / max(1, down_tiles);
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
        const int first = d0 + i * down_rows, n = min(down_rows, d1 - first);
        for (int a = 0; go && a < n_list; ++a) {
          const bf16* base = p.down + ((size_t)list->expert[a] * p.d + first + mine) * p.f;
          const int tokens = (int)list->tokens[a];
          for (int c = 0; go && c < f_chunks; ++c)
            go = bring(Stage{n, tokens, 2, min(kChunk, p.f - c * kChunk)}, base + c * kChunk);
        }
      }
      // what is on its way arrives before the block ends, whatever became of the others
      const uint64_t last = moe::globaltimer() + kDrainNs;
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
      const int n = min(down_rows, d1 - d0 - i * down_rows);
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
    const int a = gate_up.entry, first = gate_up.first, n = gate_up.rows(), expert = list->expert[a];
    const uint32_t tokens = list->tokens[a];
    for (int c = 0; c < x_chunks; ++c) {
      const Stage st{2 * n, (int)tokens, 1, min(kChunk, p.d - c * kChunk)};
      if (n > 8) me.template stage<1, 2>(st, n);
      else me.template stage<1, 1>(st, n);
    }
    me.finish([&](int row, int column, float s) {
      const float up = __shfl_xor_sync(kAll, s, 16);  // rows 16 to 31 are up's
      if (row >= n || column >= __popc(tokens)) return;
      const float h = s / (1.f + expf(-s)) * up * list->w[expert][list->order[a][column]];
      const size_t slot = list->start[a] + column;
      const bf16 hi = __float2bfloat16_rn(h);
      p.h_hi[slot * p.f + first + row] = hi;
      // an infinity or a NaN is all in the first part
      const float rest = h - __bfloat162float(hi);
      p.h_lo[slot * p.f + first + row] = __float2bfloat16_rn(isfinite(rest) ? rest : 0.f);
    });
  }
  me.tell();
  if (!grid_wait(p.sched, target += blocks, deadline, block != 0 || p.drop != 1, 0, &list->ok) || *abort) {
    if (tid == 0) *abort = 1;
    return;
  }
  if (tid == 0) mbar_arrive(&sm->h_ready);

  // 3: down
  for (int r0 = d0; r0 < d1; r0 += down_rows) {
    const int n = min(down_rows, d1 - r0);
    for (int a = 0; a < n_list; ++a) {
      const int tokens = (int)list->tokens[a];
      for (int c = 0; c < f_chunks; ++c) {
        const Stage st{n, tokens, 2, min(kChunk, p.f - c * kChunk)};
        if (n > 16) me.template stage<2, 2>(st, 16);
        else me.template stage<2, 1>(st, 8);
      }
    }
    me.finish([&](int row, int token, float s) {
      if (n <= 16) {  // the sums' rows 0 to 7 and 16 to 23 are the tile's first 16
        if (row & 8) return;
        row = (row & 7) + (row >> 4) * 8;
      }
      if (row < n && token < p.T) p.out[(size_t)token * p.d + r0 + row] = __float2bfloat16_rn(s);
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
  int T_max = 0, blocks = 0, device = -1, drop = -1;
  uint64_t limit_ns = kLimitNs;
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
  p.drop = h->drop, p.limit_ns = h->limit_ns;
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

int moe_decode_set_option(moe_decode_t* h, int key, long long v) {
  if (!h) return moe::set_error(MOE_E_INVAL, "null handle");
  switch (key) {
    case MOE_OPT_TIMEOUT_NS:
      if (v < 1000) return moe::set_error(MOE_E_INVAL, "timeout below 1 us");
      h->limit_ns = (uint64_t)v;
      break;
    case MOE_OPT_FAULT_DROP_TASK:
      if (v < -1 || v > 1) return moe::set_error(MOE_E_INVAL, "the waits are 0 and 1; -1: off");
      h->drop = (int)v;
      break;
    default:
      return moe::set_error(MOE_E_INVAL, "not an option of the layer for a few tokens");
  }
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
