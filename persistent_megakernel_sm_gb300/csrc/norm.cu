// The norms about a block: forward, and the handle (the formulas: norm.cuh).
#include "norm.cuh"

namespace {

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

// Rows team, team + teams, ... of the tensors.
// SAVE: 8-bit rows may be wanted; a kernel that cannot write them runs with fewer registers.
template <typename R, bool VEC, bool PRE_LAYER, int POST, int CH, bool SAVE>
__global__ void __launch_bounds__(kThreads, VEC && !SAVE ? 2 : 1) norm_forward(const __grid_constant__ Forward<R> f) {
  extern __shared__ __align__(16) char smem[];
  const Shape& a = f.a;
  Team team(smem + a.parts);
  const int tid = threadIdx.x, threads = blockDim.x, units = CH * threads;
  const int step = gridDim.x / team.blocks;
  float* warp_row = reinterpret_cast<float*>(smem + a.out) + (tid >> 5) * 256;
  const Kept kept{reinterpret_cast<float4*>(smem + a.vec), units};
  const float inv_d = 1.f / (float)a.d;
  int col[CH], n[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) col[c] = (team.rank * units + c * threads + tid) * 8, n[c] = max(0, min(8, a.d - col[c]));

  wait_for_previous_kernel();
  let_next_kernel_start();
  begin(a, team, smem, team.blocks * units * 8);
  auto start = [&](int t, char* slot) {
    if (t < a.T) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int unit = c * threads + tid;
        fetch<R, VEC>(slot + a.field[0], units, unit, f.residual.at(t), col[c], a.d);
        if (f.y.p) fetch<bf16, VEC>(slot + a.field[1], units, unit, f.y.at(t), col[c], a.d);
        if (f.gate_rows.p) fetch<bf16, VEC>(slot + a.field[2], units, unit, f.gate_rows.at(t), col[c], a.d);
      }
    }
    moe::cp_async_commit();
  };
  int t = blockIdx.x / team.blocks;
  for (int i = 0; i < a.stages; ++i) start(t + i * step, smem + i * a.stage);

  // 0: s g gain of the post norm, 1: the pre norm's gain, 2 and 3: their shifts
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int unit = c * threads + tid;
    const Eight gate = load_params(f.gate_columns, f.params_f32, col[c], n[c], 1.f, 0.f);
    auto with_gate = [&](Eight e) {
#pragma unroll
      for (int j = 0; j < 4; ++j) e.v[j] = mul2(e.v[j], mul2(gate.v[j], two(a.scale)));
      return e;
    };
    kept.write(0, unit, with_gate(load_params(f.post_gain, f.params_f32, col[c], n[c], 1.f, a.one)));
    kept.write(1, unit, load_params(f.pre_gain, f.params_f32, col[c], n[c], 1.f, a.one));
    if (POST == kLayer && f.post_shift) kept.write(2, unit, with_gate(load_params(f.post_shift, f.params_f32, col[c], n[c], 0.f, 0.f)));
    if (PRE_LAYER && f.pre_shift) kept.write(3, unit, load_params(f.pre_shift, f.params_f32, col[c], n[c], 0.f, 0.f));
  }
  auto param = [&](int which, int c) { return kept.read(which, c * threads + tid); };

  char* slot = smem;
#pragma unroll 1
  for (; t < a.T; t += step) {
    const float gate_t = f.gate_tokens ? __ldg(f.gate_tokens + t) : 1.f;
    wait_copies<VEC>(a.stages);
    Eight sum[CH];
    float2 post = make_float2(0.f, 1.f), pre = post;
#pragma unroll
    for (int c = 0; c < CH; ++c) sum[c] = read<R, VEC>(slot + a.field[0], units, c * threads + tid, f.residual.at(t), n[c]);
    if (f.y.p) {
      Eight y[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) y[c] = read<bf16, VEC>(slot + a.field[1], units, c * threads + tid, f.y.at(t), n[c]);
      if (POST != kNone) post = moments<POST == kLayer, CH>(team, y, n, inv_d, a.eps);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (SAVE && f.y8.codes) store_rows8<bf16, VEC>(f.y8, t, a, y[c], col[c], warp_row);
        const Eight k = param(0, c);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (POST == kLayer) y[c].v[j] = add2(y[c].v[j], two(-post.x));
          if (POST != kNone) y[c].v[j] = mul2(y[c].v[j], two(post.y));
          y[c].v[j] = mul2(y[c].v[j], k.v[j]);
        }
        if (POST == kLayer && f.post_shift) {
          const Eight b = param(2, c);
#pragma unroll
          for (int j = 0; j < 4; ++j) y[c].v[j] = add2(y[c].v[j], b.v[j]);
        }
        if (f.gate_rows.p) {
          const Eight g = read<bf16, VEC>(slot + a.field[2], units, c * threads + tid, f.gate_rows.at(t), n[c]);
#pragma unroll
          for (int j = 0; j < 4; ++j) y[c].v[j] = mul2(y[c].v[j], g.v[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[c].v[j] = fma2(y[c].v[j], two(gate_t), sum[c].v[j]);
        if (POST == kLayer && n[c] < 8) sum[c].cut(n[c]);  // 0 - mean behind the row's end
        if constexpr (sizeof(R) == 2) {
          const uint4 q = pack(sum[c]);
          store_row<VEC>(f.out.at(t), q, col[c], a.d, warp_row);
          uint32_t w[4];
          put_words(q, w);
          sum[c] = unpack(w);
        } else {
          store_row<VEC>(f.out.at(t), sum[c], col[c], a.d, warp_row);
        }
      }
    }
    if (f.norm.p) pre = moments<PRE_LAYER, CH>(team, sum, n, inv_d, a.eps);
    if (!VEC) __syncwarp();
    start(t + a.stages * step, slot);  // all of the row has been read
    slot += a.stage;
    if (slot == smem + a.vec) slot = smem;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (SAVE && f.out8.codes) store_rows8<R, VEC>(f.out8, t, a, sum[c], col[c], warp_row);
      if (!f.norm.p) continue;
      const Eight gain = param(1, c);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (PRE_LAYER) sum[c].v[j] = add2(sum[c].v[j], two(-pre.x));
        sum[c].v[j] = mul2(mul2(sum[c].v[j], two(pre.y)), gain.v[j]);
      }
      if (PRE_LAYER && f.pre_shift) {
        const Eight shift = param(3, c);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[c].v[j] = add2(sum[c].v[j], shift.v[j]);
      }
      store_row<VEC>(f.norm.at(t), sum[c], col[c], a.d, warp_row);
    }
    if (f.stats && team.rank == 0 && tid == 0) f.stats[t] = make_float4(post.x, post.y, pre.x, pre.y);
  }
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
  if (T < 0 || T > kMaxT) return moe::set_error(MOE_E_INVAL, "T must be in 0..2^30");
  if (residual_type != MOE_TYPE_F32 && residual_type != MOE_TYPE_BF16)
    return moe::set_error(MOE_E_INVAL, "the residual is MOE_TYPE_F32 or MOE_TYPE_BF16");
  const char* bad = check_params(h, params, T);
  if (!bad) bad = check_rows8(out8, T);
  if (!bad) bad = check_rows8(y8, T);
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
    const int bytes[5] = {(int)sizeof(R) * 8, y ? 16 : 0, f.gate_rows.p ? 16 : 0, 0, 0};
    const Plan p = lay_out(&f.a, vec ? chunks_of(h->d, T, 2) : 1, kThreads, vec && !out8 && !y8 ? 2 * kThreads : kThreads, bytes,
                           f.pre_shift ? 4 : f.post_shift ? 3 : 2, 1, vec);
    const int teams = std::min(T, kSms * p.per_sm / p.blocks);
    return by_kind(h, vec, p.chunks, [&](auto v, auto layer, auto post, auto c) {
      constexpr bool VEC = decltype(v)::value, LAYER = decltype(layer)::value;
      constexpr int POST = decltype(post)::value, CH = decltype(c)::value;
      auto with = [&](auto s) {
        constexpr bool SAVE = decltype(s)::value;
        auto* kernel = norm_forward<R, VEC, LAYER, POST, CH, SAVE>;
        cudaError_t e = allow_smem<ForwardKernel<R, VEC, LAYER, POST, CH, SAVE>>(kernel);
        return e == cudaSuccess ? launch(kernel, (unsigned)(teams * p.blocks), p.blocks, p.threads, p.smem,
                                         static_cast<cudaStream_t>(stream), f) : e;
      };
      return out8 || y8 ? with(std::true_type{}) : with(std::false_type{});
    });
  };
  const cudaError_t e = residual_type == MOE_TYPE_F32 ? go(0.f) : go(bf16());
  return e == cudaSuccess ? MOE_OK : moe::set_cuda_error(e, "norm_forward");
}

}  // extern "C"
