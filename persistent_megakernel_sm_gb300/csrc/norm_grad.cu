// The norms about a block: the gradient (the formulas: norm.cuh).
#include "norm.cuh"

namespace {

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

// The sums of a row, in the order in which they are reduced, of G' = grad_out + rstd t,
// x = u of the pre norm, v = u gain g of the post norm, w = gain g, b its shift.
enum { kTU, kUV, kXV, kT, kV, kUW, kXW, kW, kUB, kXB, kB, kSums };

// Fours of them that a row has: kTU, kUV and kXV, with layer norms up to all.
__host__ __device__ constexpr int quads_of(bool pre_layer, int post) { return pre_layer || post == kLayer ? 3 : 1; }

// What a thread keeps from row to row, the sums over rows, takes most of its registers:
// a row is read from its slots again once its sums are known.
template <typename R, bool VEC, bool PRE_LAYER, int POST, int CH>
__global__ void __launch_bounds__(kThreads) norm_backward(const __grid_constant__ Backward<R> f) {
  extern __shared__ __align__(16) char smem[];
  constexpr int quads = quads_of(PRE_LAYER, POST);
  constexpr bool POST_LAYER = POST == kLayer;
  const Shape& a = f.a;
  Team team(smem + a.parts);
  const int tid = threadIdx.x, threads = blockDim.x, units = CH * threads;
  const int first = blockIdx.x / team.blocks, step = gridDim.x / team.blocks;
  float* warp_row = reinterpret_cast<float*>(smem + a.out) + (tid >> 5) * 256;
  const Kept kept{reinterpret_cast<float4*>(smem + a.vec), units};
  const float inv_d = 1.f / (float)a.d;
  int cols[CH], ns[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) cols[c] = (team.rank * units + c * threads + tid) * 8, ns[c] = max(0, min(8, a.d - cols[c]));
  const bool has_y = f.y.p || f.y8.codes, has_norm = f.grad_norm.p != nullptr;
  const bool token_shift = POST_LAYER && f.grad_gate_tokens && f.post_shift;

  wait_for_previous_kernel();
  let_next_kernel_start();
  begin(a, team, smem, team.blocks * units * 8);
  auto start = [&](int t, char* slot) {
    if (t < a.T) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int unit = c * threads + tid, col = cols[c];
        if (f.grad_out.p) fetch<R, VEC>(slot + a.field[0], units, unit, f.grad_out.at(t), col, a.d);
        if (has_norm) {
          fetch<bf16, VEC>(slot + a.field[1], units, unit, f.grad_norm.at(t), col, a.d);
          if (f.out8.codes) fetch8<VEC>(slot + a.field[2], units, unit, f.out8, t, a, col);
          else fetch<R, VEC>(slot + a.field[2], units, unit, f.kept_out.at(t), col, a.d);
        }
        if (f.y8.codes) fetch8<VEC>(slot + a.field[3], units, unit, f.y8, t, a, col);
        else if (f.y.p) fetch<bf16, VEC>(slot + a.field[3], units, unit, f.y.at(t), col, a.d);
        if (f.gate_rows.p) fetch<bf16, VEC>(slot + a.field[4], units, unit, f.gate_rows.at(t), col, a.d);
      }
    }
    moe::cp_async_commit();
  };
  for (int i = 0; i < a.stages; ++i) start(first + i * step, smem + i * a.stage);

#pragma unroll
  for (int c = 0; c < CH; ++c) {  // 0: the pre norm's gain, 1: the post norm's with the gate's columns, 2: its shift
    const int unit = c * threads + tid, col = cols[c], n = ns[c];
    kept.write(0, unit, load_params(f.pre_gain, f.params_f32, col, n, 1.f, a.one));
    Eight w = load_params(f.post_gain, f.params_f32, col, n, 1.f, a.one);
    const Eight gate = load_params(f.gate_columns, f.params_f32, col, n, 1.f, 0.f);
#pragma unroll
    for (int j = 0; j < 4; ++j) w.v[j] = mul2(w.v[j], gate.v[j]);
    kept.write(1, unit, w);
    if (POST_LAYER && f.post_shift) kept.write(2, unit, load_params(f.post_shift, f.params_f32, col, n, 0.f, 0.f));
  }

  // u of the pre norm, and of the post norm (y itself where there is none)
  auto read_x = [&](const char* slot, int t, const float4& st, int c) {
    const int unit = c * threads + tid, col = cols[c], n = ns[c];
    Eight x = f.out8.codes ? read8<VEC>(slot + a.field[2], units, unit, f.out8, t, a, col, n)
                           : read<R, VEC>(slot + a.field[2], units, unit, f.kept_out.at(t), n);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (PRE_LAYER) x.v[j] = add2(x.v[j], two(-st.z));
      x.v[j] = mul2(x.v[j], two(st.w));
    }
    if (PRE_LAYER && n < 8) x.cut(n);  // 0 - mean behind the row's end
    return x;
  };
  auto read_y = [&](const char* slot, int t, const float4& st, int c) {
    const int unit = c * threads + tid, col = cols[c], n = ns[c];
    Eight y = f.y8.codes ? read8<VEC>(slot + a.field[3], units, unit, f.y8, t, a, col, n)
                         : read<bf16, VEC>(slot + a.field[3], units, unit, f.y.at(t), n);
    if (POST != kNone) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (POST_LAYER) y.v[j] = add2(y.v[j], two(-st.x));
        y.v[j] = mul2(y.v[j], two(st.y));
      }
      if (POST_LAYER && n < 8) y.cut(n);
    }
    return y;
  };
  const Eight nothing{};

  Eight acc_tu[CH]{}, acc_t[PRE_LAYER ? CH : 1]{}, acc_v[CH]{}, acc_g[POST_LAYER ? CH : 1]{};
  const bool sums_post = has_y && (POST != kNone || f.grad_gate_tokens);
  char* slot = smem;
  const float4 no_norms = make_float4(0.f, 1.f, 0.f, 1.f);
  // a row's numbers, a row ahead
  float4 st_next = f.stats && first < a.T ? __ldg(f.stats + first) : no_norms;
  float gate_next = f.gate_tokens && first < a.T ? __ldg(f.gate_tokens + first) : 1.f;
#pragma unroll 1
  for (int t = first; t < a.T; t += step) {
    const float4 st = st_next;
    const float gate_t = gate_next;
    if (t + step < a.T) {
      if (f.stats) st_next = __ldg(f.stats + t + step);
      if (f.gate_tokens) gate_next = __ldg(f.gate_tokens + t + step);
    }
    wait_copies<VEC>(a.stages);
    float total[4 * quads];
    {
      float2 sum[4 * quads];
#pragma unroll
      for (int q = 0; q < 4 * quads; ++q) sum[q] = make_float2(0.f, 0.f);
      auto more = [&](int q, float2 p, float2 v) {
        if (q < 4 * quads) sum[q < 4 * quads ? q : 0] = fma2(p, v, sum[q < 4 * quads ? q : 0]);
      };
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int unit = c * threads + tid, n = ns[c];
        Eight go = f.grad_out.p ? read<R, VEC>(slot + a.field[0], units, unit, f.grad_out.at(t), n) : nothing, x = nothing;
        if (has_norm) {  // go: grad_out + rstd t
          x = read_x(slot, t, st, c);
          const Eight gn = read<bf16, VEC>(slot + a.field[1], units, unit, f.grad_norm.at(t), n), k = kept.read(0, unit);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 tj = mul2(gn.v[j], k.v[j]);
            more(kTU, tj, x.v[j]);
            if (PRE_LAYER) more(kT, tj, two(1.f));
            go.v[j] = fma2(tj, two(st.w), go.v[j]);
          }
        }
        if (sums_post) {
          Eight w = kept.read(1, unit);
          const Eight y = read_y(slot, t, st, c);
          if (f.gate_rows.p) {
            const Eight g = read<bf16, VEC>(slot + a.field[4], units, unit, f.gate_rows.at(t), n);
#pragma unroll
            for (int j = 0; j < 4; ++j) w.v[j] = mul2(w.v[j], g.v[j]);
          }
          if (PRE_LAYER && n < 8) w.cut(n);  // a gain of 1 behind the row's end
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 v = mul2(y.v[j], w.v[j]);
            more(kUV, go.v[j], v);
            more(kXV, x.v[j], v);
            if (PRE_LAYER) more(kV, v, two(1.f));
            if (POST_LAYER) {
              more(kUW, go.v[j], w.v[j]);
              more(kXW, x.v[j], w.v[j]);
              if (PRE_LAYER) more(kW, w.v[j], two(1.f));
            }
          }
          if (token_shift) {
            const Eight b = kept.read(2, unit);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              more(kUB, go.v[j], b.v[j]);
              more(kXB, x.v[j], b.v[j]);
              if (PRE_LAYER) more(kB, b.v[j], two(1.f));
            }
          }
        }
      }
      float4 v[quads];
#pragma unroll
      for (int q = 0; q < quads; ++q)
        v[q] = make_float4(sum[4 * q].x + sum[4 * q].y, sum[4 * q + 1].x + sum[4 * q + 1].y, sum[4 * q + 2].x + sum[4 * q + 2].y,
                           sum[4 * q + 3].x + sum[4 * q + 3].y);
      team.sum(v);
#pragma unroll
      for (int q = 0; q < quads; ++q) total[4 * q] = v[q].x, total[4 * q + 1] = v[q].y, total[4 * q + 2] = v[q].z, total[4 * q + 3] = v[q].w;
    }
    const float c1 = total[kTU] * inv_d, c2 = PRE_LAYER ? total[kT] * inv_d : 0.f;
    auto of = [&](int uv, int xv, int ones) {
      auto at = [&](int q) { return total[q < 4 * quads ? q : 0]; };
      return at(uv) - (has_norm ? st.w * (c1 * at(xv) + (PRE_LAYER ? c2 * at(ones) : 0.f)) : 0.f);
    };
    // sum of G v = sum of G' v - rstd (c2 sum of v + c1 sum of x v), and so on
    const float e1 = sums_post ? a.scale * of(kUV, kXV, kV) : 0.f;
    const float m1 = e1 * gate_t * inv_d, m2 = POST_LAYER ? a.scale * gate_t * of(kUW, kXW, kW) * inv_d : 0.f;
    if (f.grad_gate_tokens && team.rank == 0 && tid == 0)
      f.grad_gate_tokens[t] = e1 + (token_shift ? a.scale * of(kUB, kXB, kB) : 0.f);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int unit = c * threads + tid, col = cols[c], n = ns[c];
      Eight g = f.grad_out.p ? read<R, VEC>(slot + a.field[0], units, unit, f.grad_out.at(t), n) : nothing;
      if (has_norm) {
        const Eight x = read_x(slot, t, st, c);
        const Eight gn = read<bf16, VEC>(slot + a.field[1], units, unit, f.grad_norm.at(t), n), k = kept.read(0, unit);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc_tu[c].v[j] = fma2(gn.v[j], x.v[j], acc_tu[c].v[j]);
          if (PRE_LAYER) acc_t[PRE_LAYER ? c : 0].v[j] = add2(gn.v[j], acc_t[PRE_LAYER ? c : 0].v[j]);
          float2 v = fma2(x.v[j], two(-c1), mul2(gn.v[j], k.v[j]));
          if (PRE_LAYER) v = add2(v, two(-c2));
          g.v[j] = fma2(v, two(st.w), g.v[j]);
        }
      }
      if (f.grad_residual.p) store_row<VEC>(f.grad_residual.at(t), g, col, a.d, warp_row);
      if (has_y || f.grad_y.p) {
        const Eight w = kept.read(1, unit), y = has_y ? read_y(slot, t, st, c) : nothing;
#pragma unroll
        for (int j = 0; j < 4; ++j) g.v[j] = mul2(g.v[j], two(a.scale * gate_t));  // from here on s g G, but for the gates below
        if (f.gate_rows.p) {
          if (f.grad_gate_rows.p) {  // s G p
            Eight p;
#pragma unroll
            for (int j = 0; j < 4; ++j) p.v[j] = mul2(y.v[j], w.v[j]);
            if (POST_LAYER && f.post_shift) {
              const Eight b = kept.read(2, unit);
#pragma unroll
              for (int j = 0; j < 4; ++j) p.v[j] = add2(p.v[j], b.v[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) p.v[j] = mul2(p.v[j], g.v[j]);
            store_row<VEC>(f.grad_gate_rows.at(t), p, col, a.d, warp_row);
          }
          const Eight gate = read<bf16, VEC>(slot + a.field[4], units, unit, f.gate_rows.at(t), n);
#pragma unroll
          for (int j = 0; j < 4; ++j) g.v[j] = mul2(g.v[j], gate.v[j]);
        }
        // a gate of columns is put on the sums over rows, and its gradient taken from
        // them, at the end: here without it
        if (has_y) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc_v[c].v[j] = fma2(g.v[j], y.v[j], acc_v[c].v[j]);
            if (POST_LAYER) acc_g[POST_LAYER ? c : 0].v[j] = add2(g.v[j], acc_g[POST_LAYER ? c : 0].v[j]);
          }
        }
        if (f.grad_y.p) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            g.v[j] = mul2(g.v[j], w.v[j]);
            if (POST != kNone) {
              g.v[j] = fma2(y.v[j], two(-m1), g.v[j]);
              if (POST_LAYER) g.v[j] = add2(g.v[j], two(-m2));
              g.v[j] = mul2(g.v[j], two(st.y));
            }
          }
          store_row<VEC>(f.grad_y.at(t), g, col, a.d, warp_row);
        }
      }
    }
    if (!VEC) __syncwarp();
    start(t + a.stages * step, slot);
    slot += a.stage;
    if (slot == smem + a.vec) slot = smem;
  }

  if (!f.sums) return;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    float* to = f.sums + (long long)first * 4 * a.d + cols[c];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j >= ns[c]) break;
      to[j] = acc_tu[c].get(j);
      if (PRE_LAYER) to[a.d + j] = acc_t[PRE_LAYER ? c : 0].get(j);
      to[2 * a.d + j] = acc_v[c].get(j);
      if (POST_LAYER) to[3 * a.d + j] = acc_g[POST_LAYER ? c : 0].get(j);
    }
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
  const bool wanted[4] = {c.pre_gain_grad != nullptr, c.pre_layer && c.pre_shift_grad, c.post_gain_grad || c.gate_grad,
                          c.post_layer && (c.post_shift_grad || c.gate_grad)};
  float v[4] = {};
  if (col < c.d) {
    for (int t0 = warp; t0 < c.teams; t0 += 32 * 5) {  // five teams' at once: 160 are all that SMs of one block have
      float x[4][5];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 5; ++i)
          x[q][i] = wanted[q] && t0 + 32 * i < c.teams ? __ldcg(c.sums + ((long long)(t0 + 32 * i) * 4 + q) * c.d + col) : 0.f;
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 5; ++i) v[q] += x[q][i];
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

}  // namespace

extern "C" {

int moe_norm_backward(const moe_norm_t* h, int T, int residual_type, const void* grad_out, long long grad_out_stride,
                      const void* grad_norm, long long grad_norm_stride, const moe_norm_params* params,
                      const moe_norm_kept* kept, void* grad_residual, long long grad_residual_stride, void* grad_y,
                      long long grad_y_stride, const moe_norm_grads* grads, void* stream) {
  if (!h) return moe::set_error(MOE_E_INVAL, "null handle");
  if (T < 0 || T > kMaxT) return moe::set_error(MOE_E_INVAL, "T must be in 0..2^30");
  if (residual_type != MOE_TYPE_F32 && residual_type != MOE_TYPE_BF16)
    return moe::set_error(MOE_E_INVAL, "the residual is MOE_TYPE_F32 or MOE_TYPE_BF16");
  if (!kept || !grads) return moe::set_error(MOE_E_INVAL, "null kept or grads");
  const char* bad = check_params(h, params, T);
  if (!bad) bad = check_rows8(kept->out8, T);
  if (!bad) bad = check_rows8(kept->y8, T);
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
  // with a post norm these go through it
  const bool through_post = h->post != kNone && (grad_y || g.post_gain || g.post_shift || g.gate);
  if (!grad_out && !grad_norm) bad = "no gradient to start from";
  else if (has_norm && h->pre == kNone) bad = "the gradient of a norm that the handle does not have";
  else if (!has_norm && (g.pre_gain || g.pre_shift)) bad = "gradients of the pre norm need that of its output";
  else if (kept->out && kept->out8) bad = "out is kept in one form";
  else if (kept->y && kept->y8) bad = "y is kept in one form";
  else if (has_norm && !kept->out && !kept->out8) bad = "the gradient of the norm needs what was kept of out";
  else if (!has_y && ((h->post != kNone && grad_y) || g.post_gain || g.post_shift || g.gate)) bad = "these gradients need what was kept of y";
  else if ((has_norm || through_post) && !kept->stats) bad = "the gradients of norms need stats";
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
  int teams = 0;
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
    const int bytes[5] = {grad_out ? size : 0, has_norm ? 16 : 0, !has_norm ? 0 : f.out8.codes ? 12 : size,
                          f.y8.codes ? 12 : f.y.p ? 16 : 0, f.gate_rows.p ? 16 : 0};
    const Plan p = lay_out(&f.a, vec ? chunks_of(h->d, T, 2) : 1, kThreads, kThreads, bytes, f.post_shift ? 3 : 2,
                           quads_of(h->pre == kLayer, h->post), vec);
    // what a team keeps of its rows is written and read once more: 8 rows at least,
    // unless that leaves SMs idle
    teams = std::min({T, kSms * p.per_sm / p.blocks, most_teams(h), std::max(kSms / p.blocks, T / 8)});
    return by_kind(h, vec, p.chunks, [&](auto v, auto layer, auto post, auto c) {
      constexpr bool VEC = decltype(v)::value, LAYER = decltype(layer)::value;
      constexpr int POST = decltype(post)::value, CH = decltype(c)::value;
      auto* kernel = norm_backward<R, VEC, LAYER, POST, CH>;
      cudaError_t e = allow_smem<BackwardKernel<R, VEC, LAYER, POST, CH>>(kernel);
      return e == cudaSuccess ? launch(kernel, (unsigned)(teams * p.blocks), p.blocks, p.threads, p.smem, s, f) : e;
    });
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
