// Backward kernel of the norms and the residual add; see norm_residual.cuh.
// Instantiated for each element type, with and without a norm of y and a
// sigmoid gate, in a file of its own.
//
// Parameter gradients are sums over tokens. Every thread keeps its features'
// sums in registers over all the tokens it visits; a CTA writes one row of
// partial sums, and a second kernel adds the rows in order: no atomics, the
// same result every time. Four sums suffice, per group of tokens that shares
// a gate vector: A = sum dh yhat, B = sum dh, S1 = sum q fhat, S0 = sum q
// (q before the gate; du for a sigmoid gate):
//   dw = A, db = B, dw_post = gate S1, db_post = gate S0,
//   dgate = w_post S1 + b_post S0.
//
// A row needs at most three sums over its features: both means; then squared
// deviations of y and f, a and a (y - mean) together (a does not depend on the
// statistics, so r is factored out: mean(a yhat) = r mean(a (y - mean))); then
// the second norm's a and a (f - mean).
//
// 64K tokens of 512 features in bf16: a norm's 49.8 us with the sum of the
// partials (268 MB, 5.4 TB/s); with everything on 93.8 us (403 MB, 4.3 TB/s),
// bound by latency at the two warps a scheduler that 230 registers leave: its
// 765 warp instructions a token (130 of them the dropout's) issue in 43 us, half
// of the slots, and its bytes take 61 (three warps of 168 registers spill: 102.7
// us where this was 100.3). float32: a norm
// of 64K tokens 93 us, 5.8 TB/s (HBM).
#pragma once

#include "norm_residual.cuh"

namespace lsh {
namespace {

// A thread's sums s into the row starting at `row`.
template <class At>
__device__ __forceinline__ void put_sums(const At& at, const f2 (&s)[At::P], float* row) {
  constexpr int V = At::P * 2 / At::NV;
#pragma unroll
  for (int k = 0; k < At::NV; ++k)
    if (at.on(k)) {
      if constexpr (V > 1) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
          const float2 a = up(s[(k * V + 4 * i) / 2]), b = up(s[(k * V + 4 * i) / 2 + 1]);
          *reinterpret_cast<float4*>(row + at.feat(k) + 4 * i) = make_float4(a.x, a.y, b.x, b.y);
        }
      } else {
        const float2 u = up(s[k / 2]);
        row[at.feat(k)] = k & 1 ? u.y : u.x;
      }
    }
}

// Parameters, in order: W, P1 = gate w_post (a sigmoid gate is not in it), P0
// = b_post (sigmoid gates only).
template <class T, int V, int PER, int TEAM, int TOK, bool BRANCH, bool NORM, bool POST, bool SIG>
__global__ void __launch_bounds__(bwd_threads<T, V, PER, TEAM, SIG>(),
                                  bwd_ctas<T, V, PER, TEAM, SIG>())
sub_bwd_kernel(const __grid_constant__ SubArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  using At = Place<T, V, PER, TEAM, TOK, V == 1 ? kNarrowThreads : BwdSize<T, SIG>::kThreads>;
  constexpr int P = At::P;
  constexpr int kP1 = NORM ? 1 : 0, kP0 = kP1 + 1;
  At at(a, smem);
  stream_wait();
  let_next_start();
  constexpr bool post = BRANCH && POST, sig = BRANCH && SIG;
  const float* gv = a.gv ? a.gv + (int64_t)at.group * (a.gate_batch ? a.D : 0) : nullptr;
  // with a norm of f always there: it also keeps features past D out of the sums
  const bool has1 = post || (BRANCH && gv), has0 = sig && a.bp;
  // the ring's tensors: y dh, dy, f, z
  const int i_dy = NORM ? 2 : 0, i_f = i_dy + (a.dy ? 1 : 0), i_z = i_f + 1;
  const int tensors = i_f + BRANCH + sig;
  if (at.on_bits != At::kAll) at.clear(at.ring, a.stages * tensors * TOK);
  const uint64_t offset = a.offset + (a.counter ? *a.counter : 0);
  const int step = at.step(), rounds = at.rounds();
  const uint32_t one = at.one(), token_bytes = tensors * one, stage_bytes = TOK * token_bytes;
  const float own = at.count(), inv_own = own > 0.f ? 1.f / own : 0.f;
  const bool lf = post && a.post == LSH_NORM_LAYER, ly = NORM && a.norm == LSH_NORM_LAYER;
  f2 sa[P], sb[P], s1[P], s0[P];
#pragma unroll
  for (int i = 0; i < P; ++i) sa[i] = sb[i] = s1[i] = s0[i] = 0ull;

  int t_in = at.first(), n_in = 0;
  uint32_t s_in = at.ring;
  auto copy = [&]() {
    if constexpr (At::kRing) {
      if (n_in < rounds) {
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
          const uint32_t to = s_in + j * token_bytes;
          if (t_in + j < a.tokens) {
            int b, l;
            at.token(t_in + j, b, l);
            const int64_t rx = At::row(a.sx, b, l);
            if constexpr (NORM) {
              at.issue(a.x, at.ox, rx, to);
              at.issue(a.dh, BRANCH ? at.ox : at.oh, BRANCH ? rx : At::row(a.sh, b, l), to + one);
            }
            if (a.dy) at.issue(a.dy, at.ox, rx, to + i_dy * one);
            if constexpr (BRANCH) {
              const int64_t rf = At::row(a.sf, b, l);
              at.issue(a.f, at.of, rf, to + i_f * one);
              if (sig) at.issue(a.z, at.of, rf, to + i_z * one);
            }
          } else {
            // nothing may be added for a token that is not there
            at.clear(to, tensors);
          }
        }
        t_in += step;
        ++n_in;
        s_in += stage_bytes;
        if (s_in == at.ring + a.stages * stage_bytes) s_in = at.ring;
      }
      cp_commit();
    }
  };
  // the first tokens are on the way while the parameters are staged
  const bool ahead = a.stages > 1;
  for (int i = ahead; i < a.stages; ++i) copy();
  if (NORM) at.stage_param(0, a.w, nullptr);
  if (has1) at.stage_param(kP1, a.wp, gv);
  if (has0) at.stage_param(kP0, a.bp, nullptr);
  __syncthreads();
  uint32_t st = at.ring;
  int t = at.first();
  for (int n = 0; n < rounds; ++n, t += step) {
    if (n > 0 || ahead) copy();
    if constexpr (At::kRing) cp_wait_for(a.stages - 1);
    int b[TOK], l[TOK];
    bool live[TOK];
#pragma unroll
    for (int j = 0; j < TOK; ++j) {
      live[j] = (At::kMulti && TOK == 1) || t + j < a.tokens;
      at.token(t + j, b[j], l[j]);
    }
    auto get_x = [&](const void* p, int i, int j, f2(&v)[P]) {
      at.get(p, a.sx, b[j], l[j], live[j], st + j * token_bytes + i * one, v);
    };
    auto get_f = [&](const void* p, int i, int j, f2(&v)[P]) {
      at.get(p, a.sf, b[j], l[j], live[j], st + j * token_bytes + i * one, v);
    };
    auto get_dh = [&](int j, f2(&v)[P]) {
      at.get(a.dh, a.sh, b[j], l[j], live[j], st + j * token_bytes + one, v);
    };
    f2 q[TOK][P];     // T, then q, then du
    f2 hat[TOK][P];   // y - mean, then f - mean, then fhat
    float r_f[TOK], mean_f[TOK];
    // a thread's own mean and squared deviations of f: those of the row follow
    // from them (Chan, Golub and LeVeque 1979) without another look at f
    float own_mean[TOK], own_sq[TOK];
    if constexpr (NORM) {
#pragma unroll
      for (int j = 0; j < TOK; ++j) {
        get_x(a.x, 0, j, hat[j]);
        mean_f[j] = 0.f;
      }
      if (lf || ly) {
        float s[2 * TOK];
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
          s[2 * j] = sum_all(hat[j]);
          s[2 * j + 1] = 0.f;
          if (lf) {
            get_f(a.f, i_f, j, q[j]);
            s[2 * j + 1] = sum_all(q[j]);
            own_mean[j] = s[2 * j + 1] * inv_own;
            at.center(q[j], own_mean[j]);
            own_sq[j] = dot_all(q[j], q[j]);
          }
        }
        at.team_sum(s);
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
          if (ly) at.center(hat[j], s[2 * j] * a.inv_d);
          mean_f[j] = s[2 * j + 1] * a.inv_d;
        }
      }
      float s[4 * TOK];
#pragma unroll
      for (int j = 0; j < TOK; ++j) {
        s[4 * j + 3] = 0.f;
        if (lf) {
          const float d = own_mean[j] - mean_f[j];
          s[4 * j + 3] = fmaf(own * d, d, own_sq[j]);
        } else if (post) {
          get_f(a.f, i_f, j, q[j]);
          s[4 * j + 3] = dot_all(q[j], q[j]);
        }
        s[4 * j] = dot_all(hat[j], hat[j]);
        get_dh(j, q[j]);
#pragma unroll
        for (int i = 0; i < P; ++i) sb[i] = add2(sb[i], q[j][i]);
      }
      at.scale_by(0, q);
#pragma unroll
      for (int j = 0; j < TOK; ++j) {
        s[4 * j + 1] = sum_all(q[j]);
        s[4 * j + 2] = dot_all(q[j], hat[j]);
      }
      at.team_sum(s);
#pragma unroll
      for (int j = 0; j < TOK; ++j) {
        const float r = inv_std(s[4 * j], a.inv_d, a.eps);
        if (post) r_f[j] = inv_std(s[4 * j + 3], a.inv_d, a.eps_post);
        const float m0 = ly ? s[4 * j + 1] * a.inv_d : 0.f, m1 = r * r * s[4 * j + 2] * a.inv_d;
        const f2 r2 = pk(r, r), k0 = pk(-r * m0, -r * m0), k1 = pk(-r * m1, -r * m1);
        {
          f2 dh[P];
          get_dh(j, dh);
#pragma unroll
          for (int i = 0; i < P; ++i) sa[i] = fma2(dh[i], mul2(hat[j][i], r2), sa[i]);
        }
#pragma unroll
        for (int i = 0; i < P; ++i) q[j][i] = fma2(q[j][i], r2, fma2(hat[j][i], k1, k0));
      }
      if (a.dy) {
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
          get_x(a.dy, i_dy, j, hat[j]);
#pragma unroll
          for (int i = 0; i < P; ++i) q[j][i] = add2(q[j][i], hat[j][i]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < TOK; ++j) get_x(a.dy, i_dy, j, q[j]);
    }
    if (a.dx) {
#pragma unroll
      for (int j = 0; j < TOK; ++j) {
        if (BRANCH && a.beta != 1.f) {
#pragma unroll
          for (int i = 0; i < P; ++i) hat[j][i] = mul2(q[j][i], pk(a.beta, a.beta));
          at.template put<false>(a.dx, a.sx, at.ox, b[j], l[j], live[j], hat[j]);
        } else {
          at.template put<false>(a.dx, a.sx, at.ox, b[j], l[j], live[j], q[j]);
        }
      }
    }
    if constexpr (BRANCH) {
#pragma unroll
      for (int j = 0; j < TOK; ++j) get_f(a.f, i_f, j, hat[j]);
      if (post) {
        if constexpr (!NORM) {
          float s[TOK];
          if (lf) {
#pragma unroll
            for (int j = 0; j < TOK; ++j) s[j] = sum_all(hat[j]);
            at.team_sum(s);
#pragma unroll
            for (int j = 0; j < TOK; ++j) at.center(hat[j], s[j] * a.inv_d);
          }
#pragma unroll
          for (int j = 0; j < TOK; ++j) s[j] = dot_all(hat[j], hat[j]);
          at.team_sum(s);
#pragma unroll
          for (int j = 0; j < TOK; ++j) r_f[j] = inv_std(s[j], a.inv_d, a.eps_post);
        }
        // fhat = f r - mean r in one step (past D it is not 0, but q is there)
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
          const float m = NORM && lf ? -mean_f[j] * r_f[j] : 0.f;
          const f2 r2 = pk(r_f[j], r_f[j]), m2 = pk(m, m);
#pragma unroll
          for (int i = 0; i < P; ++i) hat[j][i] = fma2(hat[j][i], r2, m2);
        }
      }
#pragma unroll
      for (int j = 0; j < TOK; ++j) {
        if (a.drop_t) at.drop_all(offset, b[j], l[j], a.alpha * a.drop_scale, q[j]);
        else scale_all(q[j], a.alpha);
      }
      if constexpr (sig) {
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
          f2 u[1][P], z[P];
#pragma unroll
          for (int i = 0; i < P; ++i) u[0][i] = hat[j][i];
          if (post && a.wp) at.scale_by(kP1, u);
          if (has0) at.shift_by(kP0, u);
          get_f(a.z, i_z, j, z);
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const float2 w = up(z[i]);
            float d0, d1;
            const float g0 = sigmoid<T>(w.x, d0), g1 = sigmoid<T>(w.y, d1);
            u[0][i] = mul2(u[0][i], mul2(q[j][i], pk(d0, d1)));
            q[j][i] = mul2(q[j][i], pk(g0, g1));
          }
          if (a.dz) at.template put<false>(a.dz, a.sf, at.of, b[j], l[j], live[j], u[0]);
        }
      }
#pragma unroll
      for (int j = 0; j < TOK; ++j)
#pragma unroll
        for (int i = 0; i < P; ++i) {
          s1[i] = fma2(q[j][i], hat[j][i], s1[i]);
          s0[i] = add2(s0[i], q[j][i]);
        }
      if (has1) at.scale_by(kP1, q);
      if (post) {
        float s[2 * TOK];
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
          s[2 * j] = sum_all(q[j]);
          s[2 * j + 1] = dot_all(q[j], hat[j]);
        }
        at.team_sum(s);
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
          const float r = r_f[j], m0 = lf ? s[2 * j] * a.inv_d : 0.f, m1 = s[2 * j + 1] * a.inv_d;
          const f2 r2 = pk(r, r), k0 = pk(-r * m0, -r * m0), k1 = pk(-r * m1, -r * m1);
#pragma unroll
          for (int i = 0; i < P; ++i) q[j][i] = fma2(q[j][i], r2, fma2(hat[j][i], k1, k0));
        }
      }
#pragma unroll
      for (int j = 0; j < TOK; ++j)
        at.template put<false>(a.df, a.sf, at.of, b[j], l[j], live[j], q[j]);
    }
    st += stage_bytes;
    if (st == at.ring + a.stages * stage_bytes) st = at.ring;
  }
  if constexpr (At::kRing) cp_wait<0>();
  if (a.part) {
    // a CTA's row of partial sums, A B and S1 S0: one team's straight from its
    // registers, several teams' added in order in shared memory, where the
    // parameters and the ring are done with
    constexpr int kVecs = (NORM ? 2 : 0) + (BRANCH ? 2 : 0);
    float* out = a.part + (int64_t)blockIdx.x * kVecs * a.D;
    const bool alone = a.teams == 1;
    const int64_t vec = alone ? a.D : a.teams * a.D;
    float* row = alone ? out : reinterpret_cast<float*>(smem) + at.team_id * a.D;
    if (!alone) __syncthreads();
    if constexpr (NORM) {
      put_sums(at, sa, row);
      put_sums(at, sb, row + vec);
      row += 2 * vec;
    }
    if constexpr (BRANCH) {
      put_sums(at, s1, row);
      put_sums(at, s0, row + vec);
    }
    if (!alone) {
      __syncthreads();
      const float* buf = reinterpret_cast<const float*>(smem);
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
        for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
          float t = 0.f;
          for (int w = 0; w < a.teams; ++w) t += buf[(v * a.teams + w) * a.D + c];
          out[v * a.D + c] = t;
        }
    }
  }
}

template <class Kernel>
cudaError_t run_kernel(Kernel fn, const SubArgs& a, const SubShape& s, cudaStream_t st) {
  // several teams' sums go through the same memory
  const int smem = std::max(s.smem, s.teams > 1 ? s.teams * a.D * 16 : 0);
  if (smem > kSmemDefault) {
    cudaError_t e =
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerSm);
    if (e != cudaSuccess) return e;
  }
  note_launch();
  return launch_overlapped(fn, dim3((unsigned)((int64_t)s.groups * s.parts)), s.threads, smem, st,
                           a);
}
template <class T, int V, int PER, int TEAM, int TOK, bool NORM, bool SIG>
cudaError_t run_branch(const SubCall& c, const SubArgs& a, const SubShape& s, cudaStream_t st) {
  if constexpr (NORM && !SIG && PER != kBwdWidePer && TEAM != kBig)
    if (!c.branch)
      return run_kernel(sub_bwd_kernel<T, V, PER, TEAM, TOK, false, true, false, false>, a, s, st);
  return c.post != LSH_NORM_NONE
             ? run_kernel(sub_bwd_kernel<T, V, PER, TEAM, TOK, true, NORM, true, SIG>, a, s, st)
             : run_kernel(sub_bwd_kernel<T, V, PER, TEAM, TOK, true, NORM, false, SIG>, a, s, st);
}

}  // namespace

template <class T, bool NORM, bool SIG>
cudaError_t sub_bwd_type(const SubCall& c, const SubArgs& a, const SubShape& s, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(T), TOK = BwdSize<T, SIG>::kTok;
  if (s.wide && s.per == kBwdWidePer) {
    if constexpr (NORM && !SIG)
      if (!c.branch)
        return run_kernel(s.team == 32
                              ? sub_bwd_kernel<T, V, kBwdWidePer, 32, 1, false, true, false, false>
                              : sub_bwd_kernel<T, V, kBwdWidePer, 0, 1, false, true, false, false>,
                          a, s, st);
    if constexpr (sizeof(T) == 2 && !SIG)
      if (s.team > 32) return run_branch<T, V, kBwdWidePer, 0, 1, NORM, SIG>(c, a, s, st);
    if constexpr (sizeof(T) == 2)
      return run_branch<T, V, kBwdWidePer, 32, 1, NORM, SIG>(c, a, s, st);
  }
  if constexpr (sizeof(T) == 4 || SIG)
    if (s.wide && s.team > kBwdTeam)
      return run_branch<T, V, kBwdPer, kBig, 1, NORM, SIG>(c, a, s, st);
  if (s.wide)
    return with_team(s.team, [&](auto t) {
      return run_branch<T, V, kBwdPer, t.value, t.value == 0 ? 1 : TOK, NORM, SIG>(c, a, s, st);
    });
  return s.team == 32 ? run_branch<T, 1, kNarrowPer, 32, 1, NORM, SIG>(c, a, s, st)
                      : run_branch<T, 1, kNarrowPer, 0, 1, NORM, SIG>(c, a, s, st);
}

}  // namespace lsh
