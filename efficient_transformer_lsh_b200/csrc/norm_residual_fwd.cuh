// Forward kernel of the norms and the residual add; see norm_residual.cuh.
// Instantiated for each element type in a file of its own.
#pragma once

#include "norm_residual.cuh"

namespace lsh {
namespace {

// One pass: the row of f (or x) in registers, its statistics, the gate, the
// dropout, the add, y's statistics and h, each activation read and written
// once. 64K tokens of 512 features: a norm alone 25.9 us (134 MB, 5.2 TB/s),
// with everything on 52.9 us (268 MB, 5.1 TB/s); there a token's 520 warp
// instructions (bf16 unpacking, the two statistics, ten Philox rounds for every
// 8 features) issue in 29 us, its bytes take 41, and 16 warps an SM overlap them
// in part. 4 x 8192 tokens of 4096 features, a norm: 82 us (537 MB, 6.5 TB/s:
// HBM); 8192 of them with everything on 71 us (floor 41: two barriers a
// LayerNorm, one CTA an SM).
//
// Parameters, in order: W, P1 = gate w_post (a sigmoid gate is not in it), then
// B, P0 = gate b_post where there is one of them: the products are formed once
// a CTA, not once a token.
template <class T, int V, int PER, int TEAM, int TOK, bool BRANCH, bool POST, bool SIG>
__global__ void __launch_bounds__(V == 1 || TEAM == 0 ? kFwdBig : FwdSize<T, BRANCH>::kThreads,
                                  V == 1 || TEAM == 0 ? 1 : FwdSize<T, BRANCH>::kCtas)
sub_fwd_kernel(const __grid_constant__ SubArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  using At = Place<T, V, PER, TEAM, TOK, V == 1 ? kNarrowThreads : FwdSize<T, BRANCH>::kThreads>;
  constexpr int P = At::P;
  At at(a, smem);
  stream_wait();
  let_next_start();
  constexpr bool post = BRANCH && POST, sig = BRANCH && SIG;
  const bool norm = a.norm != LSH_NORM_NONE;
  const float* gv = a.gv ? a.gv + (int64_t)at.group * (a.gate_batch ? a.D : 0) : nullptr;
  const bool has1 = BRANCH && (a.wp || gv), has0 = BRANCH && a.bp;
  constexpr int kW = 0, kP1 = 1, kB = BRANCH ? 2 : 1, kP0 = 3;
  const int tensors = 1 + BRANCH + sig;
  if (at.on_bits != At::kAll) at.clear(at.ring, a.stages * tensors * TOK);
  const uint64_t offset = a.offset + (a.counter ? *a.counter : 0);
  const int step = at.step(), rounds = at.rounds();
  const uint32_t one = at.one(), token_bytes = tensors * one, stage_bytes = TOK * token_bytes;

  int t_in = at.first(), n_in = 0;
  uint32_t s_in = at.ring;      // where the next tokens' copies go
  auto copy = [&]() {
    if constexpr (At::kRing) {
      if (n_in < rounds) {
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
          const uint32_t to = s_in + j * token_bytes;
          if (t_in + j < a.tokens) {
            int b, l;
            at.token(t_in + j, b, l);
            at.issue(a.x, at.ox, At::row(a.sx, b, l), to);
            if constexpr (BRANCH) {
              const int64_t rf = At::row(a.sf, b, l);
              at.issue(a.f, at.of, rf, to + one);
              if (sig) at.issue(a.z, at.of, rf, to + 2 * one);
            }
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
  if (norm && (a.w || a.b)) at.stage_param(kW, a.w, nullptr);
  if (has1 || has0) at.stage_param(kP1, a.wp, gv);
  if (norm && a.b) at.stage_param(kB, a.b, nullptr);
  if (has0) at.stage_param(kP0, a.bp, gv);
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
    auto get = [&](const void* p, const SubLayout& s, int i, int j, f2(&v)[P]) {
      at.get(p, s, b[j], l[j], live[j], st + j * token_bytes + i * one, v);
    };
    f2 v[TOK][P];
    // v -> xhat of each token
    auto normalize = [&](int kind, float eps) {
      float s[TOK];
      if (kind == LSH_NORM_LAYER) {
#pragma unroll
        for (int j = 0; j < TOK; ++j) s[j] = sum_all(v[j]);
        at.team_sum(s);
#pragma unroll
        for (int j = 0; j < TOK; ++j) at.center(v[j], s[j] * a.inv_d);
      }
#pragma unroll
      for (int j = 0; j < TOK; ++j) s[j] = dot_all(v[j], v[j]);
      at.team_sum(s);
#pragma unroll
      for (int j = 0; j < TOK; ++j) scale_all(v[j], inv_std(s[j], a.inv_d, eps));
    };
    if constexpr (BRANCH) {
#pragma unroll
      for (int j = 0; j < TOK; ++j) get(a.f, a.sf, 1, j, v[j]);
      if (post) normalize(a.post, a.eps_post);
      if (has0) at.scale_shift(kP1, kP0, v);
      else if (has1) at.scale_by(kP1, v);
      if constexpr (sig) {
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
          f2 z[P];
          get(a.z, a.sf, 2, j, z);
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const float2 u = up(z[i]);
            float slope;
            const float g0 = sigmoid<T>(u.x, slope), g1 = sigmoid<T>(u.y, slope);
            v[j][i] = mul2(v[j][i], pk(g0, g1));
          }
        }
      }
#pragma unroll
      for (int j = 0; j < TOK; ++j) {
        if (a.drop_t) at.drop_all(offset, b[j], l[j], a.alpha * a.drop_scale, v[j]);
        else scale_all(v[j], a.alpha);
        f2 x[P];
        get(a.x, a.sx, 0, j, x);
        const f2 beta = pk(a.beta, a.beta);
#pragma unroll
        for (int i = 0; i < P; ++i) v[j][i] = fma2(x[i], beta, v[j][i]);
        // v becomes the row as stored: h is the same whether it comes from
        // here or from a later pass over y
        at.template put<true>(a.y, a.sx, at.ox, b[j], l[j], live[j], v[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < TOK; ++j) get(a.x, a.sx, 0, j, v[j]);
    }
    if (norm) {
      normalize(a.norm, a.eps);
      if (a.b) at.scale_shift(kW, kB, v);
      else if (a.w) at.scale_by(kW, v);
#pragma unroll
      for (int j = 0; j < TOK; ++j)
        at.template put<false>(a.h, a.sh, BRANCH ? at.ox : at.oh, b[j], l[j], live[j], v[j]);
    }
    st += stage_bytes;
    if (st == at.ring + a.stages * stage_bytes) st = at.ring;
  }
  if constexpr (At::kRing) cp_wait<0>();
}

template <class T, int V, int PER, int TEAM, int TOK>
cudaError_t run(const SubCall& c, const SubArgs& a, const SubShape& s, cudaStream_t st) {
  const bool sig = c.gate == LSH_GATE_SIGMOID, post = c.post != LSH_NORM_NONE;
  auto fn = !c.branch     ? sub_fwd_kernel<T, V, PER, TEAM, TOK, false, false, false>
            : post && sig ? sub_fwd_kernel<T, V, PER, TEAM, TOK, true, true, true>
            : post        ? sub_fwd_kernel<T, V, PER, TEAM, TOK, true, true, false>
            : sig         ? sub_fwd_kernel<T, V, PER, TEAM, TOK, true, false, true>
                          : sub_fwd_kernel<T, V, PER, TEAM, TOK, true, false, false>;
  if (s.smem > kSmemDefault) {
    cudaError_t e =
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerSm);
    if (e != cudaSuccess) return e;
  }
  note_launch();
  return launch_overlapped(fn, dim3((unsigned)((int64_t)s.groups * s.parts)), s.threads, s.smem, st, a);
}

}  // namespace

template <class T>
cudaError_t sub_fwd_type(const SubCall& c, const SubArgs& a, const SubShape& s, cudaStream_t st) {
  if (s.wide)
    return with_team(s.team, [&](auto t) {
      return run<T, 16 / (int)sizeof(T), kFwdPer, t.value, 1>(c, a, s, st);
    });
  return s.team == 32 ? run<T, 1, kNarrowPer, 32, 1>(c, a, s, st)
                      : run<T, 1, kNarrowPer, 0, 1>(c, a, s, st);
}

}  // namespace lsh
