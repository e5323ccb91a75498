// Forward kernel of the norms and the residual add; see norm_residual.cuh.
// Instantiated for each element type in a file of its own.
#pragma once

#include "norm_residual.cuh"

namespace lsh {
namespace {

// Parameters, in order: P1 = gate w_post, P0 = gate b_post (a sigmoid gate is
// not in them), W, B: the products are formed once a CTA, not once a token.
template <class T, int V, int PER, int TEAM, bool BRANCH, bool POST, bool SIG>
__global__ void __launch_bounds__(V == 1 ? 32 * kMaxWarps : kFwdThreads,
                                  V == 1   ? 1
                                  : BRANCH ? kFwdCtas
                                           : kFwdNormCtas)
sub_fwd_kernel(const __grid_constant__ SubArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  using At = Place<T, V, PER, TEAM, BRANCH ? 4 : 2, 1, V == 1 ? kNarrowThreads : kFwdThreads>;
  constexpr int P = At::P;
  At at(a, smem);
  stream_wait();
  let_next_start();
  constexpr bool post = BRANCH && POST, sig = BRANCH && SIG;
  const bool norm = a.norm != LSH_NORM_NONE;
  const float* gv = a.gv ? a.gv + (int64_t)at.group * (a.gate_batch ? a.D : 0) : nullptr;
  const bool has1 = BRANCH && (a.wp || gv), has0 = BRANCH && a.bp;
  constexpr int kW = BRANCH ? 2 : 0, kB = kW + 1;
  if (has1) at.stage_param(0, a.wp, gv);
  if (has0) at.stage_param(1, a.bp, gv);
  if (norm && a.w) at.stage_param(kW, a.w, nullptr);
  if (norm && a.b) at.stage_param(kB, a.b, nullptr);
  const int tensors = 1 + BRANCH + sig;
  at.clear(at.ring, a.stages * tensors);
  __syncthreads();
  const uint64_t offset = a.offset + (a.counter ? __ldg(a.counter) : 0);
  const int step = at.step(), rounds = at.rounds();
  const uint32_t stage_bytes = tensors * at.one();

  int t_in = at.first(), n_in = 0;
  uint32_t s_in = at.ring;      // where the next token's copies go
  auto copy = [&]() {
    if constexpr (At::kRing) {
      if (n_in < rounds) {
        if (t_in < a.tokens) {
          int b, l;
          at.token(t_in, b, l);
          const int64_t rx = At::row(a.sx, b, l);
          at.issue(a.x, at.ox, rx, s_in);
          if constexpr (BRANCH) {
            const int64_t rf = At::row(a.sf, b, l);
            at.issue(a.f, at.of, rf, s_in + at.one());
            if (sig) at.issue(a.z, at.of, rf, s_in + 2 * at.one());
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
  for (int i = 1; i < a.stages; ++i) copy();
  uint32_t st = at.ring;
  int t = at.first();
  for (int n = 0; n < rounds; ++n, t += step) {
    copy();
    if constexpr (At::kRing) cp_wait_for(a.stages - 1);
    const bool live = At::kMulti || t < a.tokens;
    int b, l;
    at.token(t, b, l);
    f2 row[1][P];
    f2(&v)[P] = row[0];
    if constexpr (BRANCH) {
      at.get(a.f, a.sf, b, l, live, st + at.one(), v);
      if (post) {
        float s[1];
        if (a.post == LSH_NORM_LAYER) {
          s[0] = sum_all(v);
          at.team_sum(s);
          at.center(v, s[0] * a.inv_d);
        }
        s[0] = dot_all(v, v);
        at.team_sum(s);
        scale_all(v, inv_std(s[0], a.inv_d, a.eps_post));
      }
      if (has1) at.scale_by(0, row);
      if (has0) at.shift_by(1, row);
      if (sig) {
        f2 z[P];
        at.get(a.z, a.sf, b, l, live, st + 2 * at.one(), z);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float2 u = up(z[i]);
          float slope;
          const float g0 = sigmoid(u.x, slope), g1 = sigmoid(u.y, slope);
          v[i] = mul2(v[i], pk(g0, g1));
        }
      }
      float m = a.alpha;
      if (a.drop_t) {
        at.drop_all(offset, b, l, m * a.drop_scale, v);
        m = 1.f;
      }
      f2 x[P];
      at.get(a.x, a.sx, b, l, live, st, x);
      const f2 m2 = pk(m, m), beta = pk(a.beta, a.beta);
#pragma unroll
      for (int i = 0; i < P; ++i) v[i] = fma2(v[i], m2, mul2(x[i], beta));
      // v becomes the row as stored: h is the same whether it comes from here
      // or from a later pass over y
      at.template put<true>(a.y, a.sx, at.ox, b, l, live, v);
    } else {
      at.get(a.x, a.sx, b, l, live, st, v);
    }
    if (norm) {
      float s[1];
      if (a.norm == LSH_NORM_LAYER) {
        s[0] = sum_all(v);
        at.team_sum(s);
        at.center(v, s[0] * a.inv_d);
      }
      s[0] = dot_all(v, v);
      at.team_sum(s);
      scale_all(v, inv_std(s[0], a.inv_d, a.eps));
      if (a.w) at.scale_by(kW, row);
      if (a.b) at.shift_by(kB, row);
      at.template put<false>(a.h, a.sh, BRANCH ? at.ox : at.oh, b, l, live, v);
    }
    st += stage_bytes;
    if (st == at.ring + a.stages * stage_bytes) st = at.ring;
  }
  if constexpr (At::kRing) cp_wait<0>();
}

template <class T, int V, int PER, int TEAM>
cudaError_t run(const SubCall& c, const SubArgs& a, const SubShape& s, cudaStream_t st) {
  const bool sig = c.gate == LSH_GATE_SIGMOID, post = c.post != LSH_NORM_NONE;
  auto fn = !c.branch     ? sub_fwd_kernel<T, V, PER, TEAM, false, false, false>
            : post && sig ? sub_fwd_kernel<T, V, PER, TEAM, true, true, true>
            : post        ? sub_fwd_kernel<T, V, PER, TEAM, true, true, false>
            : sig         ? sub_fwd_kernel<T, V, PER, TEAM, true, false, true>
                          : sub_fwd_kernel<T, V, PER, TEAM, true, false, false>;
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
      return run<T, 16 / (int)sizeof(T), kFwdPer, t.value>(c, a, s, st);
    });
  return s.team == 32 ? run<T, 1, kNarrowPer, 32>(c, a, s, st)
                      : run<T, 1, kNarrowPer, 0>(c, a, s, st);
}

}  // namespace lsh
