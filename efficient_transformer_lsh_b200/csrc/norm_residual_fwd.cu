// Forward of the norms and the residual add; see norm_residual.cuh.
#include "norm_residual.cuh"

namespace lsh {
namespace {

// Parameters, in order: P1 = gate w_post, P0 = gate b_post (a sigmoid gate is
// not in them), W, B: the products are formed once a CTA, not once a token.
template <class T, int V, int PER, int TEAM, bool BRANCH>
__global__ void __launch_bounds__(V == 1 ? 32 * kMaxWarps : kTeamThreads)
sub_fwd_kernel(const __grid_constant__ SubArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  using At = Place<T, V, PER, TEAM, BRANCH ? 4 : 2>;
  constexpr int P = At::P;
  At at(a, smem);
  const bool post = BRANCH && a.post != LSH_NORM_NONE, norm = a.norm != LSH_NORM_NONE;
  const bool sig = BRANCH && a.gate == LSH_GATE_SIGMOID;
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
  const Philox rng(a.seed, a.offset + (a.counter ? __ldg(a.counter) : 0));
  const int step = at.step(), rounds = at.rounds();
  const uint32_t stage_bytes = tensors * at.tensor();

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
            at.issue(a.f, at.of, rf, s_in + at.tensor());
            if (sig) at.issue(a.z, at.of, rf, s_in + 2 * at.tensor());
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
    f2 v[P];
    if constexpr (BRANCH) {
      at.get(a.f, a.sf, b, l, live, st + at.tensor(), v);
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
      if (has1) at.scale_by(0, v);
      if (has0) at.shift_by(1, v);
      if (sig) {
        f2 z[P];
        at.get(a.z, a.sf, b, l, live, st + 2 * at.tensor(), z);
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
        at.drop_all(rng, b, l, m * a.drop_scale, v);
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
      if (a.w) at.scale_by(kW, v);
      if (a.b) at.shift_by(kB, v);
      at.template put<false>(a.h, a.sh, BRANCH ? at.ox : at.oh, b, l, live, v);
    }
    st += stage_bytes;
    if (st == at.ring + a.stages * stage_bytes) st = at.ring;
  }
  if constexpr (At::kRing) cp_wait<0>();
}

template <class T, int V, int PER, int TEAM>
cudaError_t run(const SubCall& c, const SubArgs& a, const SubShape& s, cudaStream_t st) {
  auto fn = c.branch ? sub_fwd_kernel<T, V, PER, TEAM, true>
                     : sub_fwd_kernel<T, V, PER, TEAM, false>;
  if (s.smem > kSmemDefault) {
    cudaError_t e =
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerSm);
    if (e != cudaSuccess) return e;
  }
  fn<<<(unsigned)((int64_t)s.groups * s.parts), s.threads, s.smem, st>>>(a);
  note_launch();
  return cudaGetLastError();
}
template <class T>
cudaError_t run_type(const SubCall& c, const SubArgs& a, const SubShape& s, cudaStream_t st) {
  if (s.wide)
    return with_team(s.team, [&](auto t) {
      return run<T, 16 / (int)sizeof(T), 32, t.value>(c, a, s, st);
    });
  return s.team == 32 ? run<T, 1, kNarrowPer, 32>(c, a, s, st)
                      : run<T, 1, kNarrowPer, 0>(c, a, s, st);
}

}  // namespace

SubShape sub_shape(const SubCall& c, const SubSize& z) {
  SubShape s{};
  const int D = c.H * c.d, esize = c.dtype == LSH_BF16 ? 2 : 4;
  s.groups = c.gate_batch ? c.B : 1;
  s.tokens = c.gate_batch ? c.L : c.B * c.L;
  s.wide = c.wide;
  for (const lsh_strides* t : {&c.sx, &c.sf, &c.sh})
    if ((c.H - 1) * t->h + c.d > (int64_t)INT32_MAX) s.wide = false;
  int ctas = z.ctas;
  for (;;) {
    const int per = s.wide ? z.per : kNarrowPer;
    // threads of a token: a power of two up to a warp, then whole warps
    s.team = (D + per - 1) / per;
    if (s.team > 32) {
      s.team = (s.team + 31) / 32 * 32;
    } else if (s.wide) {
      int n = 2;
      while (n < s.team) n *= 2;
      s.team = n;
    } else {
      s.team = 32;
    }
    s.teams = std::max(1, kTeamThreads / s.team);
    s.threads = s.teams * s.team;
    const int fixed = z.vecs * per * 4 * s.team + (s.team > 32 ? s.teams * 32 * kMaxWarps : 0);
    s.stages = 1;
    s.smem = fixed;
    if (s.wide) {
      const int stage = z.tensors * (s.team > 32 ? s.threads : kTeamThreads) * per * esize;
      while (ctas > 1 && fixed + 2 * stage > kSmemPerSm / ctas - 1024) --ctas;
      if (fixed + stage > kSmemPerSm / ctas - 1024) {
        s.wide = false;
        continue;
      }
      s.stages = std::min(kMaxStages, (kSmemPerSm / ctas - 1024 - fixed) / stage);
      s.smem = fixed + s.stages * stage;
    }
    break;
  }
  const int64_t rows = ((int64_t)s.tokens + s.teams - 1) / s.teams;
  s.parts = (int)std::min<int64_t>(rows, std::max(1, kSms * ctas / std::max(1, s.groups)));
  return s;
}

SubArgs sub_args(const SubCall& c, const SubShape& s) {
  SubArgs a{};
  const int V = !s.wide ? 1 : c.dtype == LSH_BF16 ? 8 : 4;
  a.x = c.x, a.f = c.f, a.dy = c.dy, a.dh = c.dh;
  a.y = c.y, a.h = c.h, a.dx = c.dx, a.df = c.df, a.dz = c.dz;
  a.wp = c.wp, a.bp = c.bp, a.w = c.w, a.b = c.b;
  a.z = c.gate == LSH_GATE_SIGMOID ? c.gatep : nullptr;
  a.gv = c.gate == LSH_GATE_VECTOR ? (const float*)c.gatep : nullptr;
  a.sx = c.sx, a.sf = c.sf, a.sh = c.sh;
  a.upr = FastDiv((uint32_t)(c.d / V));
  a.fl = FastDiv((uint32_t)std::max(1, c.L));
  a.H = c.H, a.L = c.L, a.D = c.H * c.d;
  a.units = a.D / V;
  a.gpr = (c.d + 7) / 8;
  a.tokens = s.tokens, a.parts = s.parts;
  a.team = s.team, a.teams = s.teams, a.stages = s.stages;
  a.post = c.post, a.norm = c.norm, a.gate = c.gate, a.gate_batch = c.gate_batch;
  a.eps_post = c.eps_post, a.eps = c.eps, a.alpha = c.alpha, a.beta = c.beta;
  a.inv_d = 1.f / (float)a.D;
  a.drop_t = c.drop_t, a.drop_scale = c.drop_scale;
  a.seed = c.seed, a.offset = c.offset, a.counter = c.counter, a.slice0 = c.slice0;
  return a;
}

cudaError_t launch_sub_fwd(const SubCall& c, cudaStream_t st) {
  const SubShape s = sub_shape(c, {32, 1 + c.branch + (c.gate == LSH_GATE_SIGMOID),
                                   c.branch ? 4 : 2, c.branch ? 2 : 3});
  const SubArgs a = sub_args(c, s);
  return c.dtype == LSH_BF16 ? run_type<__nv_bfloat16>(c, a, s, st) : run_type<float>(c, a, s, st);
}

}  // namespace lsh
