// Norms and the residual add: how a call is laid over the GPU, and the sum of
// the backward's partial parameter gradients.
#include "norm_residual.cuh"

namespace lsh {

// CTAs of a group when `all` share the groups.
static int max_parts(int all, int groups) { return std::max(1, all / std::max(1, groups)); }

SubShape sub_shape(const SubCall& c, const SubSize& z) {
  SubShape s{};
  s.vecs = z.vecs;
  const int D = c.H * c.d, esize = c.dtype == LSH_BF16 ? 2 : 4;
  s.groups = c.gate_batch ? c.B : 1;
  s.tokens = c.gate_batch ? c.L : c.B * c.L;
  s.wide = c.wide;
  for (const lsh_strides* t : {&c.sx, &c.sf, &c.sh})
    if (((c.H - 1) * t->h + c.d) / (16 / esize) > (int64_t)INT32_MAX ||
        std::max(t->b, t->l) / (16 / esize) > (int64_t)UINT32_MAX)
      s.wide = false;
  int ctas, fixed, big = kFwdBig;
  for (;;) {
    const bool wide_rows = s.wide && z.backward && D > 32 * kBwdPer &&
                           (!c.branch ||
                            (c.dtype == LSH_BF16 &&
                             (D <= kBwdWarpMax ||
                              (c.gate != LSH_GATE_SIGMOID && D > kBwdTeam * kBwdPer))));
    const int per = !s.wide ? kNarrowPer : wide_rows ? kBwdWidePer : z.per;
    const int threads = s.wide ? z.threads : kNarrowThreads;
    s.per = per;
    s.tok = s.wide && !wide_rows ? z.tok : 1;
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
    // Teams of several warps take one token at a time, with more of them
    // resident to cover their barriers (backward of 4 x 4096 tokens of 4096
    // features: 212 us, where two tokens took 245)
    if (s.team > 32) s.tok = 1;
    const int cta = s.wide && !z.backward && s.team > 32 ? big : threads;
    s.teams = std::max(1, cta / s.team);
    s.threads = s.teams * s.team;
    // threads resident on an SM, by the registers of each form
    int room = 512;
    if (wide_rows) room = kBwdRoom;
    else if (s.wide && z.backward && s.team > 32)
      room = s.team <= kBwdTeam ? kBwdTeamRoom : kBwdBigRoom;
    else if (s.wide && s.team <= 32) room = z.ctas * threads;
    ctas = std::max(1, room / s.threads);
    fixed = z.vecs * per * 4 * s.team + (s.team > 32 ? s.teams * 64 * kMaxWarps : 0);
    s.stages = 1;
    s.smem = fixed;
    if (s.wide) {
      const int stage = z.tensors * s.tok * (s.team > 32 ? s.threads : threads) * per * esize;
      // two stages before more CTAs, unless that many CTAs have no second
      // round to copy ahead for; but one stage before a single CTA of a
      // backward with barriers, which another one covers (8192 tokens of 4096
      // features in float32: 306 us with one CTA, 208 with two; 3 CTAs of one
      // stage for 12288 of 1536: 95, 80 with two)
      const int64_t all = ((int64_t)s.tokens + s.teams * s.tok - 1) / (s.teams * s.tok) * s.groups;
      while (ctas > 1 && fixed + stage > kSmemPerSm / ctas - 1024) --ctas;
      const int least = z.backward && s.team > 32 ? 2 : 1;
      if (all > kSms * ctas)
        while (ctas > least && fixed + 2 * stage > kSmemPerSm / ctas - 1024) --ctas;
      if (fixed + stage > kSmemPerSm / ctas - 1024) {
        if (!z.backward && s.team > 32 && s.teams > 1) big = s.team;   // fewer teams first
        else s.wide = false;
        continue;
      }
      s.stages = std::min(kMaxStages, (kSmemPerSm / ctas - 1024 - fixed) / stage);
      s.smem = fixed + s.stages * stage;
    }
    break;
  }
  const int64_t rows = ((int64_t)s.tokens + s.teams * s.tok - 1) / (s.teams * s.tok);
  s.parts = (int)std::min<int64_t>(rows, max_parts(std::min(kSms * ctas, kMaxParts), s.groups));
  // no more stages than rounds
  if (s.wide && s.parts > 0) {
    const int rounds = (int)std::min<int64_t>(kMaxStages, (rows + s.parts - 1) / s.parts);
    const int stage = (s.smem - fixed) / s.stages;
    s.stages = std::min(s.stages, rounds);
    s.smem = fixed + s.stages * stage;
  }
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
  const auto layout = [V](const lsh_strides& t) {
    return SubLayout{t, (uint32_t)(t.b / V), (uint32_t)(t.l / V)};
  };
  a.sx = layout(c.sx), a.sf = layout(c.sf), a.sh = layout(c.sh);
  a.upr = FastDiv((uint32_t)(c.d / V));
  a.fl = FastDiv((uint32_t)std::max(1, c.L));
  a.H = c.H, a.L = c.L, a.D = c.H * c.d;
  a.units = a.D / V;
  a.gpr = (c.d + 7) / 8;
  a.tokens = s.tokens, a.parts = s.parts;
  a.team = s.team, a.teams = s.teams, a.stages = s.stages, a.vecs = s.vecs;
  a.post = c.post, a.norm = c.norm, a.gate = c.gate, a.gate_batch = c.gate_batch;
  a.eps_post = c.eps_post, a.eps = c.eps, a.alpha = c.alpha, a.beta = c.beta;
  a.inv_d = 1.f / (float)a.D;
  a.drop_t = c.drop_t, a.drop_scale = c.drop_scale;
  a.key = PhiloxKeys(c.seed), a.offset = c.offset, a.counter = c.counter;
  a.ctr_h = (uint64_t)c.L * a.gpr, a.ctr_b = c.H * a.ctr_h, a.ctr0 = c.slice0 * a.ctr_h;
  return a;
}

template <class T, bool BRANCH>
static SubShape fwd_shape(const SubCall& c) {
  using Z = FwdSize<T, BRANCH>;
  return sub_shape(c, {kFwdPer, 1, Z::kThreads, 1 + BRANCH + (c.gate == LSH_GATE_SIGMOID),
                       (BRANCH ? 2 : 1) * (c.b || c.bp ? 2 : 1), Z::kCtas, false});
}

cudaError_t launch_sub_fwd(const SubCall& c, cudaStream_t st) {
  const bool bf16 = c.dtype == LSH_BF16;
  const SubShape s = bf16 ? c.branch ? fwd_shape<__nv_bfloat16, true>(c)
                                     : fwd_shape<__nv_bfloat16, false>(c)
                     : c.branch ? fwd_shape<float, true>(c)
                                : fwd_shape<float, false>(c);
  const SubArgs a = sub_args(c, s);
  return bf16 ? sub_fwd_type<__nv_bfloat16>(c, a, s, st) : sub_fwd_type<float>(c, a, s, st);
}

namespace {

struct FinalArgs {
  const float* part;
  int D, groups, parts, vecs, norm, branch;
  const float *wp, *bp, *gv;
  int gate_batch;
  float *dgate, *dwp, *dbp, *dw, *db;
};

// Adds the CTAs' rows, in a fixed order. Block (x, y): COLS features, y = 0 the
// norm's pair, y = 1 the branch's; R = 512 / COLS threads a feature add rows i,
// i + R, ... of a group, all loads in flight, then a warp's, then the warps in
// order. 8 features (one sector) below 2048, so that there are blocks for the
// SMs (a norm's backward of 64K tokens of 512 features 49.8 us, 51.9 with 32);
// 32 from there, where 8 make several waves of blocks of a few loads each (8192
// tokens of 4096 with a branch: 125 us, 128 with 8).
constexpr int kFinalThreads = 512, kFinalWarps = kFinalThreads / 32, kFinalWide = 2048;
template <int COLS>
__global__ void __launch_bounds__(kFinalThreads)
sub_final_kernel(const __grid_constant__ FinalArgs a) {
  __shared__ float buf[2][kFinalWarps][COLS];
  constexpr int kRows = kFinalThreads / COLS;
  stream_wait();
  let_next_start();
  const int col = threadIdx.x % COLS, i = threadIdx.x / COLS;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * COLS + col;
  const bool on = c < a.D;
  const bool branch = a.norm ? blockIdx.y == 1 : true;
  const int v0 = branch && a.norm ? 2 : 0;
  const int64_t row = (int64_t)a.vecs * a.D;
  // Few groups: one after the other, kRows threads a feature each. Many (a gate
  // for each of 16 sequences or more): a warp takes every 16th group, which
  // has few rows then, with four threads a feature.
  const bool many = a.groups >= kFinalWarps;
  const int lanes = many ? kRows / kFinalWarps : kRows;
  float t1 = 0.f, t0 = 0.f;   // totals over the groups
  for (int g = many ? w : 0; g < a.groups; g += many ? kFinalWarps : 1) {
    float s1 = 0.f, s0 = 0.f;
    if (on) {
      const float* r = a.part + (int64_t)g * a.parts * row + v0 * a.D + c;
#pragma unroll 8
      for (int p = i % lanes; p < a.parts; p += lanes) {
        s1 += r[p * row];
        s0 += r[p * row + a.D];
      }
    }
#pragma unroll
    for (int o = COLS; o < 32; o <<= 1) {
      s1 += __shfl_xor_sync(0xffffffffu, s1, o);
      s0 += __shfl_xor_sync(0xffffffffu, s0, o);
    }
    if (!many) {
      __syncthreads();
      if (lane < COLS) {
        buf[0][w][col] = s1;
        buf[1][w][col] = s0;
      }
      __syncthreads();
      s1 = s0 = 0.f;
#pragma unroll
      for (int k = 0; k < kFinalWarps; ++k) {
        s1 += buf[0][k][col];
        s0 += buf[1][k][col];
      }
    }
    if (branch && on) {
      const float gate = a.gv ? a.gv[(a.gate_batch ? (int64_t)g * a.D : 0) + c] : 1.f;
      if (a.dgate && lane < COLS && (many || w == 0))
        a.dgate[(int64_t)g * a.D + c] =
            (a.wp ? a.wp[c] : 1.f) * s1 + (a.bp ? a.bp[c] * s0 : 0.f);
      t1 = fmaf(gate, s1, t1);
      t0 = fmaf(gate, s0, t0);
    } else {
      t1 += s1;
      t0 += s0;
    }
  }
  if (many) {
    __syncthreads();
    if (lane < COLS) {
      buf[0][w][col] = t1;
      buf[1][w][col] = t0;
    }
    __syncthreads();
    t1 = t0 = 0.f;
#pragma unroll
    for (int k = 0; k < kFinalWarps; ++k) {
      t1 += buf[0][k][col];
      t0 += buf[1][k][col];
    }
  }
  if (i == 0 && on) {
    float* o1 = branch ? a.dwp : a.dw;
    float* o0 = branch ? a.dbp : a.db;
    if (o1) o1[c] = t1;
    if (o0) o0[c] = t0;
  }
}

template <class T, bool SIG>
cudaError_t run_bwd(const SubCall& c, const SubArgs& a, const SubShape& s, cudaStream_t st) {
  return c.norm != LSH_NORM_NONE ? sub_bwd_type<T, true, SIG>(c, a, s, st)
                                 : sub_bwd_type<T, false, SIG>(c, a, s, st);
}

template <class T, bool SIG>
SubShape bwd_shape(const SubCall& c, int tensors) {
  using Z = BwdSize<T, SIG>;
  const int norm = c.norm != LSH_NORM_NONE;
  return sub_shape(c, {kBwdPer, Z::kTok, Z::kThreads, tensors, norm + c.branch + (SIG && c.bp),
                       Z::kCtas, true});
}

}  // namespace

size_t sub_bwd_ws_bytes(int B, int H, int L, int d, bool branch, bool gate_batch) {
  // no call's kernel has more CTAs than this, whatever its layout
  const int D = H * d, groups = gate_batch ? B : 1;
  const int64_t tokens = gate_batch ? L : (int64_t)B * L;
  const int64_t parts = std::min<int64_t>(tokens, max_parts(kMaxParts, groups));
  return align_up((size_t)groups * parts * (branch ? 4 : 2) * D * 4, 256);
}

cudaError_t launch_sub_bwd(const SubCall& c, void* ws, cudaStream_t st) {
  const bool norm = c.norm != LSH_NORM_NONE;
  const int tensors = 2 * norm + (c.dy != nullptr) + c.branch + (c.gate == LSH_GATE_SIGMOID);
  const bool sig = c.gate == LSH_GATE_SIGMOID, bf16 = c.dtype == LSH_BF16;
  const SubShape s = bf16 ? sig ? bwd_shape<__nv_bfloat16, true>(c, tensors)
                                : bwd_shape<__nv_bfloat16, false>(c, tensors)
                     : sig ? bwd_shape<float, true>(c, tensors)
                           : bwd_shape<float, false>(c, tensors);
  SubArgs a = sub_args(c, s);
  const bool sums = c.dgate || c.dwp || c.dbp || c.dw || c.db;
  a.part = sums ? (float*)ws : nullptr;
  if ((int64_t)c.B * c.L == 0 && !sums) return cudaSuccess;
  if ((int64_t)c.B * c.L > 0) {
    cudaError_t e;
    e = bf16 ? sig ? run_bwd<__nv_bfloat16, true>(c, a, s, st)
                   : run_bwd<__nv_bfloat16, false>(c, a, s, st)
        : sig ? run_bwd<float, true>(c, a, s, st)
              : run_bwd<float, false>(c, a, s, st);
    if (e != cudaSuccess || !sums) return e;
  }
  FinalArgs f{};
  f.part = a.part;
  f.D = a.D, f.groups = s.groups, f.parts = s.parts;
  f.norm = norm, f.branch = c.branch;
  f.vecs = 2 * (f.norm + f.branch);
  f.wp = c.wp, f.bp = c.bp, f.gv = a.gv, f.gate_batch = c.gate_batch;
  f.dgate = c.dgate, f.dwp = c.dwp, f.dbp = c.dbp, f.dw = c.dw, f.db = c.db;
  note_launch();
  const int cols = a.D < kFinalWide ? 8 : 32;
  return launch_overlapped(cols == 8 ? sub_final_kernel<8> : sub_final_kernel<32>,
                           dim3((unsigned)((a.D + cols - 1) / cols),
                                (unsigned)(f.norm + f.branch)),
                           kFinalThreads, 0, st, f);
}

}  // namespace lsh
