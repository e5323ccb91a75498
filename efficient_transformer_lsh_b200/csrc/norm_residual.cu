// Norms before and after a sublayer, its gate, dropout and residual add.
//
//   forward   u = post(f) (or f);  y = beta x + alpha drop(gate u);  h = norm(y)
//   backward  T = dy + r (a - [LayerNorm] mean a - yhat mean(a yhat)), a = dh w
//             dx = beta T;  q = alpha drop(T);  du = q gate;  df = post's
//             backward of du, the same expression with f's statistics
//
// A norm without a branch is the case y = x that is not stored (forward) and
// T = dres + ... (backward): the same two kernels.
//
// One warp holds a token of up to 512 features (16 a lane) in registers, one
// CTA of up to 512 threads a wider one, so that every activation is read once
// and written once and a row's sums are shuffles (plus one shared-memory
// exchange per sum for CTAs). Statistics take two passes over the registers
// (mean, then squared deviations): one pass of sums of squares would lose
// what a mean far from zero leaves. The backward recomputes them from the
// stored row, which it reads anyway.
//
// Parameter gradients are sums over tokens. Every thread keeps its features'
// sums in registers over all the tokens it visits; a CTA writes one row of
// partial sums, and a second kernel adds the rows in order: no atomics, the
// same result every time. Four sums suffice, per group of tokens that shares
// a gate vector: A = sum dh yhat, B = sum dh, S1 = sum q fhat, S0 = sum q
// (q before the gate; du for a sigmoid gate):
//   dw = A, db = B, dw_post = gate S1, db_post = gate S0,
//   dgate = w_post S1 + b_post S0.
#include <algorithm>

#include "internal.h"
#include "sublayer.cuh"
#include "sublayer.h"

namespace lsh {
namespace {

constexpr int kPer = 16;          // features a thread holds
constexpr int kWarps = 8;         // warps of a CTA in the warp-per-token form
constexpr int kMaxThreads = kNormMaxD / kPer;
constexpr int kMaxCtaWarps = kMaxThreads / 32;
constexpr int kFwdWarps = 148 * 32;   // warps that fill the GPU
constexpr int kBwdCtas = 296;

struct SubArgs {
  const void *x, *f, *z, *dy, *dh;
  void *y, *h, *dx, *df, *dz;
  const float *wp, *bp, *gv, *w, *b;
  float* part;
  lsh_strides sx, sf, sh;
  FastDiv upr, fl;        // vectors of a head row; L
  int H, L, D, units, gpr;
  int tokens, parts;      // tokens of a group; CTAs of a group
  int post, norm, gate, gate_batch;
  float eps_post, eps, alpha, beta, inv_d;
  uint32_t drop_t;
  float drop_scale;
  uint64_t seed, offset;
  const uint64_t* counter;
  int64_t slice0;
};

// Sums of N values over the token's threads, the same on each of them. `red`
// holds two buffers used in turn, so one barrier a call is enough.
template <int N, bool CTA>
__device__ __forceinline__ void token_sum(float (&v)[N], float* red, int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if constexpr (CTA) {
    float* r = red + turn * (2 * kMaxCtaWarps);
    turn ^= 1;
    const int nw = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) r[i * kMaxCtaWarps + (threadIdx.x >> 5)] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.f;
      for (int k = 0; k < nw; ++k) s += r[i * kMaxCtaWarps + k];
      v[i] = s;
    }
  }
}

// v -> xhat; returns r.
template <int V, int NV, bool CTA>
__device__ __forceinline__ float normalize(float (&v)[NV][V], const bool (&on)[NV], int kind,
                                           float inv_d, float eps, float* red, int& turn) {
  if (kind == LSH_NORM_LAYER) {
    float m[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) m[0] += v[k][i];
    token_sum<1, CTA>(m, red, turn);
    const float mean = m[0] * inv_d;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] = on[k] ? v[k][i] - mean : 0.f;
  }
  float s[1] = {0.f};
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) s[0] = fmaf(v[k][i], v[k][i], s[0]);
  token_sum<1, CTA>(s, red, turn);
  const float r = 1.f / sqrtf(fmaf(s[0], inv_d, eps));
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) v[k][i] *= r;
  return r;
}

// g = 1 / (1 + exp(-z)); slope = g (1 - g), without the cancellation in 1 - g.
__device__ __forceinline__ float sigmoid(float z, float& slope) {
  const float e = expf(-fabsf(z)), i = 1.f / (1.f + e);
  slope = e * i * i;
  return z >= 0.f ? i : e * i;
}

// The token and feature a thread works on. Group g of a per-batch gate is
// batch g; otherwise the one group is all B L tokens in order.
template <class T, int V, int NV>
struct Place {
  bool on[NV];
  int feat[NV], head[NV], c[NV];
  int b, l;

  __device__ __forceinline__ void units(const SubArgs& a, int first, int step) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int u = first + k * step;
      on[k] = u < a.units;
      const int uu = on[k] ? u : 0;
      head[k] = (int)a.upr.div((uint32_t)uu);
      c[k] = (uu - head[k] * (int)a.upr.d) * V;
      feat[k] = uu * V;
    }
  }
  __device__ __forceinline__ void token(const SubArgs& a, int group, int t) {
    if (a.gate_batch) {
      b = group;
      l = t;
    } else {
      b = (int)a.fl.div((uint32_t)t);
      l = t - b * a.L;
    }
  }
  __device__ __forceinline__ int64_t off(const lsh_strides& s, int k) const {
    return b * s.b + head[k] * s.h + l * s.l + c[k];
  }
  __device__ __forceinline__ void load(const void* p, const lsh_strides& s, Vec<T, V> (&r)[NV]) const {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (on[k]) r[k].load((const T*)p + off(s, k));
      else r[k].zero();
    }
  }
  __device__ __forceinline__ void store(void* p, const lsh_strides& s, const Vec<T, V> (&r)[NV]) const {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (on[k]) r[k].store((T*)p + off(s, k));
  }
  __device__ __forceinline__ void drop_all(const SubArgs& a, const Philox& rng, float (&v)[NV][V]) const {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const uint64_t row = (uint64_t)((a.slice0 + (int64_t)b * a.H + head[k]) * a.L + l);
      drop<V>(v[k], rng, row * (uint32_t)a.gpr, c[k], a.drop_t, a.drop_scale);
    }
  }
};

template <class T, int V, int NV>
__device__ __forceinline__ void get_all(const Vec<T, V> (&r)[NV], float (&v)[NV][V]) {
#pragma unroll
  for (int k = 0; k < NV; ++k) r[k].get(v[k]);
}
template <class T, int V, int NV>
__device__ __forceinline__ void set_all(Vec<T, V> (&r)[NV], const float (&v)[NV][V]) {
#pragma unroll
  for (int k = 0; k < NV; ++k) r[k].set(v[k]);
}
// out = v * w + b with absent parameters as ones and zeros.
template <int V, int NV>
__device__ __forceinline__ void affine(float (&v)[NV][V], const int (&feat)[NV], const float* w,
                                       const float* b) {
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    float p[V];
    if (w) {
      load_params<V>(w + feat[k], p);
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] *= p[i];
    }
    if (b) {
      load_params<V>(b + feat[k], p);
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] += p[i];
    }
  }
}

template <class T, int V, bool CTA, bool BRANCH>
__global__ void __launch_bounds__(CTA ? kMaxThreads : 32 * kWarps)
sub_fwd_kernel(const __grid_constant__ SubArgs a) {
  constexpr int NV = kPer / V;
  __shared__ float red[CTA ? 4 * kMaxCtaWarps : 1];
  int turn = 0;
  const int group = blockIdx.x / a.parts, part = blockIdx.x - group * a.parts;
  const int first = CTA ? part : part * kWarps + (threadIdx.x >> 5);
  const int step = CTA ? a.parts : a.parts * kWarps;
  Place<T, V, NV> at;
  at.units(a, CTA ? threadIdx.x : threadIdx.x & 31, CTA ? blockDim.x : 32);
  const Philox rng(a.seed, a.offset + (a.counter ? __ldg(a.counter) : 0));
  const float* gv = a.gv ? a.gv + (int64_t)group * (a.gate_batch ? a.D : 0) : nullptr;
  for (int t = first; t < a.tokens; t += step) {
    at.token(a, group, t);
    Vec<T, V> xr[NV];
    float v[NV][V];
    at.load(a.x, a.sx, xr);
    if constexpr (BRANCH) {
      Vec<T, V> fr[NV];
      at.load(a.f, a.sf, fr);
      get_all<T, V, NV>(fr, v);
      if (a.post != LSH_NORM_NONE) {
        normalize<V, NV, CTA>(v, at.on, a.post, a.inv_d, a.eps_post, red, turn);
        affine<V, NV>(v, at.feat, a.wp, a.bp);
      }
      if (a.gate == LSH_GATE_VECTOR) {
        affine<V, NV>(v, at.feat, gv, nullptr);
      } else if (a.gate == LSH_GATE_SIGMOID) {
        float z[NV][V];
        at.load(a.z, a.sf, fr);
        get_all<T, V, NV>(fr, z);
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float slope;
            v[k][i] *= sigmoid(z[k][i], slope);
          }
      }
      if (a.drop_t) at.drop_all(a, rng, v);
      float x[NV][V];
      get_all<T, V, NV>(xr, x);
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i)
          v[k][i] = at.on[k] ? fmaf(a.alpha, v[k][i], a.beta * x[k][i]) : 0.f;
      set_all<T, V, NV>(xr, v);
      at.store(a.y, a.sx, xr);
      if (a.norm == LSH_NORM_NONE) continue;
    }
    // the row as stored: h is the same whether it comes from here or from a
    // later pass over y
    get_all<T, V, NV>(xr, v);
    normalize<V, NV, CTA>(v, at.on, a.norm, a.inv_d, a.eps, red, turn);
    affine<V, NV>(v, at.feat, a.w, a.b);
    set_all<T, V, NV>(xr, v);
    at.store(a.h, a.sh, xr);
  }
}

// v = (a - [LayerNorm] mean a - hat mean(a hat)) r + add
template <int V, int NV, bool CTA>
__device__ __forceinline__ void norm_back(float (&a)[NV][V], const float (&hat)[NV][V], int kind,
                                          float r, float inv_d, float* red, int& turn) {
  float s[2] = {0.f, 0.f};
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[0] += a[k][i];
      s[1] = fmaf(a[k][i], hat[k][i], s[1]);
    }
  token_sum<2, CTA>(s, red, turn);
  const float m0 = kind == LSH_NORM_LAYER ? s[0] * inv_d : 0.f, m1 = s[1] * inv_d;
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) a[k][i] = r * (a[k][i] - m0 - hat[k][i] * m1);
}

// Partial sums of a CTA: [rows of the grid][2 or 4][D], A B then S1 S0.
template <int V, int NV, bool CTA>
__device__ __forceinline__ void write_part(const float (&s)[NV][V], const int (&feat)[NV],
                                           const bool (&on)[NV], float* out, int D, float* buf) {
  if constexpr (CTA) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (on[k]) {
#pragma unroll
        for (int i = 0; i < V; ++i) out[feat[k] + i] = s[k][i];
      }
  } else {
    // warp w's sums in row w; the rows are added in order
    __syncthreads();
    float* row = buf + (threadIdx.x >> 5) * (32 * kPer);
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (on[k]) {
#pragma unroll
        for (int i = 0; i < V; ++i) row[feat[k] + i] = s[k][i];
      }
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += 32 * kWarps) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) t += buf[w * (32 * kPer) + c];
      out[c] = t;
    }
  }
}

template <class T, int V, bool CTA, bool BRANCH, bool NORM>
__global__ void __launch_bounds__(CTA ? kMaxThreads : 32 * kWarps)
sub_bwd_kernel(const __grid_constant__ SubArgs a) {
  constexpr int NV = kPer / V;
  __shared__ float red[CTA ? 4 * kMaxCtaWarps : kWarps * 32 * kPer];
  int turn = 0;
  const int group = blockIdx.x / a.parts, part = blockIdx.x - group * a.parts;
  const int first = CTA ? part : part * kWarps + (threadIdx.x >> 5);
  const int step = CTA ? a.parts : a.parts * kWarps;
  Place<T, V, NV> at;
  at.units(a, CTA ? threadIdx.x : threadIdx.x & 31, CTA ? blockDim.x : 32);
  const Philox rng(a.seed, a.offset + (a.counter ? __ldg(a.counter) : 0));
  const float* gv = a.gv ? a.gv + (int64_t)group * (a.gate_batch ? a.D : 0) : nullptr;
  float sa[NV][V], sb[NV][V], s1[NV][V], s0[NV][V];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) sa[k][i] = sb[k][i] = s1[k][i] = s0[k][i] = 0.f;

  for (int t = first; t < a.tokens; t += step) {
    at.token(a, group, t);
    Vec<T, V> r0[NV];
    float q[NV][V];   // T, then q, then du
    if constexpr (NORM) {
      Vec<T, V> r1[NV];
      float hat[NV][V];
      at.load(a.x, a.sx, r0);
      at.load(a.dh, a.sh, r1);
      get_all<T, V, NV>(r0, hat);
      get_all<T, V, NV>(r1, q);
      const float r = normalize<V, NV, CTA>(hat, at.on, a.norm, a.inv_d, a.eps, red, turn);
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          sa[k][i] = fmaf(q[k][i], hat[k][i], sa[k][i]);
          sb[k][i] += q[k][i];
        }
      affine<V, NV>(q, at.feat, a.w, nullptr);
      if (a.dy) at.load(a.dy, a.sx, r1);
      norm_back<V, NV, CTA>(q, hat, a.norm, r, a.inv_d, red, turn);
      if (a.dy) {
        float dy[NV][V];
        get_all<T, V, NV>(r1, dy);
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < V; ++i) q[k][i] += dy[k][i];
      }
    } else {
      at.load(a.dy, a.sx, r0);
      get_all<T, V, NV>(r0, q);
    }
    if (a.dx) {
      float o[NV][V];
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) o[k][i] = BRANCH ? a.beta * q[k][i] : q[k][i];
      set_all<T, V, NV>(r0, o);
      at.store(a.dx, a.sx, r0);
    }
    if constexpr (BRANCH) {
      float hat[NV][V], z[NV][V];
      const bool sig = a.gate == LSH_GATE_SIGMOID;
      at.load(a.f, a.sf, r0);
      get_all<T, V, NV>(r0, hat);
      if (sig) {
        at.load(a.z, a.sf, r0);
        get_all<T, V, NV>(r0, z);
      }
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) q[k][i] = at.on[k] ? q[k][i] * a.alpha : 0.f;
      if (a.drop_t) at.drop_all(a, rng, q);
      float r = 0.f;
      if (a.post != LSH_NORM_NONE)
        r = normalize<V, NV, CTA>(hat, at.on, a.post, a.inv_d, a.eps_post, red, turn);
      if (sig) {
        float u[NV][V];
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < V; ++i) u[k][i] = hat[k][i];
        if (a.post != LSH_NORM_NONE) affine<V, NV>(u, at.feat, a.wp, a.bp);
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float slope;
            const float g = sigmoid(z[k][i], slope);
            u[k][i] *= q[k][i] * slope;
            q[k][i] *= g;
          }
        if (a.dz) {
          set_all<T, V, NV>(r0, u);
          at.store(a.dz, a.sf, r0);
        }
      }
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          s1[k][i] = fmaf(q[k][i], hat[k][i], s1[k][i]);
          s0[k][i] += q[k][i];
        }
      if (a.gate == LSH_GATE_VECTOR) affine<V, NV>(q, at.feat, gv, nullptr);
      if (a.post != LSH_NORM_NONE) {
        affine<V, NV>(q, at.feat, a.wp, nullptr);
        norm_back<V, NV, CTA>(q, hat, a.post, r, a.inv_d, red, turn);
      }
      set_all<T, V, NV>(r0, q);
      at.store(a.df, a.sf, r0);
    }
  }
  if (a.part) {
    constexpr int kVecs = (NORM ? 2 : 0) + (BRANCH ? 2 : 0);
    float* out = a.part + (int64_t)blockIdx.x * kVecs * a.D;
    if constexpr (NORM) {
      write_part<V, NV, CTA>(sa, at.feat, at.on, out, a.D, red);
      write_part<V, NV, CTA>(sb, at.feat, at.on, out + a.D, a.D, red);
      out += 2 * (int64_t)a.D;
    }
    if constexpr (BRANCH) {
      write_part<V, NV, CTA>(s1, at.feat, at.on, out, a.D, red);
      write_part<V, NV, CTA>(s0, at.feat, at.on, out + a.D, a.D, red);
    }
  }
}

struct FinalArgs {
  const float* part;
  int D, groups, parts, vecs, norm, branch;
  const float *wp, *bp, *gv;
  int gate_batch;
  float *dgate, *dwp, *dbp, *dw, *db;
};

// Adds the CTAs' rows, in order. Block (x, y): 32 features, y = 0 the norm's
// pair, y = 1 the branch's; warp w of 32 adds rows w, w + 32, ... of a group,
// then warp 0 adds the warps' sums.
__global__ void __launch_bounds__(1024) sub_final_kernel(const FinalArgs a) {
  __shared__ float buf[2][32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const bool on = c < a.D;
  const bool branch = a.norm ? blockIdx.y == 1 : true;
  const int v0 = branch && a.norm ? 2 : 0;
  float t1 = 0.f, t0 = 0.f;   // warp 0: totals over the groups
  for (int g = 0; g < a.groups; ++g) {
    float s1 = 0.f, s0 = 0.f;
    if (on) {
      for (int p = w; p < a.parts; p += 32) {
        const float* r = a.part + ((int64_t)(g * (int64_t)a.parts + p) * a.vecs + v0) * a.D + c;
        s1 += __ldg(r);
        s0 += __ldg(r + a.D);
      }
    }
    buf[0][w][lane] = s1;
    buf[1][w][lane] = s0;
    __syncthreads();
    if (w == 0 && on) {
      s1 = s0 = 0.f;
      for (int k = 0; k < 32; ++k) {
        s1 += buf[0][k][lane];
        s0 += buf[1][k][lane];
      }
      if (branch) {
        const float gate = a.gv ? a.gv[(a.gate_batch ? (int64_t)g * a.D : 0) + c] : 1.f;
        if (a.dgate && (a.gate_batch || a.groups == 1))
          a.dgate[(int64_t)g * a.D + c] =
              (a.wp ? a.wp[c] : 1.f) * s1 + (a.bp ? a.bp[c] * s0 : 0.f);
        t1 = fmaf(gate, s1, t1);
        t0 = fmaf(gate, s0, t0);
      } else {
        t1 += s1;
        t0 += s0;
      }
    }
    __syncthreads();
  }
  if (w == 0 && on) {
    float* o1 = branch ? a.dwp : a.dw;
    float* o0 = branch ? a.dbp : a.db;
    if (o1) o1[c] = t1;
    if (o0) o0[c] = t0;
  }
}

struct Shape {
  bool cta;
  int threads, groups, tokens, parts;
};
Shape shape_of(int B, int H, int L, int d, bool gate_batch, int ctas) {
  Shape s;
  const int D = H * d;
  s.cta = D > 32 * kPer;
  s.threads = s.cta ? ((D + kPer - 1) / kPer + 31) / 32 * 32 : 32 * kWarps;
  s.groups = gate_batch ? B : 1;
  s.tokens = gate_batch ? L : B * L;
  const int64_t rows = s.cta ? s.tokens : (s.tokens + kWarps - 1) / kWarps;
  s.parts = (int)std::min<int64_t>(rows, std::max(1, ctas / std::max(1, s.groups)));
  return s;
}
int fwd_ctas(int D) { return kFwdWarps / (D > 32 * kPer ? (D + 32 * kPer - 1) / (32 * kPer) : kWarps); }

SubArgs args_of(const SubCall& c, const Shape& s) {
  SubArgs a{};
  const int V = c.wide ? 8 : 1;
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
  a.post = c.post, a.norm = c.norm, a.gate = c.gate, a.gate_batch = c.gate_batch;
  a.eps_post = c.eps_post, a.eps = c.eps, a.alpha = c.alpha, a.beta = c.beta;
  a.inv_d = 1.f / (float)a.D;
  a.drop_t = c.drop_t, a.drop_scale = c.drop_scale;
  a.seed = c.seed, a.offset = c.offset, a.counter = c.counter, a.slice0 = c.slice0;
  return a;
}

template <class T, int V, bool CTA>
void fwd_branch(const SubCall& c, const SubArgs& a, const Shape& s, cudaStream_t st) {
  const unsigned grid = (unsigned)(s.groups * (int64_t)s.parts);
  if (c.branch) sub_fwd_kernel<T, V, CTA, true><<<grid, s.threads, 0, st>>>(a);
  else sub_fwd_kernel<T, V, CTA, false><<<grid, s.threads, 0, st>>>(a);
}
template <class T, int V, bool CTA>
void bwd_branch(const SubCall& c, const SubArgs& a, const Shape& s, cudaStream_t st) {
  const unsigned grid = (unsigned)(s.groups * (int64_t)s.parts);
  if (!c.branch) sub_bwd_kernel<T, V, CTA, false, true><<<grid, s.threads, 0, st>>>(a);
  else if (c.norm) sub_bwd_kernel<T, V, CTA, true, true><<<grid, s.threads, 0, st>>>(a);
  else sub_bwd_kernel<T, V, CTA, true, false><<<grid, s.threads, 0, st>>>(a);
}
#define LSH_DISPATCH(fn, c, a, s, st)                                           \
  do {                                                                          \
    if ((c).dtype == LSH_BF16) {                                                \
      if ((c).wide) (s).cta ? fn<__nv_bfloat16, 8, true>(c, a, s, st)           \
                            : fn<__nv_bfloat16, 8, false>(c, a, s, st);         \
      else (s).cta ? fn<__nv_bfloat16, 1, true>(c, a, s, st)                    \
                   : fn<__nv_bfloat16, 1, false>(c, a, s, st);                  \
    } else {                                                                    \
      if ((c).wide) (s).cta ? fn<float, 8, true>(c, a, s, st)                   \
                            : fn<float, 8, false>(c, a, s, st);                 \
      else (s).cta ? fn<float, 1, true>(c, a, s, st)                            \
                   : fn<float, 1, false>(c, a, s, st);                          \
    }                                                                           \
  } while (0)

}  // namespace

cudaError_t launch_sub_fwd(const SubCall& c, cudaStream_t st) {
  const Shape s = shape_of(c.B, c.H, c.L, c.d, c.gate_batch, fwd_ctas(c.H * c.d));
  const SubArgs a = args_of(c, s);
  LSH_DISPATCH(fwd_branch, c, a, s, st);
  note_launch();
  return cudaGetLastError();
}

size_t sub_bwd_ws_bytes(int B, int H, int L, int d, bool branch, bool gate_batch) {
  const Shape s = shape_of(B, H, L, d, gate_batch, kBwdCtas);
  return align_up((size_t)s.groups * s.parts * (branch ? 4 : 2) * H * d * 4, 256);
}

cudaError_t launch_sub_bwd(const SubCall& c, void* ws, cudaStream_t st) {
  const Shape s = shape_of(c.B, c.H, c.L, c.d, c.gate_batch, kBwdCtas);
  SubArgs a = args_of(c, s);
  const bool sums = c.dgate || c.dwp || c.dbp || c.dw || c.db;
  a.part = sums ? (float*)ws : nullptr;
  if ((int64_t)c.B * c.L == 0 && !sums) return cudaSuccess;
  if ((int64_t)c.B * c.L > 0) {
    LSH_DISPATCH(bwd_branch, c, a, s, st);
    note_launch();
  }
  if (sums) {
    FinalArgs f{};
    f.part = a.part;
    f.D = a.D, f.groups = s.groups, f.parts = s.parts;
    f.norm = c.norm != LSH_NORM_NONE, f.branch = c.branch;
    f.vecs = 2 * (f.norm + f.branch);
    f.wp = c.wp, f.bp = c.bp, f.gv = a.gv, f.gate_batch = c.gate_batch;
    f.dgate = c.dgate, f.dwp = c.dwp, f.dbp = c.dbp, f.dw = c.dw, f.db = c.db;
    sub_final_kernel<<<dim3((unsigned)((a.D + 31) / 32), (unsigned)(f.norm + f.branch)), 1024, 0,
                       st>>>(f);
    note_launch();
  }
  return cudaGetLastError();
}

}  // namespace lsh
