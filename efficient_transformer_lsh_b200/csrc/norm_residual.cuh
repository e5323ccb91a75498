// Norms before and after a sublayer, its gate, dropout and residual add: what
// the forward and backward kernels share.
//
//   forward   u = post(f) (or f);  y = beta x + alpha drop(gate u);  h = norm(y)
//   backward  T = dy + r (a - [LayerNorm] mean a - yhat mean(a yhat)), a = dh w
//             dx = beta T;  q = alpha drop(T);  du = q gate;  df = post's
//             backward of du, the same expression with f's statistics
//
// A norm without a branch is the case y = x that is not stored (forward) and
// T = dres + ... (backward): the same two kernels.
//
// Every activation is read once and written once: a team of threads holds a
// token's features in registers, PER a thread, and a row's sums are shuffles
// (plus one exchange through shared memory per sum for teams of several
// warps). Statistics take two passes over the registers (mean, then squared
// deviations): one pass of sums of squares would lose what a mean far from
// zero leaves.
//
// The bound is HBM where the copies of coming tokens are in flight while a
// token is computed: each thread copies its own features of each input of the
// next tokens to a ring in shared memory (cp.async, 16 bytes a copy) and reads
// them back itself, so the ring needs no barrier. Beyond that it is latency: a
// token's dependent steps (statistics, shuffles, shared memory) at the few warps
// that the registers leave, with issue slots about half used. Fewer steps help:
// arithmetic runs on pairs (fma.rn.f32x2 and its like), and
// teams are as small as registers allow (16 threads for 512 features), so that
// addresses, shuffles and statistics, which cost the same for any team of at
// most a warp, serve several tokens at once.
#pragma once

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "sublayer.cuh"
#include "sublayer.h"

namespace lsh {

constexpr int kMaxWarps = 16;     // of a team
constexpr int kNarrowPer = 16;    // features a thread of the element-wise kernels
constexpr int kMaxStages = 4;
constexpr int kSms = 148;
constexpr int kSmemPerSm = 226 * 1024;
constexpr int kSmemDefault = 48 * 1024;   // of a CTA without asking for more

// Strides in elements and, for the kernels that move vectors of 16 bytes, of
// batch and token in such vectors: 32-bit factors of one multiplication each.
struct SubLayout {
  lsh_strides s;
  uint32_t b, l;
};

struct SubArgs {
  const void *x, *f, *z, *dy, *dh;
  void *y, *h, *dx, *df, *dz;
  const float *wp, *bp, *gv, *w, *b;
  float* part;
  SubLayout sx, sf, sh;
  FastDiv upr, fl;        // vectors of a head row; L
  int H, L, D, units, gpr;
  int tokens, parts;      // tokens of a group; CTAs of a group
  int team, teams;        // threads of a team; teams of a CTA
  int stages, vecs;       // of the ring; parameter vectors in shared memory
  int post, norm, gate, gate_batch;
  float eps_post, eps, alpha, beta, inv_d;
  uint32_t drop_t;
  float drop_scale;
  PhiloxKeys key;
  uint64_t offset;
  const uint64_t* counter;
  uint64_t ctr0, ctr_b, ctr_h;   // dropout groups before the first row; of a batch; of a head
};

// ---- pairs of floats in one 64-bit register pair ----
using f2 = unsigned long long;
__device__ __forceinline__ f2 pk(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 up(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float both(f2 v) {
  const float2 u = up(v);
  return u.x + u.y;
}

// Sums over a thread's features.
template <int N>
__device__ __forceinline__ float sum_all(const f2 (&v)[N]) {
  f2 a = v[0], b = v[1];
#pragma unroll
  for (int i = 2; i < N; i += 2) a = add2(a, v[i]), b = add2(b, v[i + 1]);
  return both(add2(a, b));
}
template <int N>
__device__ __forceinline__ float dot_all(const f2 (&u)[N], const f2 (&v)[N]) {
  f2 a = mul2(u[0], v[0]), b = mul2(u[1], v[1]);
#pragma unroll
  for (int i = 2; i < N; i += 2) a = fma2(u[i], v[i], a), b = fma2(u[i + 1], v[i + 1], b);
  return both(add2(a, b));
}
template <int N>
__device__ __forceinline__ void scale_all(f2 (&v)[N], float m) {
  const f2 k = pk(m, m);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = mul2(v[i], k);
}

// g = 1 / (1 + exp(-z)); slope = g (1 - g), without the cancellation in 1 - g.
// For z < 0 the exponential's relative error is the gate's, for either sign the
// slope's. The approximate one is off by 2 + floor(1.173 |z|) units of 2^-23
// (the programming guide's bound): 2^-16 where exp(-|z|) is last a normal number,
// far below a bf16 result's 2^-8. float32 results take expf, right to two units
// at any z (everything on, forward and backward: 32K tokens of 512 features 62.4
// and 96.9 us, 60.9 and 96.3 with the approximate one; 8192 of 4096 250 and 488,
// 224 and 475); in bf16 it would cost more (64K of 512: 77 and 127 us, 69.8 and
// 120 with the approximate one). The approximate quotient is right to two units
// (its divisor is in [1, 2]).
template <class T>
__device__ __forceinline__ float sigmoid(float z, float& slope) {
  const float e = sizeof(T) == 4 ? expf(-fabsf(z)) : __expf(-fabsf(z));
  const float i = __fdividef(1.f, 1.f + e);
  slope = e * i * i;
  return z >= 0.f ? i : e * i;
}

__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 u;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "r"(at)
               : "memory");
  return u;
}
__device__ __forceinline__ void sts16(uint32_t at, uint4 u) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(u.x), "r"(u.y), "r"(u.z),
               "r"(u.w)
               : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_wait_for(int pending) {
  switch (pending) {
    case 0: cp_wait<0>(); break;
    case 1: cp_wait<1>(); break;
    case 2: cp_wait<2>(); break;
    default: cp_wait<3>(); break;
  }
}

// The features and tokens of a thread, its ring and its parameters. Feature
// e = k V + i of a thread is element i of vector k `team` + lane of the token
// (V features; neighbouring threads hold neighbouring vectors); features past
// D (off) read as zero everywhere, parameters included. Vectors of 16 bytes
// (V = 8 or 4) go through the ring; V = 1 (odd sizes, unaligned arrays) loads
// element by element.
// Group g of a per-batch gate is batch g; otherwise the one group is all B L
// tokens in order. A team takes TOK neighbouring tokens at a time, so that
// parameters, flags and addresses are read once for them, and a warp's teams
// neighbouring ones; `live` is false for a token past the last, which a team
// only goes along with.
// TEAM: threads of a token up to a warp, or 0 or less: whole warps, a.team of
// them.
template <class T, int V, int PER, int TEAM, int TOK, int THREADS>
struct Place {
  static constexpr bool kMulti = TEAM <= 0;
  static constexpr int NV = PER / V;
  static constexpr int P = PER / 2;                          // pairs
  static constexpr bool kRing = V > 1;
  static constexpr int kSlots = PER * (int)sizeof(T) / 16;   // 16 bytes each
  static constexpr int kKeep = kRing ? NV : 1;
  static constexpr uint32_t kAll = (uint32_t)((1ull << NV) - 1);
  const SubArgs& a;
  int group, part, team_id, lane;   // lane: thread of the team
  int ox[kKeep], of[kKeep], oh[kKeep];   // a vector's place in a token, in vectors
  uint32_t on_bits, ring, par;
  float* red;
  int turn = 0;

  __device__ __forceinline__ Place(const SubArgs& args, unsigned char* smem) : a(args) {
    group = blockIdx.x / a.parts;
    part = blockIdx.x - group * a.parts;
    team_id = (int)threadIdx.x / team();
    lane = (int)threadIdx.x - team_id * team();
    on_bits = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (lane + k * team() < a.units) on_bits |= 1u << k;
    if constexpr (kRing) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        ox[k] = (int)(place(a.sx, k) / V);
        of[k] = (int)(place(a.sf, k) / V);
        oh[k] = (int)(place(a.sh, k) / V);
      }
    }
    par = (uint32_t)__cvta_generic_to_shared(smem) + lane * 16;
    unsigned char* p = smem + a.vecs * (PER / 4) * team() * 16;
    red = reinterpret_cast<float*>(p) + team_id * (16 * kMaxWarps);
    if (kMulti) p += a.teams * (64 * kMaxWarps);
    ring = (uint32_t)__cvta_generic_to_shared(p) + threadIdx.x * 16;
  }
  // bytes from a slot to the next, from a token's vectors of a tensor to the next
  __device__ __forceinline__ uint32_t slot() const {
    return kMulti ? blockDim.x * 16 : THREADS * 16;
  }
  __device__ __forceinline__ uint32_t one() const { return kSlots * slot(); }
  __device__ __forceinline__ int team() const { return kMulti ? a.team : TEAM; }
  __device__ __forceinline__ bool on(int k) const { return on_bits >> k & 1; }
  __device__ __forceinline__ int unit(int k) const { return on(k) ? lane + k * team() : 0; }
  __device__ __forceinline__ int feat(int k) const { return unit(k) * V; }
  __device__ __forceinline__ int head(int k) const { return (int)a.upr.div((uint32_t)unit(k)); }
  __device__ __forceinline__ int col(int k) const {
    return (unit(k) - head(k) * (int)a.upr.d) * V;
  }
  __device__ __forceinline__ int64_t place(const SubLayout& s, int k) const {
    return head(k) * s.s.h + col(k);
  }

  // ---- tokens ----
  __device__ __forceinline__ int first() const { return (part * a.teams + team_id) * TOK; }
  __device__ __forceinline__ int step() const { return a.parts * a.teams * TOK; }
  // Rounds that every team of a warp (of a CTA where one is the team) makes,
  // uniform over the warp.
  __device__ __forceinline__ int rounds() const {
    const int lead = __shfl_sync(0xffffffffu, first(), 0);
    return lead < a.tokens ? (a.tokens - 1 - lead) / step() + 1 : 0;
  }
  __device__ __forceinline__ void token(int t, int& b, int& l) const {
    if (a.gate_batch) {
      b = group;
      l = t;
    } else {
      b = (int)a.fl.div((uint32_t)t);
      l = t - b * a.L;
    }
  }
  // a token's place: in vectors for the ring's kernels, else in elements
  static __device__ __forceinline__ int64_t row(const SubLayout& s, int b, int l) {
    if constexpr (kRing) return (int64_t)((uint64_t)(uint32_t)b * s.b + (uint64_t)(uint32_t)l * s.l);
    return b * s.s.b + l * s.s.l;
  }

  // Sums of N values over the team, the same on each of its threads. Several
  // values share one butterfly: the first exchanges split the values between
  // the halves of the team instead of adding the same sums on both (for 2, 4,
  // 8 values 14, 22, 40 instructions a warp instead of 20, 40, 80). `red`
  // holds two buffers used in turn, so one barrier a call is enough.
  template <int N>
  __device__ __forceinline__ void team_sum(float (&v)[N]) {
    constexpr int W = kMulti ? 32 : TEAM;
    constexpr int S = N < W / 2 ? N : 1;   // values to split
    const unsigned all = 0xffffffffu;
    const int me = threadIdx.x & 31;
    if constexpr (S > 1) {
      float x[N];
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = v[i];
#pragma unroll
      for (int n = N / 2, o = W / 2; n > 0; n /= 2, o /= 2) {
        const bool upper = me & o;
#pragma unroll
        for (int i = 0; i < n; ++i) {
          const float keep = upper ? x[i + n] : x[i], send = upper ? x[i] : x[i + n];
          x[i] = keep + __shfl_xor_sync(all, send, o);
        }
      }
#pragma unroll
      for (int o = W / N / 2; o > 0; o >>= 1) x[0] += __shfl_xor_sync(all, x[0], o);
      if constexpr (kMulti) {
        v[0] = x[0];   // lane i W / N has value i
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __shfl_sync(all, x[0], i * (W / N), W);
      }
    } else {
#pragma unroll
      for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(all, v[i], o);
    }
    if constexpr (kMulti) {
      float* r = red + turn * (8 * kMaxWarps);
      turn ^= 1;
      const int nw = a.team >> 5;
      if ((me & (W / N - 1)) == 0) r[(lane >> 5) * N + me / (W / N)] = v[0];
      asm volatile("bar.sync %0, %1;" ::"r"(team_id + 1), "r"(a.team) : "memory");
      // the warps' values in order, two at a time where there are two
      if constexpr (N == 1) {
        v[0] = 0.f;
#pragma unroll 4
        for (int k = 0; k < nw; ++k) v[0] += r[k];
      } else {
        f2 s[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) s[i] = 0ull;
#pragma unroll 4
        for (int k = 0; k < nw; ++k)
#pragma unroll
          for (int i = 0; i < N / 2; ++i)
            s[i] = add2(s[i], *reinterpret_cast<const f2*>(r + k * N + 2 * i));
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          const float2 u = up(s[i]);
          v[2 * i] = u.x;
          v[2 * i + 1] = u.y;
        }
      }
    }
  }

  // ---- inputs ----
  // Off features' slots are cleared once and never written again.
  __device__ __forceinline__ void clear(uint32_t from, int tensors) const {
    if constexpr (kRing)
      for (int i = 0; i < tensors * kSlots; ++i)
        sts16(from + i * slot(), make_uint4(0u, 0u, 0u, 0u));
  }
  __device__ __forceinline__ void issue(const void* p, const int (&o)[kKeep], int64_t row,
                                        uint32_t at) const {
    const uint4* q = (const uint4*)p + row;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (on(k)) cp_async16(at + k * slot(), q + o[k]);
  }
  // `at`: the tensor's slots of this stage; V = 1: from memory.
  __device__ __forceinline__ void get(const void* p, const SubLayout& s, int b, int l, bool live,
                                      uint32_t at, f2 (&v)[P]) const {
    if constexpr (kRing) {
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        const uint4 u = lds16(at + j * slot());
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        if constexpr (sizeof(T) == 2) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[4 * j + i] =
                pk(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        } else {
          v[2 * j] = pk(__uint_as_float(w[0]), __uint_as_float(w[1]));
          v[2 * j + 1] = pk(__uint_as_float(w[2]), __uint_as_float(w[3]));
        }
      }
    } else {
      const T* q = (const T*)p + row(s, b, l);
      float e[PER];
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        Vec<T, 1> r;
        r.zero();
        if (live && on(k)) r.load(q + place(s, k));
        float one[1];
        r.get(one);
        e[k] = one[0];
      }
#pragma unroll
      for (int i = 0; i < P; ++i) v[i] = pk(e[2 * i], e[2 * i + 1]);
    }
  }

  // ---- outputs ----
  // Stores v; with BACK v becomes what was stored.
  template <bool BACK>
  __device__ __forceinline__ void put(void* p, const SubLayout& s, const int (&o)[kKeep],
                                      int b, int l, bool live, f2 (&v)[P]) const {
    T* q = kRing ? (T*)((uint4*)p + row(s, b, l)) : (T*)p + row(s, b, l);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float e[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 u = up(v[(k * V + i) / 2]);
        e[i] = (k * V + i) & 1 ? u.y : u.x;
      }
      Vec<T, V> r;
      r.set(e);
      if (live && on(k))
        r.store(kRing ? (T*)((uint4*)q + o[kRing ? k : 0]) : q + place(s, k));
      if (BACK && sizeof(T) == 2) {
        r.get(e);
        if constexpr (kRing) {
#pragma unroll
          for (int i = 0; i < V / 2; ++i) v[V / 2 * k + i] = pk(e[2 * i], e[2 * i + 1]);
        } else {
          const float2 u = up(v[k / 2]);
          v[k / 2] = k & 1 ? pk(u.x, e[0]) : pk(e[0], u.y);
        }
      }
    }
  }

  // ---- parameters ----
  // Features 4 j .. 4 j + 3 of the thread of p times q (absent: ones); 0 past D.
  __device__ __forceinline__ float4 param4(const float* p, const float* q, int j) const {
    if constexpr (kRing) {
      const int at = feat(4 * j / V) + 4 * j % V;
      float4 u = make_float4(1.f, 1.f, 1.f, 1.f);
      if (p) u = *reinterpret_cast<const float4*>(p + at);
      if (q) {
        const float4 w = *reinterpret_cast<const float4*>(q + at);
        u = make_float4(u.x * w.x, u.y * w.y, u.z * w.z, u.w * w.w);
      }
      return on(4 * j / V) ? u : make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
      float e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = 4 * j + i;
        e[i] = p ? p[feat(k)] : 1.f;
        if (q) e[i] *= q[feat(k)];
        if (!on(k)) e[i] = 0.f;
      }
      return make_float4(e[0], e[1], e[2], e[3]);
    }
  }
  // Parameters sit in shared memory as [vector][PER / 4][team] groups of four.
  __device__ __forceinline__ void stage_param(int vec, const float* p, const float* q) const {
    // the teams of the CTA share the groups out
    for (int j = team_id; j < PER / 4; j += a.teams) {
      const float4 u = param4(p, q, j);
      sts16(par + (vec * (PER / 4) + j) * team() * 16,
            make_uint4(__float_as_uint(u.x), __float_as_uint(u.y), __float_as_uint(u.z),
                       __float_as_uint(u.w)));
    }
  }
  __device__ __forceinline__ void params(int vec, int j, f2& lo, f2& hi) const {
    const uint4 u = lds16(par + (vec * (PER / 4) + j) * team() * 16);
    lo = pk(__uint_as_float(u.x), __uint_as_float(u.y));
    hi = pk(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  template <int N>
  __device__ __forceinline__ void scale_by(int vec, f2 (&v)[N][P]) const {
#pragma unroll
    for (int j = 0; j < PER / 4; ++j) {
      f2 lo, hi;
      params(vec, j, lo, hi);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        v[n][2 * j] = mul2(v[n][2 * j], lo);
        v[n][2 * j + 1] = mul2(v[n][2 * j + 1], hi);
      }
    }
  }
  template <int N>
  __device__ __forceinline__ void shift_by(int vec, f2 (&v)[N][P]) const {
#pragma unroll
    for (int j = 0; j < PER / 4; ++j) {
      f2 lo, hi;
      params(vec, j, lo, hi);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        v[n][2 * j] = add2(v[n][2 * j], lo);
        v[n][2 * j + 1] = add2(v[n][2 * j + 1], hi);
      }
    }
  }

  // v = v p + q
  template <int N>
  __device__ __forceinline__ void scale_shift(int vp, int vq, f2 (&v)[N][P]) const {
#pragma unroll
    for (int j = 0; j < PER / 4; ++j) {
      f2 lo, hi, blo, bhi;
      params(vp, j, lo, hi);
      params(vq, j, blo, bhi);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        v[n][2 * j] = fma2(v[n][2 * j], lo, blo);
        v[n][2 * j + 1] = fma2(v[n][2 * j + 1], hi, bhi);
      }
    }
  }

  // ---- dropout: kept values times m, others 0 ----
  __device__ __forceinline__ void drop_all(uint64_t offset, int b, int l, float m,
                                           f2 (&v)[P]) const {
    const uint64_t first = a.ctr0 + (uint32_t)b * a.ctr_b + (uint64_t)(uint32_t)l * (uint32_t)a.gpr;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float e[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 u = up(v[(k * V + i) / 2]);
        e[i] = (k * V + i) & 1 ? u.y : u.x;
      }
      const int c = col(k);
      const uint64_t n = first + (uint32_t)head(k) * a.ctr_h + (uint32_t)c / 8;
      drop<V>(e, philox(a.key, n, offset), c, a.drop_t);
      if constexpr (kRing) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) v[V / 2 * k + i] = pk(e[2 * i], e[2 * i + 1]);
      } else {
        const float2 u = up(v[k / 2]);
        v[k / 2] = k & 1 ? pk(u.x, e[0]) : pk(e[0], u.y);
      }
    }
    scale_all(v, m);
  }
  // Features of the thread that exist.
  __device__ __forceinline__ float count() const { return (float)(__popc(on_bits) * V); }
  // v - m on the features that exist, 0 elsewhere
  __device__ __forceinline__ void center(f2 (&v)[P], float m) const {
    if constexpr (kRing) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const float n = on(k) ? -m : 0.f;
        const f2 d = pk(n, n);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) v[V / 2 * k + i] = add2(v[V / 2 * k + i], d);
      }
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i)
        v[i] = add2(v[i], pk(on(2 * i) ? -m : 0.f, on(2 * i + 1) ? -m : 0.f));
    }
  }
};

// 1 / sqrt(v): the approximation and one Newton step, r (3 - v r^2) / 2
__device__ __forceinline__ float inv_std(float sum_sq, float inv_d, float eps) {
  const float v = fmaf(sum_sq, inv_d, eps), r = rsqrtf(v);
  const float e = fmaf(-v * r, r, 1.f);
  return isinf(v) ? r : fmaf(0.5f * r, e, r);
}

// How a problem is laid over the GPU, with `ctas` CTAs of an SM resident where
// two ring stages of each fit, else fewer. `wide` goes by room and reach too:
// one stage has to fit (all but the float32 backward of more than 7168 features
// with dy, a sigmoid gate, b_post and a norm of y), a token's vectors have to
// lie within 2^31 vectors of its first, and strides below 2^32 vectors.
struct SubShape {
  int per, team, teams, threads, tok, groups, tokens, parts, stages, vecs, smem;
  bool wide;
};
struct SubSize {
  int per, tok, threads, tensors, vecs, ctas;   // of the wide kernel
  bool backward;
};
SubShape sub_shape(const SubCall& c, const SubSize& z);
SubArgs sub_args(const SubCall& c, const SubShape& s);

// Calls f with the team size as a compile-time constant.
template <class F>
cudaError_t with_team(int team, F f) {
  switch (team) {
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
    case 8: return f(std::integral_constant<int, 8>());
    case 16: return f(std::integral_constant<int, 16>());
    case 32: return f(std::integral_constant<int, 32>());
    default: return f(std::integral_constant<int, 0>());
  }
}

// Features a thread, tokens a team, threads of a CTA of several teams and CTAs
// of an SM, for the wide kernels. Forward: 32 features, so that a warp takes
// two tokens of 512. Backward: the four sums of parameter gradients already
// take four registers a feature, so 16 features, and a few warps with all the
// registers they can use, rather than more that spill (64K tokens of 512
// features with everything on: bf16 with two tokens at a time 94 us at 255
// registers, 2 x 128 threads an SM, 109 at 168, 3 x 128; float32 with one token
// 75 for 32K at 255 registers, 80 at 168, 98 at 128). A sigmoid gate's kernel
// takes one token and 168 registers (111 us; 133 at 128, 118 at 255).
constexpr int kFwdPer = 32;
template <class T, bool BRANCH>
struct FwdSize {
  // bf16 with a branch: four CTAs of 128 threads rather than two of 256 (64K
  // tokens of 512 features 52.9 us, 56; float32 prefers the two: 32K
  // tokens 49.8 us, 52.7 with three of 128)
  static constexpr bool kSmall = BRANCH && sizeof(T) == 2;
  static constexpr int kThreads = kSmall ? 128 : 256;
  static constexpr int kCtas = kSmall ? 4 : BRANCH ? 2 : 3;
};
// Teams of several warps, forward: one large CTA an SM, whose teams share the
// parameters in shared memory (64 KB of them for 4096 features).
constexpr int kFwdBig = 512;
constexpr int kBwdPer = 16;
constexpr int kNarrowThreads = 256;
template <class T, bool SIG>
struct BwdSize {
  static constexpr int kTok = sizeof(T) == 2 && !SIG ? 2 : 1;
  static constexpr int kThreads = 128;
  static constexpr int kCtas = SIG ? 3 : 2;
};

// Rows wider than 512 features in the backward. A norm's own (two sums a
// feature, not four) holds 32 features a thread at any width, and so does
// bf16 with a branch up to 1024, where that makes a warp of a token (2 x 12288
// tokens of 1024 features: 75 us; 96 with two warps of 16 features a thread).
// Wider ones take several warps of 16: 168 registers up to 192 threads (12288
// tokens of 2048 features: 80 us; 92 with 32 features a thread, 100 at 128
// registers). Past that, bf16 has 32 features a thread again (8192 tokens of
// 4096: 125 us; 143 with 16 at 128 registers), float32 and sigmoid gates 16 at
// 128 registers for two teams an SM (with 32, before there were two: float32
// as fast, a sigmoid gate's 344 us where this was 302).
constexpr int kBwdWidePer = 32, kBwdWarpMax = 1024;
constexpr int kBwdRoom = 256;                           // threads an SM at 255 registers
constexpr int kBwdTeam = 192, kBwdTeamRoom = 384;       // at 168
constexpr int kBwdBigRoom = 512;                        // at 128
constexpr int kBig = -1;                                // TEAM of the last
template <class T, int V, int PER, int TEAM, bool SIG>
constexpr int bwd_threads() {
  if (V == 1) return TEAM != 0 ? kNarrowThreads : 32 * kMaxWarps;
  if (PER == kBwdWidePer) return kBwdRoom;
  return TEAM == kBig ? kBwdBigRoom : TEAM == 0 ? kBwdTeam : BwdSize<T, SIG>::kThreads;
}
template <class T, int V, int PER, int TEAM, bool SIG>
constexpr int bwd_ctas() {
  if (V == 1) return TEAM != 0 ? 2 : 1;
  if (PER == kBwdWidePer || TEAM == kBig) return 1;
  return TEAM == 0 ? kBwdTeamRoom / kBwdTeam : BwdSize<T, SIG>::kCtas;
}

template <class T>
cudaError_t sub_fwd_type(const SubCall& c, const SubArgs& a, const SubShape& s, cudaStream_t st);
template <class T, bool NORM, bool SIG>
cudaError_t sub_bwd_type(const SubCall& c, const SubArgs& a, const SubShape& s, cudaStream_t st);

// CTAs of a call, and so rows of partial sums of a backward one, at most.
constexpr int kMaxParts = 4 * kSms;

}  // namespace lsh
