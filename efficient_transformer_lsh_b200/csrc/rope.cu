// Rotary positions: pairs of a head row's features turned by position * freq.
//
// The angle is formed as a phase in turns, by the integer product position *
// turns modulo 2^64 (turns = freq / 2 pi as a 64-bit fraction): the integer
// wrap is the reduction modulo one turn, exact, so that only the table's
// rounding grows with the position (2^-65 of a turn each), where a float32
// product of position and frequency would lose the phase (0.03 rad at position
// 2^20). Its top 32 bits, signed, are half turns in [-1, 1).
//
// Sine and cosine of a (token, pair) serve every head: a thread keeps those
// of its pairs in registers and walks the heads, four rows in flight; with one
// or two heads it takes four or two tokens instead. bf16 takes the hardware's
// approximate sine and cosine (absolute error below 2^-21 on one turn, where
// a bf16 result is rounded at 2^-8 of its value), float32 the accurate ones.
//
// Bound by HBM: 33.5 M elements in bf16 take 23 us with 8 heads (134 MB, 5.8
// TB/s), 67 M with 2 heads 44 us (6.0 TB/s); with one head the angles, one for
// every two elements, still show (28.6 us).
#include <algorithm>

#include "internal.h"
#include "sublayer.cuh"
#include "sublayer.h"

namespace lsh {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;   // rows a thread has in flight

struct RopeArgs {
  const void* in;
  const float* add;        // the sum's second term
  void* out;
  lsh_strides si, so;
  const uint64_t* turns;
  const int32_t* pos;
  int64_t pos0;
  FastDiv fl, fu;          // L; vectors of a head row (pairs, then copies)
  int H, L, tokens, tile;  // tile: tokens of a CTA
  int half, rot, heads;    // rot / 2; heads of a CTA
  int pair_units, pos_batch;
  float amp, sign;
};

// P pairs of one unit: P low and P high features, or 2 P adjacent ones in one
// access. A single adjacent pair is two accesses, so that it needs no more
// than its elements' alignment.
template <class T, int P, bool INTER>
struct Pairs {
  static constexpr bool kJoined = INTER && P > 1;
  Vec<T, kJoined ? 2 * P : P> a;
  Vec<T, kJoined ? 1 : P> b;
  __device__ __forceinline__ void load(const T* p, int second) {
    a.load(p);
    if constexpr (!kJoined) b.load(p + second);
  }
  __device__ __forceinline__ void store(T* p, int second) const {
    a.store(p);
    if constexpr (!kJoined) b.store(p + second);
  }
  // firsts and seconds of the pairs (copied features: any split)
  __device__ __forceinline__ void get(float (&p)[P], float (&q)[P]) const {
    if constexpr (kJoined) {
      float v[2 * P];
      a.get(v);
#pragma unroll
      for (int i = 0; i < P; ++i) p[i] = v[2 * i], q[i] = v[2 * i + 1];
    } else {
      a.get(p);
      b.get(q);
    }
  }
  __device__ __forceinline__ void set(const float (&p)[P], const float (&q)[P]) {
    if constexpr (kJoined) {
      float v[2 * P];
#pragma unroll
      for (int i = 0; i < P; ++i) v[2 * i] = p[i], v[2 * i + 1] = q[i];
      a.set(v);
    } else {
      a.set(p);
      b.set(q);
    }
  }
  __device__ __forceinline__ void turn(const float (&c)[P], const float (&s)[P]) {
    float p[P], q[P];
    get(p, q);
    turn_pairs(p, q, c, s);
    set(p, q);
  }
  static __device__ __forceinline__ void turn_pairs(float (&p)[P], float (&q)[P],
                                                    const float (&c)[P], const float (&s)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float u = p[i], v = q[i];
      p[i] = u * c[i] - v * s[i];
      q[i] = v * c[i] + u * s[i];
    }
  }
};

// Sine and cosine, times amp, of the angle at a position.
template <bool FAST>
__device__ __forceinline__ void angle(const RopeArgs& a, int64_t pos, uint64_t turns, float& co,
                                      float& si) {
  // half turns: 24 of the 32 bits survive, an angle error of pi 2^-25
  const float x = (float)(int32_t)(((uint64_t)pos * turns) >> 32) * 0x1p-31f;
  if constexpr (FAST) __sincosf(x * 3.14159265f, &si, &co);
  else sincospif(x, &si, &co);
  co *= a.amp;
  si *= a.amp * a.sign;
}

// HB: heads of a token in flight; kAhead / HB tokens of a thread.
template <class T, int P, bool INTER, int HB>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int TB = kAhead / HB;
  stream_wait();
  let_next_start();
  const int tt = (int)a.fu.div(threadIdx.x), u = (int)threadIdx.x - tt * (int)a.fu.d;
  if (tt >= a.tile) return;
  const int h0 = blockIdx.y * a.heads, h1 = min(a.H, h0 + a.heads);
  // second: from a pair's first feature to its second (copies: the next P)
  const bool pair = u < a.pair_units;
  const int c = pair ? u * (INTER ? 2 * P : P) : a.rot + (u - a.pair_units) * 2 * P;
  const int second = pair && !INTER ? a.half : P;
  const int t0 = blockIdx.x * a.tile * TB + tt;
  const T* in[TB];
  T* out[TB];
  int64_t pos[TB];
#pragma unroll
  for (int i = 0; i < TB; ++i) {
    const int t = t0 + i * a.tile;
    const int b = (int)a.fl.div((uint32_t)t), l = t - b * a.L;
    in[i] = (const T*)a.in + (b * a.si.b + l * a.si.l + c);
    out[i] = (T*)a.out + (b * a.so.b + l * a.so.l + c);
    pos[i] = a.pos0 + l;
    if (a.pos && t < a.tokens)
      pos[i] = a.pos0 + a.pos[(int64_t)b * a.pos_batch * a.L + l];
  }
  Pairs<T, P, INTER> r[TB][HB];
  auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < TB; ++i)
#pragma unroll
      for (int k = 0; k < HB; ++k)
        if (t0 + i * a.tile < a.tokens && h + k < h1) r[i][k].load(in[i] + (h + k) * a.si.h, second);
  };
  load(h0);   // on the way while the angles are formed
  uint64_t turns[P];
#pragma unroll
  for (int i = 0; i < P; ++i) turns[i] = pair ? a.turns[u * P + i] : 0;
  float cs[TB == 1 ? P : 1], sn[TB == 1 ? P : 1];
  constexpr bool kFast = sizeof(T) == 2;
  if constexpr (TB == 1) {
    if (pair) {
#pragma unroll
      for (int i = 0; i < P; ++i) angle<kFast>(a, pos[0], turns[i], cs[i], sn[i]);
    }
    for (int h = h0; h < h1; h += HB) {
      if (h != h0) load(h);
#pragma unroll
      for (int k = 0; k < HB; ++k)
        if (t0 < a.tokens && h + k < h1) {
          if (pair) r[0][k].turn(cs, sn);
          r[0][k].store(out[0] + (h + k) * a.so.h, second);
        }
    }
  } else {
#pragma unroll
    for (int i = 0; i < TB; ++i) {
      float c1[P], s1[P];
      if (pair) {
#pragma unroll
        for (int p = 0; p < P; ++p) angle<kFast>(a, pos[i], turns[p], c1[p], s1[p]);
      }
#pragma unroll
      for (int k = 0; k < HB; ++k)
        if (t0 + i * a.tile < a.tokens && h0 + k < h1) {
          if (pair) r[i][k].turn(c1, s1);
          r[i][k].store(out[i] + (h0 + k) * a.so.h, second);
        }
    }
  }
}

template <class T, int P, bool INTER, int HB>
cudaError_t run_heads(const RopeArgs& a, cudaStream_t s) {
  const int per = a.tile * (kAhead / HB);
  note_launch();
  return launch_overlapped(rope_kernel<T, P, INTER, HB>,
                           dim3((unsigned)((a.tokens + per - 1) / per),
                                (unsigned)((a.H + a.heads - 1) / a.heads)),
                           kThreads, 0, s, a);
}
template <class T, int P, bool INTER>
cudaError_t run(const RopeArgs& a, cudaStream_t s) {
  if (a.H == 1) return run_heads<T, P, INTER, 1>(a, s);
  if (a.H == 2) return run_heads<T, P, INTER, 2>(a, s);
  return run_heads<T, P, INTER, 4>(a, s);
}
template <class T, int P>
cudaError_t run_order(const RopeArgs& a, bool inter, cudaStream_t s) {
  return inter ? run<T, P, true>(a, s) : run<T, P, false>(a, s);
}

// dx = (dqk turned back) + dv; a.in is dqk, float32 and contiguous like dv.
// 33.5 M elements to bf16: 50.8 us (336 MB, 6.6 TB/s: HBM).
template <class T, int P, bool INTER>
__global__ void __launch_bounds__(kThreads)
rope_sum_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int HB = 2;   // heads in flight, two float32 arrays each
  stream_wait();
  let_next_start();
  const int tt = (int)a.fu.div(threadIdx.x), u = (int)threadIdx.x - tt * (int)a.fu.d;
  const int t = blockIdx.x * a.tile + tt;
  if (tt >= a.tile || t >= a.tokens) return;
  const int h0 = blockIdx.y * a.heads, h1 = min(a.H, h0 + a.heads);
  const bool pair = u < a.pair_units;
  const int c = pair ? u * (INTER ? 2 * P : P) : a.rot + (u - a.pair_units) * 2 * P;
  const int second = pair && !INTER ? a.half : P;
  const int b = (int)a.fl.div((uint32_t)t), l = t - b * a.L;
  const int64_t from = b * a.si.b + l * a.si.l + c;
  T* out = (T*)a.out + (b * a.so.b + l * a.so.l + c);
  float cs[P], sn[P];
  if (pair) {
    const int64_t pos =
        a.pos0 + (a.pos ? (int64_t)a.pos[(int64_t)b * a.pos_batch * a.L + l] : (int64_t)l);
#pragma unroll
    for (int i = 0; i < P; ++i)
      angle<sizeof(T) == 2>(a, pos, a.turns[u * P + i], cs[i], sn[i]);
  }
  for (int h = h0; h < h1; h += HB) {
    Pairs<float, P, INTER> g[HB], v[HB];
#pragma unroll
    for (int k = 0; k < HB; ++k)
      if (h + k < h1) {
        g[k].load((const float*)a.in + from + (h + k) * a.si.h, second);
        v[k].load(a.add + from + (h + k) * a.si.h, second);
      }
#pragma unroll
    for (int k = 0; k < HB; ++k)
      if (h + k < h1) {
        float p[P], q[P], vp[P], vq[P];
        g[k].get(p, q);
        v[k].get(vp, vq);
        if (pair) Pairs<float, P, INTER>::turn_pairs(p, q, cs, sn);
#pragma unroll
        for (int i = 0; i < P; ++i) p[i] += vp[i], q[i] += vq[i];
        Pairs<T, P, INTER> o;
        o.set(p, q);
        o.store(out + (h + k) * a.so.h, second);
      }
  }
}

template <class T, int P>
cudaError_t run_sum(const RopeArgs& a, bool inter, cudaStream_t s) {
  note_launch();
  return launch_overlapped(inter ? rope_sum_kernel<T, P, true> : rope_sum_kernel<T, P, false>,
                           dim3((unsigned)((a.tokens + a.tile - 1) / a.tile),
                                (unsigned)((a.H + a.heads - 1) / a.heads)),
                           kThreads, 0, s, a);
}

RopeArgs rope_args(const lsh_rope_problem& q, const lsh_strides& sin, const lsh_strides& sout,
                   const void* in, const uint64_t* turns, const int32_t* pos, int64_t pos0,
                   void* out, bool inverse, int vp, int ahead) {
  RopeArgs a{};
  a.in = in, a.out = out, a.si = sin, a.so = sout;
  a.turns = turns, a.pos = pos, a.pos0 = pos0;
  a.H = q.H, a.L = q.L, a.tokens = q.B * q.L;
  a.half = q.rot / 2, a.rot = q.rot;
  a.pair_units = a.half / vp;
  const int units = a.pair_units + (q.d - q.rot) / (2 * vp);
  a.fl = FastDiv((uint32_t)q.L), a.fu = FastDiv((uint32_t)units);
  a.pos_batch = q.pos_batch;
  a.amp = q.amp, a.sign = inverse ? -1.f : 1.f;
  a.tile = std::max(1, kThreads / units);
  // enough CTAs for the GPU before a thread walks more heads
  const int64_t ctas = ((int64_t)a.tokens + a.tile - 1) / a.tile;
  const int64_t split = std::min<int64_t>((q.H + ahead - 1) / ahead,
                                          std::max<int64_t>(1, 148 * 8 / ctas));
  a.heads = (int)((q.H + split - 1) / split);
  return a;
}

}  // namespace

cudaError_t launch_rope_sum(const lsh_rope_problem& q, const lsh_strides& sx, const float* dqk,
                            const float* dv, const uint64_t* turns, const int32_t* pos,
                            int64_t pos0, void* dx, int vp, cudaStream_t s) {
  const lsh_strides flat = {(int64_t)q.H * q.L * q.d, (int64_t)q.L * q.d, q.d};
  RopeArgs a = rope_args(q, flat, sx, dqk, turns, pos, pos0, dx, true, vp, 2);
  a.add = dv;
  if (q.dtype == LSH_BF16) {
    if (vp == 4) return run_sum<__nv_bfloat16, 4>(a, q.interleaved, s);
    if (vp == 2) return run_sum<__nv_bfloat16, 2>(a, q.interleaved, s);
    return run_sum<__nv_bfloat16, 1>(a, q.interleaved, s);
  }
  if (vp == 4) return run_sum<float, 4>(a, q.interleaved, s);
  if (vp == 2) return run_sum<float, 2>(a, q.interleaved, s);
  return run_sum<float, 1>(a, q.interleaved, s);
}

cudaError_t launch_rope(const lsh_rope_problem& q, const lsh_strides& sin, const lsh_strides& sout,
                        const void* in, const uint64_t* turns, const int32_t* pos, int64_t pos0,
                        void* out, bool inverse, int vp, cudaStream_t s) {
  const RopeArgs a = rope_args(q, sin, sout, in, turns, pos, pos0, out, inverse, vp, kAhead);
  if (q.dtype == LSH_BF16) {
    if (vp == 8) return run<__nv_bfloat16, 8, false>(a, s);
    if (vp == 4) return run_order<__nv_bfloat16, 4>(a, q.interleaved, s);
    if (vp == 2) return run_order<__nv_bfloat16, 2>(a, q.interleaved, s);
    return run_order<__nv_bfloat16, 1>(a, q.interleaved, s);
  }
  if (vp == 4) return run<float, 4, false>(a, s);
  if (vp == 2) return run_order<float, 2>(a, q.interleaved, s);
  return run_order<float, 1>(a, q.interleaved, s);
}

}  // namespace lsh
