// Rotary positions: pairs of a head row's features turned by position * freq.
//
// The angle is formed as a phase in turns, by the integer product position *
// turns modulo 2^64 (turns = freq / 2 pi as a 64-bit fraction): the integer
// wrap is the reduction modulo one turn, exact at any distance, where a
// float32 product of position and frequency would lose the phase (0.03 rad
// at position 2^20). Its top 32 bits, signed, are half turns in [-1, 1).
//
// Sine and cosine of a (token, pair) serve every head: a thread keeps those
// of its pairs in registers and walks the heads, four rows in flight; with one
// or two heads it takes four or two tokens instead. bf16 takes the hardware's
// approximate sine and cosine (absolute error below 2^-21 on one turn, where
// a bf16 result is rounded at 2^-9 of its value), float32 the accurate ones.
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

// P pairs of one unit: P low and P high features, or 2 P adjacent ones.
template <class T, int P, bool INTER>
struct Pairs {
  Vec<T, INTER ? 2 * P : P> a;
  Vec<T, INTER ? 1 : P> b;
  __device__ __forceinline__ void load(const T* p, int second) {
    a.load(p);
    if constexpr (!INTER) b.load(p + second);
  }
  __device__ __forceinline__ void store(T* p, int second) const {
    a.store(p);
    if constexpr (!INTER) b.store(p + second);
  }
  __device__ __forceinline__ void turn(const float (&c)[P], const float (&s)[P]) {
    if constexpr (INTER) {
      float v[2 * P];
      a.get(v);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float p = v[2 * i], q = v[2 * i + 1];
        v[2 * i] = p * c[i] - q * s[i];
        v[2 * i + 1] = q * c[i] + p * s[i];
      }
      a.set(v);
    } else {
      float v[P], u[P];
      a.get(v);
      b.get(u);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float p = v[i], q = u[i];
        v[i] = p * c[i] - q * s[i];
        u[i] = q * c[i] + p * s[i];
      }
      a.set(v);
      b.set(u);
    }
  }
};

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
  const int second = pair ? a.half : P;
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
      pos[i] = a.pos0 + __ldg(a.pos + (int64_t)b * a.pos_batch * a.L + l);
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
  for (int i = 0; i < P; ++i) turns[i] = pair ? __ldg(a.turns + u * P + i) : 0;
  float cs[TB == 1 ? P : 1], sn[TB == 1 ? P : 1];
  auto angle = [&](int64_t at, int i, float& co, float& si) {
    // half turns: 24 of the 32 bits survive, an angle error of pi 2^-25
    const float x = (float)(int32_t)(((uint64_t)at * turns[i]) >> 32) * 0x1p-31f;
    if constexpr (sizeof(T) == 2) __sincosf(x * 3.14159265f, &si, &co);
    else sincospif(x, &si, &co);
    co *= a.amp;
    si *= a.amp * a.sign;
  };
  if constexpr (TB == 1) {
    if (pair) {
#pragma unroll
      for (int i = 0; i < P; ++i) angle(pos[0], i, cs[i], sn[i]);
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
        for (int p = 0; p < P; ++p) angle(pos[i], p, c1[p], s1[p]);
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

}  // namespace

cudaError_t launch_rope(const lsh_rope_problem& q, const lsh_strides& sin, const lsh_strides& sout,
                        const void* in, const uint64_t* turns, const int32_t* pos, int64_t pos0,
                        void* out, bool inverse, int vp, cudaStream_t s) {
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
  const int64_t split = std::min<int64_t>((q.H + kAhead - 1) / kAhead,
                                          std::max<int64_t>(1, 148 * 8 / ctas));
  a.heads = (int)((q.H + split - 1) / split);
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
