// Dropout whose mask is a function of (seed, offset, position): Philox4x32-10
// gives 128 bits for each group of 8 features of a row, 16 bits a feature, so
// the mask costs one call of ten rounds per 8 features and no memory.
//
// Bound by HBM in float32; in bf16, where a group of 8 is one 16-byte access,
// as much by the instructions of the ten rounds (two wide products and two
// exclusive-ors each) and of the 8 comparisons. The rest is kept small: rows
// are walked in the order of x's strides, and dimensions that follow on in x,
// y and the counters alike are merged on the host, all of them for contiguous
// arrays, which then need no division of indices. 134 MB in all: 33.5 M bf16
// elements 25.7 us (5.2 TB/s), 16.8 M float32 ones 21.9 us (6.1 TB/s).
#include <algorithm>

#include "internal.h"
#include "sublayer.cuh"
#include "sublayer.h"

namespace lsh {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;   // vectors a thread has in flight

// Row r = (i2 n1 + i1) n0 + i0 starts at i0 x[0] + i1 x[1] + i2 x[2] of x, the
// like of y, and has the counters from i0 c[0] + i1 c[1] + i2 c[2].
struct DropArgs {
  const void* x;
  void* y;
  int64_t sx[3], sy[3];
  uint64_t sc[3], ctr0;
  FastDiv upr, n0, n1;
  int rows, tile;   // tile: rows of a CTA
  uint32_t t;
  float scale;
  PhiloxKeys key;
  uint64_t offset;
  const uint64_t* counter;
};

// DIMS: 3, or 1 where all dimensions merge, or 0 where the rows also follow on
// in x, y and the counters without a gap.
template <class T, int V, int DIMS>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const __grid_constant__ DropArgs a) {
  stream_wait();
  let_next_start();
  const uint64_t offset = a.offset + (a.counter ? *a.counter : 0);
  const int row0 = blockIdx.x * a.tile;
  const int n = min(a.tile, a.rows - row0) * (int)a.upr.d;
  for (int j0 = threadIdx.x; j0 < n; j0 += kThreads * kUnits) {
    Vec<T, V> r[kUnits];
    int64_t out[kUnits];
    uint64_t ctr[kUnits];
    int c[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int j = j0 + k * kThreads;
      if (DIMS == 0 && j < n) {
        c[k] = 0;
        const int64_t u = (int64_t)row0 * a.upr.d + j;
        out[k] = u * V;
        ctr[k] = a.ctr0 + u;
        r[k].load((const T*)a.x + out[k]);
      } else if (j < n) {
        const int rr = (int)a.upr.div((uint32_t)j);
        c[k] = (j - rr * (int)a.upr.d) * V;
        const int row = row0 + rr;
        int64_t in = c[k];
        out[k] = c[k];
        ctr[k] = a.ctr0 + (uint32_t)c[k] / 8;
        if constexpr (DIMS == 1) {
          in += row * a.sx[0];
          out[k] += row * a.sy[0];
          ctr[k] += (uint32_t)row * a.sc[0];
        } else {
          const uint32_t q = a.n0.div((uint32_t)row), i0 = row - q * a.n0.d;
          const uint32_t i2 = a.n1.div(q), i1 = q - i2 * a.n1.d;
          in += i0 * a.sx[0] + i1 * a.sx[1] + i2 * a.sx[2];
          out[k] += i0 * a.sy[0] + i1 * a.sy[1] + i2 * a.sy[2];
          ctr[k] += i0 * a.sc[0] + i1 * a.sc[1] + i2 * a.sc[2];
        }
        r[k].load((const T*)a.x + in);
      }
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      if (j0 + k * kThreads < n) {
        float v[V];
        r[k].get(v);
        if (a.t) {
          drop<V>(v, philox(a.key, ctr[k], offset), c[k], a.t);
#pragma unroll
          for (int i = 0; i < V; ++i) v[i] *= a.scale;
        }
        r[k].set(v);
        r[k].store((T*)a.y + out[k]);
      }
    }
  }
}

template <class T, int V>
cudaError_t run(const DropArgs& a, int dims, cudaStream_t s) {
  note_launch();
  return launch_overlapped(dims == 0   ? dropout_kernel<T, V, V == 8 ? 0 : 1>
                           : dims == 1 ? dropout_kernel<T, V, 1>
                                       : dropout_kernel<T, V, 3>,
                           dim3((unsigned)((a.rows + a.tile - 1) / a.tile)), kThreads, 0, s, a);
}

}  // namespace

cudaError_t launch_dropout(const lsh_dropout_problem& q, uint32_t t, float scale, const void* x,
                           uint64_t seed, uint64_t offset, const uint64_t* counter, void* y,
                           bool wide, cudaStream_t s) {
  DropArgs a{};
  const int V = wide ? 8 : 1;
  const uint64_t gpr = (q.d + 7) / 8, head = gpr * q.L;
  struct Dim {
    int64_t n, x, y;
    uint64_t c;
  } d[3] = {{q.L, q.x.l, q.y.l, gpr}, {q.H, q.x.h, q.y.h, head}, {q.B, q.x.b, q.y.b, head * q.H}};
  // dimensions of one element need no place in the order
  std::stable_sort(d, d + 3, [](const Dim& u, const Dim& v) {
    if ((u.n > 1) != (v.n > 1)) return u.n > 1;
    return u.n > 1 && u.x < v.x;
  });
  int m = 0;
  for (int i = 1; i < 3; ++i) {
    Dim& u = d[m];
    const Dim& v = d[i];
    if (v.n <= 1) continue;
    if (v.x == u.n * u.x && v.y == u.n * u.y && v.c == u.n * u.c) u.n *= v.n;
    else d[++m] = v;
  }
  for (int i = m + 1; i < 3; ++i) d[i] = {1, 0, 0, 0};
  for (int i = 0; i < 3; ++i) a.sx[i] = d[i].x, a.sy[i] = d[i].y, a.sc[i] = d[i].c;
  a.n0 = FastDiv((uint32_t)d[0].n), a.n1 = FastDiv((uint32_t)d[1].n);
  a.x = x, a.y = y;
  a.upr = FastDiv((uint32_t)(q.d / V));
  a.rows = q.B * q.H * q.L;
  a.tile = std::max(1, kThreads * kUnits / (int)a.upr.d);
  a.t = t, a.scale = scale, a.key = PhiloxKeys(seed), a.offset = offset, a.counter = counter;
  a.ctr0 = q.slice0 * head;
  const bool dense = wide && m == 0 && d[0].x == q.d && d[0].y == q.d && d[0].c == gpr;
  const int dims = dense ? 0 : m == 0 ? 1 : 3;
  if (q.dtype == LSH_BF16)
    return wide ? run<__nv_bfloat16, 8>(a, dims, s) : run<__nv_bfloat16, 1>(a, dims, s);
  return wide ? run<float, 8>(a, dims, s) : run<float, 1>(a, dims, s);
}

}  // namespace lsh
