// Dropout whose mask is a function of (seed, offset, position): Philox4x32-10
// gives 128 bits for each group of 8 features of a row, 16 bits a feature, so
// the mask costs one call of ten rounds per 8 features and no memory.
#include <algorithm>

#include "internal.h"
#include "sublayer.cuh"
#include "sublayer.h"

namespace lsh {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;   // vectors a thread has in flight

struct DropArgs {
  const void* x;
  void* y;
  lsh_strides sx, sy;
  FastDiv upr, fl, fh;
  int H, L, gpr, rows, tile;   // tile: rows of a CTA
  uint32_t t;
  float scale;
  PhiloxKeys key;
  uint64_t offset;
  const uint64_t* counter;
  int64_t slice0;
};

// A CTA takes `tile` rows; vector j of them is row j / upr, feature j mod upr.
template <class T, int V>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const __grid_constant__ DropArgs a) {
  const uint64_t offset = a.offset + (a.counter ? __ldg(a.counter) : 0);
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
      if (j < n) {
        const int rr = (int)a.upr.div((uint32_t)j);
        c[k] = (j - rr * (int)a.upr.d) * V;
        const int row = row0 + rr;
        const int s = (int)a.fl.div((uint32_t)row), l = row - s * a.L;
        const int b = (int)a.fh.div((uint32_t)s), h = s - b * a.H;
        r[k].load((const T*)a.x + (b * a.sx.b + h * a.sx.h + l * a.sx.l + c[k]));
        out[k] = b * a.sy.b + h * a.sy.h + l * a.sy.l + c[k];
        ctr[k] = (uint64_t)(a.slice0 * a.L + row) * (uint32_t)a.gpr + (uint32_t)c[k] / 8;
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
void run(const DropArgs& a, cudaStream_t s) {
  dropout_kernel<T, V><<<(unsigned)((a.rows + a.tile - 1) / a.tile), kThreads, 0, s>>>(a);
}

}  // namespace

cudaError_t launch_dropout(const lsh_dropout_problem& q, uint32_t t, float scale, const void* x,
                           uint64_t seed, uint64_t offset, const uint64_t* counter, void* y,
                           bool wide, cudaStream_t s) {
  DropArgs a{};
  const int V = wide ? 8 : 1;
  a.x = x, a.y = y, a.sx = q.x, a.sy = q.y;
  a.upr = FastDiv((uint32_t)(q.d / V));
  a.fl = FastDiv((uint32_t)q.L), a.fh = FastDiv((uint32_t)q.H);
  a.H = q.H, a.L = q.L, a.gpr = (q.d + 7) / 8;
  a.rows = q.B * q.H * q.L;
  a.tile = std::max(1, kThreads * kUnits / (int)a.upr.d);
  a.t = t, a.scale = scale, a.key = PhiloxKeys(seed), a.offset = offset, a.counter = counter;
  a.slice0 = q.slice0;
  if (q.dtype == LSH_BF16) wide ? run<__nv_bfloat16, 8>(a, s) : run<__nv_bfloat16, 1>(a, s);
  else wide ? run<float, 8>(a, s) : run<float, 1>(a, s);
  note_launch();
  return cudaGetLastError();
}

}  // namespace lsh
