// Host-side interface between the C ABI of the sublayer operators
// (sublayer_api.cu) and their kernel files.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "lsh.h"

namespace lsh {

constexpr int kNormMaxD = 8192;   // features of a token: 512 threads x 16
constexpr int kRopeMaxHead = 512;

// One call of the norm / residual kernels, every pointer resolved; strides in
// elements. Norms alone are the case without a branch (f == nullptr).
struct SubCall {
  int B, H, L, d, dtype;
  int post, norm, gate, gate_batch;
  float eps_post, eps, alpha, beta;
  uint32_t drop_t;        // keep where the 16-bit lane >= drop_t (0: no dropout)
  float drop_scale;
  uint64_t seed, offset;
  const uint64_t* counter;
  int64_t slice0;
  lsh_strides sx, sf, sh; // residual stream; branch; h and dh
  const void *x, *f, *gatep, *dy, *dh;   // backward: x holds y
  const float *wp, *bp, *w, *b;
  void *y, *h, *dx, *df, *dz;
  float *dgate, *dwp, *dbp, *dw, *db;
  bool branch, wide;      // wide: 16-byte accesses of 8 features are aligned
};
cudaError_t launch_sub_fwd(const SubCall& c, cudaStream_t s);
size_t sub_bwd_ws_bytes(int B, int H, int L, int d, bool branch, bool gate_batch);
cudaError_t launch_sub_bwd(const SubCall& c, void* ws, cudaStream_t s);

cudaError_t launch_dropout(const lsh_dropout_problem& q, uint32_t t, float scale, const void* x,
                           uint64_t seed, uint64_t offset, const uint64_t* counter, void* y,
                           bool wide, cudaStream_t s);

cudaError_t launch_rope(const lsh_rope_problem& q, const lsh_strides& sin, const lsh_strides& sout,
                        const void* in, const uint64_t* turns, const int32_t* pos, int64_t pos0,
                        void* out, bool inverse, int vp, cudaStream_t s);
cudaError_t launch_rope_sum(const lsh_rope_problem& q, const lsh_strides& sx, const float* dqk,
                            const float* dv, const uint64_t* turns, const int32_t* pos,
                            int64_t pos0, void* dx, int vp, cudaStream_t s);

}  // namespace lsh
