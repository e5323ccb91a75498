// Device helpers of the sublayer operators: vectors of V elements, division
// by a launch constant, and the dropout's random lanes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace lsh {

// Programmatic dependent launch: a kernel of this file's users lets the next
// one of the stream be set up while it runs, and waits for all earlier work of
// the stream before it touches memory. Every thread of every kernel waits, so
// that the end of a kernel means the end of all before it. All loads after the
// wait are plain ones: a load that the compiler may take for one of constant
// memory (ld.global.nc) could be moved before it.
__device__ __forceinline__ void stream_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <class Args>
cudaError_t launch_overlapped(void (*fn)(const Args), dim3 grid, unsigned threads, size_t smem,
                              cudaStream_t s, const Args& a) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, fn, a);
}

// V consecutive elements of type T as 32-bit words (one half word for V = 1
// bf16), loaded and stored in accesses of at most 16 bytes.
template <class T, int V>
struct Vec {
  static constexpr int kBytes = V * (int)sizeof(T);
  static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kBytes == 2) {
      w[0] = *reinterpret_cast<const unsigned short*>(p);
    } else if constexpr (kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (kBytes == 8) {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      w[0] = u.x;
      w[1] = u.y;
    } else {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 u = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = u.x;
        w[4 * i + 1] = u.y;
        w[4 * i + 2] = u.z;
        w[4 * i + 3] = u.w;
      }
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kBytes == 2) {
      *reinterpret_cast<unsigned short*>(p) = (unsigned short)w[0];
    } else if constexpr (kBytes == 4) {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    } else if constexpr (kBytes == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        reinterpret_cast<uint4*>(p)[i] =
            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
  }
  __device__ __forceinline__ void get(float (&v)[V]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = __uint_as_float(w[i]);
    } else if constexpr (V == 1) {
      v[0] = __uint_as_float(w[0] << 16);
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
  // bf16: round to nearest even.
  __device__ __forceinline__ void set(const float (&v)[V]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = __float_as_uint(v[i]);
    } else if constexpr (V == 1) {
      w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<uint32_t*>(&h);
      }
    }
  }
};

// n / d and n mod d for 0 <= n < 2^31 by one multiplication: with s =
// ceil(log2 d) and m = ceil(2^(32+s) / d) - 2^32, (umulhi(n, m) + n) >> s is
// the quotient for every 32-bit n, and the sum stays below 2^32 for n < 2^31.
struct FastDiv {
  uint32_t d, m, s;
  FastDiv() = default;
  explicit FastDiv(uint32_t div) : d(div), s(0) {
    while ((1ull << s) < d) ++s;
    m = (uint32_t)((((1ull << s) - d) << 32) / d + 1);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return (__umulhi(n, m) + n) >> s;
  }
};

// Ten rounds of Philox4x32 (Salmon et al., SC 2011): two 32 x 32 -> 64-bit
// products a round, keys stepped by two odd constants. The round keys are a
// function of the seed alone, formed on the host, so that they are constant
// operands of the exclusive-ors.
struct PhiloxKeys {
  uint32_t k0[10], k1[10];
  PhiloxKeys() = default;
  explicit PhiloxKeys(uint64_t seed) {
    uint32_t a = (uint32_t)seed, b = (uint32_t)(seed >> 32);
    for (int r = 0; r < 10; ++r) {
      k0[r] = a, k1[r] = b;
      a += 0x9E3779B9u, b += 0xBB67AE85u;
    }
  }
};
__device__ __forceinline__ uint4 philox(const PhiloxKeys& key, uint64_t n, uint64_t offset) {
  uint32_t x0 = (uint32_t)n, x1 = (uint32_t)(n >> 32), x2 = (uint32_t)offset,
           x3 = (uint32_t)(offset >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p = (uint64_t)x0 * 0xD2511F53u, q = (uint64_t)x2 * 0xCD9E8D57u;
    x0 = (uint32_t)(q >> 32) ^ x1 ^ key.k0[r];
    x1 = (uint32_t)q;
    x2 = (uint32_t)(p >> 32) ^ x3 ^ key.k1[r];
    x3 = (uint32_t)p;
  }
  return make_uint4(x0, x1, x2, x3);
}

// v[i] = kept ? v[i] : 0 for the V features starting at feature c (a multiple
// of V) of a row, r being the random words of the group of 8 that c is in.
// Lane x is kept when x >= t, t in 1 .. 65536, which is x 2^16 > t 2^16 - 1:
// with that bound in 32 bits (t = 65536 keeps nothing) the high half of a word
// is compared in place, its low half bits below the bound's.
template <int V>
__device__ __forceinline__ void drop(float (&v)[V], const uint4& r, int c, uint32_t t) {
  static_assert(V == 8 || V == 4 || V == 1, "a group, half of one, or one element");
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  if constexpr (V > 1) {
    const uint32_t bound = (t << 16) - 1u;
    const bool high = V == 4 && (c & 4);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t u = high ? w[(i / 2 + 2) & 3] : w[i / 2];
      const uint32_t lane = (i & 1) ? u : u << 16;
      v[i] = lane > bound ? v[i] : 0.f;
    }
  } else {
    const int i = c & 7;
    const uint32_t u = (i & 4) ? ((i & 2) ? w[3] : w[2]) : ((i & 2) ? w[1] : w[0]);
    const uint32_t lane = (i & 1) ? u >> 16 : u & 0xffffu;
    v[0] = lane >= t ? v[0] : 0.f;
  }
}

}  // namespace lsh
