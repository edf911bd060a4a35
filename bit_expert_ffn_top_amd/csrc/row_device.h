// Rows of fp32 or bfloat16 values, several consecutive ones per lane.
#pragma once

#include "moe_common.h"

namespace bitffn {

// Two fp32 values as bfloat16, round to nearest even (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, bf2{static_cast<__bf16>(lo), static_cast<__bf16>(hi)});
}

typedef float nf4 __attribute__((ext_vector_type(4)));
typedef uint32_t nu4 __attribute__((ext_vector_type(4)));
typedef uint32_t nu2 __attribute__((ext_vector_type(2)));

// N (4 or 8) values of a row: fp32 in 16-byte parts, bfloat16 in one part of 2N
// bytes that needs only 8-byte alignment (rows of an odd number of fours).
// STREAM: past the caches.  `half`: only the first four are there (N = 8, the end
// of such a row); the others are zeros.
template <typename T, int N>
struct RowPart;

template <int N>
struct RowPart<float, N> {
  nf4 v[N / 4];
  template <bool STREAM = false>
  __device__ __forceinline__ void load(const float* p, bool half = false) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const nf4* q = reinterpret_cast<const nf4*>(p) + i;
      if (i == 0 || !half)
        v[i] = STREAM ? __builtin_nontemporal_load(q) : *q;
      else
        v[i] = nf4{0.0f, 0.0f, 0.0f, 0.0f};
    }
  }
  template <bool STREAM = false>
  __device__ __forceinline__ void store(float* p, bool half = false) const {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      nf4* q = reinterpret_cast<nf4*>(p) + i;
      if (i > 0 && half) break;
      if (STREAM)
        __builtin_nontemporal_store(v[i], q);
      else
        *q = v[i];
    }
  }
  __device__ __forceinline__ float get(int i) const { return v[i / 4][i % 4]; }
  __device__ __forceinline__ void set(const float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i / 4][i % 4] = f[i];
  }
};

template <int N>
struct RowPart<uint16_t, N> {
  typedef uint32_t part __attribute__((ext_vector_type(N / 2), aligned(8)));
  typedef uint32_t first __attribute__((ext_vector_type(2)));
  part v;
  template <bool STREAM = false>
  __device__ __forceinline__ void load(const uint16_t* p, bool half = false) {
    if (N == 8 && half) {
      const first f = *reinterpret_cast<const first*>(p);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) v[i] = i < 2 ? f[i] : 0u;
    } else {
      const part* q = reinterpret_cast<const part*>(p);
      v = STREAM ? __builtin_nontemporal_load(q) : *q;
    }
  }
  template <bool STREAM = false>
  __device__ __forceinline__ void store(uint16_t* p, bool half = false) const {
    if (N == 8 && half) {
      *reinterpret_cast<first*>(p) = first{v[0], v[1]};
    } else {
      part* q = reinterpret_cast<part*>(p);
      if (STREAM)
        __builtin_nontemporal_store(v, q);
      else
        *q = v;
    }
  }
  __device__ __forceinline__ float get(int i) const {
    return i % 2 ? __builtin_bit_cast(float, v[i / 2] & 0xFFFF0000u) : bf16_bits_to_float(v[i / 2]);
  }
  __device__ __forceinline__ void set(const float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) v[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
  }
};

}  // namespace bitffn
