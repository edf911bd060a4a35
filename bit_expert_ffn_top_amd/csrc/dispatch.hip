// Tokens to the experts and back: the pairs' rows in group order, the weighted
// sum of them in the tokens' order, and the gradients of both.
#include "moe_internal.h"
#include "row_device.h"

namespace bitffn {
namespace {

constexpr int kMaxE = MOE_MAX_EXPERTS;
constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxOwn = 2048;   // pairs of one workgroup's tokens

// The row of a pair = pairs of smaller experts + earlier pairs of its expert.
// Every workgroup counts all pairs in LDS, those before its own tokens first,
// so the call is one launch; ranks among its own pairs are counted directly,
// which keeps equal ids of a token in order.  A wavefront then reads a token's
// row once and writes it to its k places.
template <typename V>   // uint4 or uint2: the part of a row one lane moves
__global__ __launch_bounds__(kThreads) void dispatch_kernel(
    const V* __restrict__ x, int T, int nv, const int32_t* __restrict__ idx, int k, int E,
    int tokens, V* __restrict__ rows, int32_t* __restrict__ offsets,
    int32_t* __restrict__ pair_pos) {
  __shared__ int32_t s_count[kMaxE];
  __shared__ int32_t s_before[kMaxE];
  __shared__ int32_t s_sum[kThreads];
  __shared__ int32_t s_own[kMaxOwn];
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * tokens, t1 = min(T, t0 + tokens);
  const int n = T * k, p0 = t0 * k, own = (t1 - t0) * k;
  for (int e = tid; e < kMaxE; e += kThreads) s_count[e] = 0;
  __syncthreads();
  for (int p = tid; p < p0; p += kThreads) {
    const int e = idx[p];
    if (e >= 0 && e < E) atomicAdd(&s_count[e], 1);
  }
  __syncthreads();
  for (int e = tid; e < kMaxE; e += kThreads) s_before[e] = s_count[e];
  __syncthreads();
  for (int p = p0 + tid; p < n; p += kThreads) {
    const int e = idx[p];
    if (e >= 0 && e < E) atomicAdd(&s_count[e], 1);
    if (p < p0 + own) s_own[p - p0] = e >= 0 && e < E ? e : -1;
  }
  __syncthreads();
  // exclusive scan over the experts, four per thread
  constexpr int kPer = kMaxE / kThreads;
  int c[kPer], sum = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    c[j] = sum;
    sum += s_count[tid * kPer + j];
  }
  s_sum[tid] = sum;
  __syncthreads();
  for (int off = 1; off < kThreads; off <<= 1) {
    const int v = tid >= off ? s_sum[tid - off] : 0;
    __syncthreads();
    s_sum[tid] += v;
    __syncthreads();
  }
  const int base = s_sum[tid] - sum;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = tid * kPer + j;
    s_before[e] += base + c[j];
    if (blockIdx.x == 0 && e < E) offsets[e] = base + c[j];
  }
  if (blockIdx.x == 0 && tid == kThreads - 1) offsets[E] = s_sum[tid];
  __syncthreads();
  for (int q0 = 0; q0 < own; q0 += kThreads) {
    const int q = q0 + tid;
    int at = -1;
    if (q < own) {
      const int e = s_own[q];
      if (e >= 0) {
        at = s_before[e];
        for (int r = 0; r < q; ++r) at += s_own[r] == e;
      }
      pair_pos[p0 + q] = at;
    }
  }
  __syncthreads();   // pair_pos of this workgroup is read back below
  const int lane = tid & 63;
  for (int t = t0 + (tid >> 6); t < t1; t += kWaves) {
    const V* src = x + static_cast<int64_t>(t) * nv;
    for (int j = lane; j < nv; j += 64) {
      const V v = src[j];
      for (int i = 0; i < k; ++i) {
        const int at = pair_pos[t * k + i];
        if (at >= 0) rows[static_cast<int64_t>(at) * nv + j] = v;
      }
    }
  }
}

__device__ __forceinline__ bool has_row(int p, int R) { return p >= 0 && p < R; }

// One thread per N consecutive columns of one token, the k terms in i order.
template <typename RT, typename YT, int N>
__global__ __launch_bounds__(kThreads) void combine_rows_kernel(
    const RT* __restrict__ rows, int R, int T, int d, int k, const int32_t* __restrict__ pair_pos,
    const float* __restrict__ w, const void* base, int base_dtype, YT* y) {
  const int dn = d / N;
  const int64_t gid = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (gid >= static_cast<int64_t>(T) * dn) return;
  const int t = static_cast<int>(gid / dn);
  const int c = static_cast<int>(gid - static_cast<int64_t>(t) * dn) * N;
  const int64_t at = static_cast<int64_t>(t) * d + c;
  float acc[N];
#pragma unroll
  for (int j = 0; j < N; ++j) acc[j] = 0.0f;
  if (base && base_dtype == MOE_DTYPE_F32) {
    RowPart<float, N> b;
    b.load(static_cast<const float*>(base) + at);
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = b.get(j);
  } else if (base) {
    RowPart<uint16_t, N> b;
    b.load(static_cast<const uint16_t*>(base) + at);
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = b.get(j);
  }
  for (int i = 0; i < k; ++i) {
    const int64_t q = static_cast<int64_t>(t) * k + i;
    const int p = pair_pos[q];
    if (!has_row(p, R)) continue;
    const float wi = w ? w[q] : 1.0f;
    RowPart<RT, N> r;
    r.load(rows + static_cast<int64_t>(p) * d + c);
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = fmaf(wi, r.get(j), acc[j]);
  }
  RowPart<YT, N> out;
  out.set(acc);
  out.store(y + at);
}

// One workgroup per token, one wavefront per pair at a time: the product with
// dy for dw, and dy times the weight for drows.
template <typename GT, typename RT, int N>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(
    const GT* __restrict__ dy, const RT* __restrict__ rows, int R, int d, int k,
    const int32_t* __restrict__ pair_pos, const float* __restrict__ w, RT* __restrict__ drows,
    float* __restrict__ dw) {
  const int lane = threadIdx.x & 63;
  const int64_t t = blockIdx.x;
  for (int i = threadIdx.x >> 6; i < k; i += kWaves) {
    const int64_t q = t * k + i;
    const int p = pair_pos[q];
    float sum = 0.0f;
    if (has_row(p, R)) {
      const float wi = w ? w[q] : 1.0f;
      for (int c = lane * N; c < d; c += 64 * N) {
        RowPart<GT, N> g;
        g.load(dy + t * d + c);
        const int64_t at = static_cast<int64_t>(p) * d + c;
        if (dw) {
          RowPart<RT, N> r;
          r.load(rows + at);
#pragma unroll
          for (int j = 0; j < N; ++j) sum = fmaf(g.get(j), r.get(j), sum);
        }
        if (drows) {
          float f[N];
#pragma unroll
          for (int j = 0; j < N; ++j) f[j] = wi * g.get(j);
          RowPart<RT, N> out;
          out.set(f);
          out.store(drows + at);
        }
      }
    }
    if (dw) {
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
      if (lane == 0) dw[q] = sum;
    }
  }
}

template <typename RT, typename YT>
hipError_t combine_rows_as(const void* rows, int64_t R, int T, int d, int k,
                           const int32_t* pair_pos, const float* w, const void* base,
                           int base_dtype, void* y, hipStream_t s) {
  const int n = d % 8 == 0 ? 8 : 4;
  const int64_t blocks = (static_cast<int64_t>(T) * (d / n) + kThreads - 1) / kThreads;
  const auto go = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(
        static_cast<const RT*>(rows), static_cast<int>(R), T, d, k, pair_pos, w, base, base_dtype,
        static_cast<YT*>(y));
  };
  if (n == 8)
    go(combine_rows_kernel<RT, YT, 8>);
  else
    go(combine_rows_kernel<RT, YT, 4>);
  return hipGetLastError();
}

template <typename GT, typename RT>
hipError_t combine_backward_as(const void* dy, const void* rows, int64_t R, int T, int d, int k,
                               const int32_t* pair_pos, const float* w, void* drows, float* dw,
                               hipStream_t s) {
  const auto go = [&](auto kernel) {
    kernel<<<T, kThreads, 0, s>>>(static_cast<const GT*>(dy), static_cast<const RT*>(rows),
                                  static_cast<int>(R), d, k, pair_pos, w, static_cast<RT*>(drows),
                                  dw);
  };
  if (d % 8 == 0)
    go(combine_backward_kernel<GT, RT, 8>);
  else
    go(combine_backward_kernel<GT, RT, 4>);
  return hipGetLastError();
}

}  // namespace

size_t dispatch_workspace_bytes(int, int, int) { return 0; }

hipError_t launch_dispatch(const void* x, int dtype, int T, int d, const int32_t* idx, int k, int E,
                           void* rows, int32_t* offsets, int32_t* pair_pos, void*, hipStream_t s) {
  const int bytes = d * (dtype == MOE_DTYPE_F32 ? 4 : 2);
  const int tokens = max(1, min((T + 1023) / 1024, kMaxOwn / k));
  const int blocks = max(1, (T + tokens - 1) / tokens);
  if (bytes % 16 == 0)
    dispatch_kernel<uint4><<<blocks, kThreads, 0, s>>>(static_cast<const uint4*>(x), T, bytes / 16,
                                                       idx, k, E, tokens, static_cast<uint4*>(rows),
                                                       offsets, pair_pos);
  else
    dispatch_kernel<uint2><<<blocks, kThreads, 0, s>>>(static_cast<const uint2*>(x), T, bytes / 8,
                                                       idx, k, E, tokens, static_cast<uint2*>(rows),
                                                       offsets, pair_pos);
  return hipGetLastError();
}

hipError_t launch_combine_rows(const void* rows, int rows_dtype, int64_t R, int T, int d, int k,
                               const int32_t* pair_pos, const float* w, const void* base,
                               int base_dtype, void* y, int y_dtype, hipStream_t s) {
  const bool rf = rows_dtype == MOE_DTYPE_F32, yf = y_dtype == MOE_DTYPE_F32;
  const auto f = rf ? (yf ? combine_rows_as<float, float> : combine_rows_as<float, uint16_t>)
                    : (yf ? combine_rows_as<uint16_t, float> : combine_rows_as<uint16_t, uint16_t>);
  return f(rows, R, T, d, k, pair_pos, w, base, base_dtype, y, s);
}

hipError_t launch_combine_backward(const void* dy, int dy_dtype, const void* rows, int rows_dtype,
                                   int64_t R, int T, int d, int k, const int32_t* pair_pos,
                                   const float* w, void* drows, float* dw, hipStream_t s) {
  const bool gf = dy_dtype == MOE_DTYPE_F32, rf = rows_dtype == MOE_DTYPE_F32;
  const auto f = gf ? (rf ? combine_backward_as<float, float> : combine_backward_as<float, uint16_t>)
                    : (rf ? combine_backward_as<uint16_t, float>
                          : combine_backward_as<uint16_t, uint16_t>);
  return f(dy, rows, R, T, d, k, pair_pos, w, drows, dw, s);
}

}  // namespace bitffn
