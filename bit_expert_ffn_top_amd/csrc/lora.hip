// Low-rank adapters of many requests beside a projection that they share:
//   y[t] = base[t] + scale[m] * B_m (A_m x[t]),   m the adapter of t's request
#include "moe_internal.h"
#include "row_device.h"

namespace bitffn {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

struct LoraArgs {
  const void* base;
  const void* x;
  const uint16_t* a;
  const uint16_t* b;
  const int32_t* seq;
  const int32_t* adapter;
  const float* scale;
  void* y;
  int T, d_in, d_out, n_adapters, rank, n_seq;
};

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(uint16_t v) { return bf16_bits_to_float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) {
  *p = static_cast<uint16_t>(pack_bf16(v, 0.0f));
}

// One workgroup per row.  A row's request ends at the first bound above the row,
// and bounds below an earlier one never come first.
template <typename XT, typename YT>
__global__ __launch_bounds__(kThreads) void lora_kernel(LoraArgs g) {
  __shared__ float s_h[MOE_MAX_RANK];
  __shared__ int s_end;
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
  int req = t;
  if (g.seq) {
    if (tid == 0) s_end = g.n_seq + 1;
    __syncthreads();
    int end = g.n_seq + 1;
    for (int s = tid; s <= g.n_seq; s += kThreads)
      if (g.seq[s] > t) {
        end = s;
        break;
      }
    atomicMin(&s_end, end);
    __syncthreads();
    if (s_end == 0 || s_end > g.n_seq) return;
    req = s_end - 1;
  }
  const YT* base = static_cast<const YT*>(g.base) + static_cast<int64_t>(t) * g.d_out;
  YT* y = static_cast<YT*>(g.y) + static_cast<int64_t>(t) * g.d_out;
  const int m = g.adapter[req];
  if (m < 0 || m >= g.n_adapters) {
    if (y != base)
      for (int c = tid; c < g.d_out; c += kThreads) y[c] = base[c];
    return;
  }
  const float scale = g.scale ? g.scale[m] : 1.0f;
  const XT* x = static_cast<const XT*>(g.x) + static_cast<int64_t>(t) * g.d_in;
  for (int r = tid >> 6; r < g.rank; r += kWaves) {
    const uint16_t* a = g.a + (static_cast<int64_t>(m) * g.rank + r) * g.d_in;
    float sum = 0.0f;
    for (int c = lane; c < g.d_in; c += 64) sum = fmaf(bf16_bits_to_float(a[c]), as_float(x[c]), sum);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
    if (lane == 0) s_h[r] = scale * sum;
  }
  __syncthreads();
  for (int c = tid; c < g.d_out; c += kThreads) {
    const uint16_t* b = g.b + (static_cast<int64_t>(m) * g.d_out + c) * g.rank;
    float sum = 0.0f;
    for (int r = 0; r < g.rank; ++r) sum = fmaf(bf16_bits_to_float(b[r]), s_h[r], sum);
    put(y + c, as_float(base[c]) + sum);
  }
}

}  // namespace

hipError_t launch_lora(const void* base, const void* x, int x_dtype, int64_t T, int d_in, int d_out,
                       const uint16_t* a, const uint16_t* b, int n_adapters, int rank,
                       const int32_t* seq, int n_seq, const int32_t* adapter, const float* scale,
                       void* y, int y_dtype, hipStream_t s) {
  const LoraArgs g{base, x, a, b, seq, adapter, scale, y, static_cast<int>(T),
                   d_in, d_out, n_adapters, rank, n_seq};
  const bool xf = x_dtype == MOE_DTYPE_F32, yf = y_dtype == MOE_DTYPE_F32;
  const auto f = xf ? (yf ? lora_kernel<float, float> : lora_kernel<float, uint16_t>)
                    : (yf ? lora_kernel<uint16_t, float> : lora_kernel<uint16_t, uint16_t>);
  f<<<static_cast<unsigned>(T), kThreads, 0, s>>>(g);
  return hipGetLastError();
}

}  // namespace bitffn
