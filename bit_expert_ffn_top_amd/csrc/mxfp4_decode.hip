// Decode / verify FFN over 4-bit experts for 1..4 tokens, activations in fp32
// (moe_mxfp4_ffn_decode).  Two launches:
//   gate/up  h[t][i][j] = silu(g) u for every pair (t, i) whose slot is in the
//            pool, and for the shared expert (i = k);
//   down     y[t] = x[t] + sum_i w_i D_i h[t][i], all pairs of a token in one
//            workgroup, so no partial result goes through memory.
// A wavefront gives each weight row LPR lanes (16, 32 or 64, the least power
// of two that covers the row's blocks, so that few lanes idle); a lane holds
// one 32-value block of 8 consecutive rows at a time: 8 loads of 16 bytes in
// flight, each block dequantized by 16 conversions and multiplied with the 32
// activations the lane holds in registers for all 8 rows.  Products and sums
// in fp32, in a fixed order.  Bound: HBM (the weights, 17/32 byte per value,
// read once per token that uses them).
#include "moe_internal.h"
#include "mx_device.h"

namespace bitffn {
namespace {

constexpr int MD_THREADS = 256;
constexpr int MD_WAVES = MD_THREADS / 64;
constexpr int MD_ROWS = 8;   // consecutive weight rows per lane group

typedef uint32_t du4 __attribute__((ext_vector_type(4)));

struct DecodeArgs {
  const uint8_t* gc;   // gate/up codes, scales
  const uint8_t* gs;
  const uint8_t* dc;   // down codes, scales
  const uint8_t* ds;
  const float* x;
  const int32_t* slot;
  const float* w;
  float* h;            // [T][k+1][f]
  float* y;
  int T, k, d, f, n_mats, shared_slot;
};

// Slot of pair i of token t (the shared expert for i = k); -1: none.
__device__ __forceinline__ int pair_slot(const DecodeArgs& a, int t, int i) {
  if (i == a.k) return a.shared_slot;
  const int s = a.slot[t * a.k + i];
  return s >= 0 && s < a.n_mats ? s : -1;
}

// acc[r] += wgt * (rows row0 + r, r < 8, of the matrix at codes/scales, times
// v), the part of this lane: blocks kb = l, l + LPR, ...
template <int LPR>
__device__ __forceinline__ void dot_rows(const uint8_t* __restrict__ codes,
                                         const uint8_t* __restrict__ scales, int64_t row0, int nb,
                                         const float* __restrict__ v, int l, float wgt,
                                         float (&acc)[MD_ROWS]) {
  for (int kb = l; kb < nb; kb += LPR) {
    du4 c[MD_ROWS];
    uint32_t s[MD_ROWS];
#pragma unroll
    for (int r = 0; r < MD_ROWS; ++r) {
      const int64_t at = (row0 + r) * nb + kb;
      c[r] = __builtin_nontemporal_load(reinterpret_cast<const du4*>(codes + 16 * at));
      s[r] = scales[at];
    }
    float4 xv[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) xv[j] = reinterpret_cast<const float4*>(v + 32 * kb)[j];
#pragma unroll
    for (int r = 0; r < MD_ROWS; ++r) {
      float sum = 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float f[8];
        mx_values8(c[r][q], s[r], f);
        const float4 a = xv[2 * q], b = xv[2 * q + 1];
        sum = fmaf(f[0], a.x, sum);
        sum = fmaf(f[1], a.y, sum);
        sum = fmaf(f[2], a.z, sum);
        sum = fmaf(f[3], a.w, sum);
        sum = fmaf(f[4], b.x, sum);
        sum = fmaf(f[5], b.y, sum);
        sum = fmaf(f[6], b.z, sum);
        sum = fmaf(f[7], b.w, sum);
      }
      acc[r] = fmaf(wgt, sum, acc[r]);
    }
  }
}

// The 8 sums over each group of LPR lanes: three halving exchanges leave one
// of them per lane, row 4 (l & 1) + (l & 2) + (l >> 2 & 1), the rest are plain
// butterflies.
template <int LPR>
__device__ __forceinline__ float reduce_rows(float (&v)[MD_ROWS], int l) {
#pragma unroll
  for (int st = 0; st < 3; ++st) {
    const int half = 4 >> st;
    const bool up = (l >> st) & 1;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float send = up ? v[i] : v[i + half];
      const float keep = up ? v[i + half] : v[i];
      v[i] = keep + __shfl_xor(send, 1 << st, 64);
    }
  }
  float s = v[0];
#pragma unroll
  for (int off = 8; off < LPR; off <<= 1) s += __shfl_xor(s, off, 64);
  return s;
}

__device__ __forceinline__ int reduced_row(int l) {
  return 4 * (l & 1) + (l & 2) + ((l >> 2) & 1);
}

template <int LPR>
__global__ __launch_bounds__(MD_THREADS) void mx_decode_gate_up_kernel(DecodeArgs a) {
  constexpr int SUB = 64 / LPR;
  const int t = static_cast<int>(blockIdx.y) / (a.k + 1), i = static_cast<int>(blockIdx.y) % (a.k + 1);
  const int s = pair_slot(a, t, i);
  if (s < 0) return;
  const int lane = threadIdx.x & 63, l = lane % LPR;
  const int row0 = (static_cast<int>(blockIdx.x) * MD_WAVES + (static_cast<int>(threadIdx.x) >> 6)) *
                       (MD_ROWS * SUB) + MD_ROWS * (lane / LPR);
  if (row0 >= 2 * a.f) return;   // uniform per wavefront: 2f is a multiple of 64
  float acc[MD_ROWS] = {};
  dot_rows<LPR>(a.gc, a.gs, static_cast<int64_t>(s) * 2 * a.f + row0, a.d / 32,
                a.x + static_cast<int64_t>(t) * a.d, l, 1.0f, acc);
  const float g = reduce_rows<LPR>(acc, l);
  const float u = __shfl_xor(g, 4, 64);   // the odd row of the pair
  if (l < 4)
    a.h[(static_cast<int64_t>(t) * (a.k + 1) + i) * a.f + (row0 + reduced_row(l)) / 2] = silu(g) * u;
}

template <int LPR>
__global__ __launch_bounds__(MD_THREADS) void mx_decode_down_kernel(DecodeArgs a) {
  constexpr int SUB = 64 / LPR;
  constexpr int WG_ROWS = MD_ROWS * SUB;
  __shared__ float part[MD_WAVES][WG_ROWS];
  const int t = blockIdx.y;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane % LPR;
  const int base = static_cast<int>(blockIdx.x) * WG_ROWS;
  const int row0 = base + MD_ROWS * (lane / LPR);
  float acc[MD_ROWS] = {};
  for (int i = wave; i <= a.k; i += MD_WAVES) {   // pairs of this wavefront, in order
    const int s = pair_slot(a, t, i);
    if (s < 0) continue;
    dot_rows<LPR>(a.dc, a.ds, static_cast<int64_t>(s) * a.d + row0, a.f / 32,
                  a.h + (static_cast<int64_t>(t) * (a.k + 1) + i) * a.f, l,
                  i == a.k ? 1.0f : a.w[t * a.k + i], acc);
  }
  const float v = reduce_rows<LPR>(acc, l);
  if (l < 8) part[wave][MD_ROWS * (lane / LPR) + reduced_row(l)] = v;
  __syncthreads();
  if (threadIdx.x < WG_ROWS) {
    const int64_t at = static_cast<int64_t>(t) * a.d + base + threadIdx.x;
    float y = a.x[at];
#pragma unroll
    for (int w = 0; w < MD_WAVES; ++w) y += part[w][threadIdx.x];
    a.y[at] = y;
  }
}

template <int LPR>
void launch_gate_up(const DecodeArgs& a, hipStream_t s) {
  constexpr int per = MD_WAVES * MD_ROWS * (64 / LPR);
  const dim3 grid((2 * a.f + per - 1) / per, a.T * (a.k + 1));
  mx_decode_gate_up_kernel<LPR><<<grid, MD_THREADS, 0, s>>>(a);
}

template <int LPR>
void launch_down(const DecodeArgs& a, hipStream_t s) {
  const dim3 grid(a.d / (MD_ROWS * (64 / LPR)), a.T);
  mx_decode_down_kernel<LPR><<<grid, MD_THREADS, 0, s>>>(a);
}

}  // namespace

size_t mx_decode_workspace_bytes(int T, int k, int f) {
  return static_cast<size_t>(align256(static_cast<int64_t>(T) * (k + 1) * f * 4));
}

hipError_t launch_mx_decode(const moe_mxfp4& GU, const moe_mxfp4& D, int shared_slot,
                            const float* x, int T, int k, const int32_t* slot, const float* w,
                            float* y, void* ws, hipStream_t s) {
  DecodeArgs a;
  a.gc = static_cast<const uint8_t*>(GU.codes);
  a.gs = static_cast<const uint8_t*>(GU.scales);
  a.dc = static_cast<const uint8_t*>(D.codes);
  a.ds = static_cast<const uint8_t*>(D.scales);
  a.x = x;
  a.slot = slot;
  a.w = w;
  a.h = static_cast<float*>(ws);
  a.y = y;
  a.T = T;
  a.k = k;
  a.d = GU.cols;
  a.f = D.cols;
  a.n_mats = GU.n_mats;
  a.shared_slot = shared_slot;
  const int nd = a.d / 32, nf = a.f / 32;
  nd <= 16 ? launch_gate_up<16>(a, s) : nd <= 32 ? launch_gate_up<32>(a, s) : launch_gate_up<64>(a, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  nf <= 16 ? launch_down<16>(a, s) : nf <= 32 ? launch_down<32>(a, s) : launch_down<64>(a, s);
  return hipGetLastError();
}

}  // namespace bitffn
