// Verification of drafted tokens: how many are accepted, and the token that
// follows, drawn by inverting the cumulative sum of what is left of the target's
// probabilities.
#include "moe_internal.h"
#include "row_device.h"

namespace bitffn {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kPer = 4;                       // consecutive values of a thread
constexpr int kBlock = kThreads * kPer;       // values summed together
constexpr int kMaxBlocks = (1 << 24) / kBlock;

struct VerifyArgs {
  const void* p;
  const void* q;
  const int32_t* draft;
  const int32_t* n_draft;
  const float* u_accept;
  const float* u_sample;
  int32_t* tokens;
  int32_t* n_accepted;
  int n, V;
};

__device__ __forceinline__ double prob(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ double prob(const uint16_t* p, int64_t i) {
  return bf16_bits_to_float(p[i]);
}

// Value v of what is left: p - q (q: a row, or the draft `gone` alone), 0 where
// that is not above 0 or infinite.
template <typename PT>
__device__ __forceinline__ double left(const PT* p, const PT* q, int gone, int64_t v) {
  double r = prob(p, v);
  if (q)
    r -= prob(q, v);
  else if (v == gone)
    r = 0.0;
  return r > 0.0 && r < INFINITY ? r : 0.0;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

// One workgroup per request.
template <typename PT>
__global__ __launch_bounds__(kThreads) void verify_kernel(VerifyArgs a) {
  __shared__ double s_block[kMaxBlocks];
  __shared__ double s_wave[kWaves];
  __shared__ int s_pick, s_last, s_found;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t b = blockIdx.x;
  const int V = a.V;
  const int given = a.n_draft ? min(max(a.n_draft[b], 0), a.n) : a.n;
  const PT* p0 = static_cast<const PT*>(a.p) + b * (a.n + 1) * V;
  const PT* q0 = a.q ? static_cast<const PT*>(a.q) + b * a.n * V : nullptr;
  // accepted drafts: lane i of every wavefront judges draft i
  bool ok = false;
  int x = -1;
  if (lane < given) {
    x = a.draft[b * a.n + lane];
    if (x >= 0 && x < V) {
      const double qx = q0 ? prob(q0 + static_cast<int64_t>(lane) * V, x) : 1.0;
      ok = static_cast<double>(a.u_accept[b * a.n + lane]) * qx < prob(p0 + static_cast<int64_t>(lane) * V, x);
    }
  }
  const int m = __builtin_ctzll(~__ballot(ok));   // n <= 63: lane 63 accepts nothing
  if (wave == 0 && lane <= a.n) a.tokens[b * (a.n + 1) + lane] = lane < m ? x : -1;
  if (tid == 0) a.n_accepted[b] = m;
  const PT* p = p0 + static_cast<int64_t>(m) * V;
  const PT* q = nullptr;
  int gone = -1;
  if (m < given) {
    if (q0)
      q = q0 + static_cast<int64_t>(m) * V;
    else
      gone = __shfl(x, m);
  }
  const int blocks = (V + kBlock - 1) / kBlock;
  double total = 0.0;
  for (int round = 0; round < 2; ++round) {
    for (int k = 0; k < blocks; ++k) {
      double sum = 0.0;
      for (int j = 0; j < kPer; ++j) {
        const int64_t v = static_cast<int64_t>(k) * kBlock + tid * kPer + j;
        if (v < V) sum += left(p, q, gone, v);
      }
      sum = wave_sum(sum);
      if (lane == 0) s_wave[wave] = sum;
      __syncthreads();
      if (tid == 0) {
        for (int w = 0; w < kWaves; ++w) total += s_wave[w];
        s_block[k] = total;
      }
      __syncthreads();
    }
    total = s_block[blocks - 1];
    if (total > 0.0) break;
    q = nullptr;   // nothing left: the target's own probabilities
    gone = -1;
  }
  const float u = a.u_sample[b];
  const double want = static_cast<double>(u < 0.0f ? 0.0f : u) * total;
  if (tid == 0) {
    int k = 0;
    while (k < blocks && !(s_block[k] > want)) ++k;
    if (k == blocks)   // none: the last block that adds anything
      for (--k; k > 0 && !(s_block[k] > s_block[k - 1]);) --k;
    s_found = k;
    s_pick = 1 << 24;
    s_last = -1;
  }
  __syncthreads();
  // that block again: sums up to and including each value
  const int k = s_found;
  double c[kPer], sum = 0.0;
  int last = -1;
  for (int j = 0; j < kPer; ++j) {
    const int64_t v = static_cast<int64_t>(k) * kBlock + tid * kPer + j;
    const double r = v < V ? left(p, q, gone, v) : 0.0;
    sum += r;
    c[j] = sum;
    if (r > 0.0) last = static_cast<int>(v);
  }
  double scan = sum;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const double up = __shfl_up(scan, off);
    if (lane >= off) scan += up;
  }
  if (lane == 63) s_wave[wave] = scan;
  __syncthreads();
  double before = k > 0 ? s_block[k - 1] : 0.0;
  for (int w = 0; w < wave; ++w) before += s_wave[w];
  before += scan - sum;
  int pick = 1 << 24;
  for (int j = kPer - 1; j >= 0; --j) {
    const double r = j > 0 ? c[j] - c[j - 1] : c[0];
    if (r > 0.0 && before + c[j] > want) pick = k * kBlock + tid * kPer + j;
  }
  if (pick < 1 << 24) atomicMin(&s_pick, pick);
  if (last >= 0) atomicMax(&s_last, last);
  __syncthreads();
  if (tid == 0) a.tokens[b * (a.n + 1) + m] = s_pick < 1 << 24 ? s_pick : s_last;
}

}  // namespace

size_t verify_workspace_bytes(int, int) { return 0; }

hipError_t launch_verify_drafts(const void* p, const void* q, int dtype, int B, int n, int V,
                                const int32_t* draft, const int32_t* n_draft,
                                const float* u_accept, const float* u_sample, int32_t* tokens,
                                int32_t* n_accepted, void*, hipStream_t s) {
  const VerifyArgs a{p, q, draft, n_draft, u_accept, u_sample, tokens, n_accepted, n, V};
  if (dtype == MOE_DTYPE_F32)
    verify_kernel<float><<<B, kThreads, 0, s>>>(a);
  else
    verify_kernel<uint16_t><<<B, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace bitffn
