// Decode / verify FFN over 4-bit experts for 1..4 tokens, activations in fp32
// (moe_mxfp4_ffn_decode).  Two launches:
//   gate/up  h[t][i][j] = silu(g) u for every pair (t, i) whose slot is in the
//            pool, and for the shared expert (i = k);
//   down     y[t] = x[t] + sum_i w_i D_i h[t][i], all pairs of all tokens in one
//            workgroup per few output rows, so no partial result goes through
//            memory.
// Each expert is read once for all tokens that chose it: the first pair with a
// slot does the work of all pairs with it.
//
// A wavefront gives each weight row LPR lanes (16, 32 or 64, the least power of
// two that covers the row's blocks, so that few lanes idle); a lane holds one or
// two 32-value blocks of several consecutive rows, all requested at once, each
// dequantized by 16 conversions and multiplied with the 32 activations that
// belong to it.  Neighbouring lanes want activations 128 bytes apart, which
// costs the path from the caches four times what it moves; x therefore goes
// through LDS (16-byte piece c of block b at position c ^ swz(b), no two of 16
// lanes on one bank), and h is laid out piece by piece, so that the lanes of one
// load are neighbours.
// Products and sums in fp32, each in an order that no other token changes.
// Bound: HBM (the weights, 17/32 byte per value).
#include "moe_internal.h"
#include "mx_device.h"

namespace bitffn {
namespace {

constexpr int MD_UP_ROWS = 8;      // consecutive weight rows per lane group: gate/up
constexpr int MD_UP_THREADS = 256;
constexpr int MD_DOWN_ROWS = 4;    // and down
constexpr int MD_DOWN_THREADS = 1024;
constexpr int MD_MAX_ITER = 2;     // blocks of a row per lane: 4096 columns over 64 lanes

typedef uint32_t du4 __attribute__((ext_vector_type(4)));

struct DecodeArgs {
  const uint8_t* gc;   // gate/up codes, scales
  const uint8_t* gs;
  const uint8_t* dc;   // down codes, scales
  const uint8_t* ds;
  const float* x;
  const int32_t* slot;
  const float* w;
  float* h;            // [T][k+1][8][f/32][4]: piece c of block b of pair (t, i)
  float* y;
  int T, k, d, f, n_mats, shared_slot;
};

__host__ __device__ constexpr int md_swz(int b) { return (b & 7) ^ ((b >> 3) & 1); }

// Lane p < T k: the slot of pair p, -1 if it is none.
__device__ __forceinline__ int lane_slot(const DecodeArgs& a) {
  const int lane = threadIdx.x & 63;
  const int s = lane < a.T * a.k ? a.slot[lane] : -1;
  return s >= 0 && s < a.n_mats ? s : -1;
}

// Row of h of pair p, and of token t's shared expert.
__device__ __forceinline__ int64_t h_row(const DecodeArgs& a, int p) {
  return static_cast<int64_t>(p / a.k) * (a.k + 1) + p % a.k;
}
__device__ __forceinline__ int64_t h_shared(const DecodeArgs& a, int t) {
  return static_cast<int64_t>(t) * (a.k + 1) + a.k;
}

// This lane's blocks l, l + LPR of rows row0 .. row0 + ROWS - 1.
template <int ROWS, int ITER>
struct Blocks {
  du4 c[ITER][ROWS];
  uint32_t s[ITER][ROWS];

  template <int LPR>
  __device__ __forceinline__ void load(const uint8_t* __restrict__ codes,
                                       const uint8_t* __restrict__ scales, int64_t row0, int nb, int l) {
#pragma unroll
    for (int it = 0; it < ITER; ++it)
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        // a lane past the row's end repeats its last block, with activations 0
        const int64_t at = (row0 + r) * nb + min(l + it * LPR, nb - 1);
        c[it][r] = __builtin_nontemporal_load(reinterpret_cast<const du4*>(codes + 16 * at));
        s[it][r] = scales[at];
      }
  }

  // sum[r] += block it of row r times v
  __device__ __forceinline__ void dot(int it, const float4 (&v)[8], float (&sum)[ROWS]) const {
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      float acc = sum[r];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float f[8];
        uint32_t word = c[it][r][q];
        opaque(word);   // its values are formed here, not kept over the loop of tokens
        mx_values8(word, s[it][r], f);
        const float4 x = v[2 * q], y = v[2 * q + 1];
        acc = fmaf(f[0], x.x, acc);
        acc = fmaf(f[1], x.y, acc);
        acc = fmaf(f[2], x.z, acc);
        acc = fmaf(f[3], x.w, acc);
        acc = fmaf(f[4], y.x, acc);
        acc = fmaf(f[5], y.y, acc);
        acc = fmaf(f[6], y.z, acc);
        acc = fmaf(f[7], y.w, acc);
      }
      sum[r] = acc;
    }
  }
};

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}
// v of lane l ^ 1, l ^ 2, l ^ 8 (inside a row of 16 lanes), l ^ 4
__device__ __forceinline__ float from1(float v) { return dpp<0xB1>(v); }
__device__ __forceinline__ float from2(float v) { return dpp<0x4E>(v); }
__device__ __forceinline__ float from8(float v) { return dpp<0x128>(v); }
__device__ __forceinline__ float from4(float v) { return dpp<0x1B>(dpp<0x141>(v)); }   // mirrored 8, mirrored 4

// The ROWS (4 or 8) sums over each group of LPR lanes.  Exchanges that halve
// what a lane keeps leave one row per lane (reduced_row), plain additions join
// the other lanes with the same row.
template <int ROWS, int LPR>
__device__ __forceinline__ float reduce_rows(const float (&v)[ROWS], int l) {
  float a[ROWS / 2], b[ROWS / 4], s;
#pragma unroll
  for (int i = 0; i < ROWS / 2; ++i) {
    const bool up = l & 1;
    a[i] = (up ? v[i + ROWS / 2] : v[i]) + from1(up ? v[i] : v[i + ROWS / 2]);
  }
#pragma unroll
  for (int i = 0; i < ROWS / 4; ++i) {
    const bool up = l & 2;
    b[i] = (up ? a[i + ROWS / 4] : a[i]) + from2(up ? a[i] : a[i + ROWS / 4]);
  }
  if constexpr (ROWS == 8) {
    const bool up = l & 8;
    s = (up ? b[1] : b[0]) + from8(up ? b[0] : b[1]);
  } else {
    s = b[0] + from8(b[0]);
  }
  s += from4(s);
#pragma unroll
  for (int off = 16; off < LPR; off <<= 1) s += __shfl_xor(s, off, 64);
  return s;
}

template <int ROWS>
__device__ __forceinline__ int reduced_row(int l) {
  return ROWS == 8 ? 4 * (l & 1) + (l & 2) + ((l >> 3) & 1) : 2 * (l & 1) + ((l >> 1) & 1);
}

template <int LPR, int ITER>
__global__ __launch_bounds__(MD_UP_THREADS) void mx_decode_gate_up_kernel(DecodeArgs a) {
  constexpr int SUB = 64 / LPR, WAVES = MD_UP_THREADS / 64;
  extern __shared__ float4 s_x[];   // a token's x, 8 pieces per block
  const int tid = threadIdx.x, lane = tid & 63, l = lane % LPR, n = a.T * a.k, p = blockIdx.y;
  const int slots = lane_slot(a);
  const int s = p < n ? __builtin_amdgcn_readlane(slots, p) : a.shared_slot;
  if (s < 0) return;
  // the pairs (bits) or tokens (shared expert) that this workgroup works for
  uint64_t todo = p < n ? __ballot(slots == s) : (1ull << a.T) - 1;
  if (p < n && __ffsll(static_cast<unsigned long long>(todo)) - 1 != p) return;   // an earlier pair's workgroup does it
  const int row0 = (static_cast<int>(blockIdx.x) * WAVES + (tid >> 6)) * (MD_UP_ROWS * SUB) + MD_UP_ROWS * (lane / LPR);
  const bool rows = row0 < 2 * a.f;   // uniform per wavefront: 2f is a multiple of 64
  const int nb = a.d / 32, nf = a.f / 32;
  Blocks<MD_UP_ROWS, ITER> w;
  w.template load<LPR>(a.gc, a.gs, static_cast<int64_t>(s) * 2 * a.f + (rows ? row0 : 0), nb, l);
  for (; todo; todo &= todo - 1) {
    const int q = __ffsll(static_cast<unsigned long long>(todo)) - 1;
    const int t = p < n ? q / a.k : q;
    const float4* __restrict__ x = reinterpret_cast<const float4*>(a.x + static_cast<int64_t>(t) * a.d);
    __syncthreads();   // the token before has been read
    for (int i = tid; i < 8 * nb; i += MD_UP_THREADS) s_x[(i & ~7) | ((i & 7) ^ md_swz(i >> 3))] = x[i];
    __syncthreads();
    float sum[MD_UP_ROWS] = {};
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
      const int b = l + it * LPR, bc = min(b, nb - 1);
      float4 v[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float4 q4 = s_x[8 * bc + (c ^ md_swz(bc))];
        v[c] = b < nb ? q4 : make_float4(0, 0, 0, 0);
      }
      w.dot(it, v, sum);
    }
    const float g = reduce_rows<MD_UP_ROWS, LPR>(sum, l);
    const float u = from8(g);   // the odd row of the pair
    if (rows && l < 4) {        // bits 0 and 1 name the even row
      const int j = (row0 + reduced_row<MD_UP_ROWS>(l)) / 2;
      float* __restrict__ h = a.h + (p < n ? h_row(a, q) : h_shared(a, t)) * a.f;
      h[((j % 32 / 4) * nf + j / 32) * 4 + j % 4] = silu(g) * u;
    }
  }
}

template <int LPR, int ITER>
__global__ __launch_bounds__(MD_DOWN_THREADS) void mx_decode_down_kernel(DecodeArgs a) {
  constexpr int SUB = 64 / LPR, WAVES = MD_DOWN_THREADS / 64, WG_ROWS = MD_DOWN_ROWS * SUB;
  __shared__ float part[MOE_MAX_DECODE_PAIRS + MOE_MAX_DECODE_T][WG_ROWS];
  __shared__ int s_slot[MOE_MAX_DECODE_PAIRS];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l = lane % LPR, n = a.T * a.k;
  const int base = static_cast<int>(blockIdx.x) * WG_ROWS;
  const int row0 = base + MD_DOWN_ROWS * (lane / LPR);
  const int nf = a.f / 32;
  const int slots = lane_slot(a);
  if (wave == 0) s_slot[lane] = slots;
  // the pairs that do the work of all pairs with their slot
  bool first = slots >= 0;
  if (a.T > 1)
    for (int q = 0; q < n; ++q)
      if (__builtin_amdgcn_readlane(slots, q) == slots && q < lane) first = false;
  uint64_t leaders = __ballot(first);
  const int jobs = __popcll(leaders) + (a.shared_slot >= 0 ? 1 : 0);
  for (int i = 0; i < wave; ++i) leaders &= leaders - 1;
  for (int j = wave; j < jobs; j += WAVES) {
    const bool routed = leaders != 0;
    const int p = routed ? __ffsll(static_cast<unsigned long long>(leaders)) - 1 : 0;
    const int s = routed ? __builtin_amdgcn_readlane(slots, p) : a.shared_slot;
    Blocks<MD_DOWN_ROWS, ITER> w;
    w.template load<LPR>(a.dc, a.ds, static_cast<int64_t>(s) * a.d + row0, nf, l);
    uint64_t todo = !routed ? (1ull << a.T) - 1 : a.T > 1 ? __ballot(slots == s) : 1ull << p;
    for (; todo; todo &= todo - 1) {
      const int q = __ffsll(static_cast<unsigned long long>(todo)) - 1;
      const float4* __restrict__ h =
          reinterpret_cast<const float4*>(a.h + (routed ? h_row(a, q) : h_shared(a, q)) * a.f);
      float sum[MD_DOWN_ROWS] = {};
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        const int b = l + it * LPR, bc = min(b, nf - 1);
        float4 v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float4 q4 = h[c * nf + bc];
          v[c] = b < nf ? q4 : make_float4(0, 0, 0, 0);
        }
        w.dot(it, v, sum);
      }
      const float r = reduce_rows<MD_DOWN_ROWS, LPR>(sum, l);
      if (l < 4) part[routed ? q : MOE_MAX_DECODE_PAIRS + q][MD_DOWN_ROWS * (lane / LPR) + reduced_row<MD_DOWN_ROWS>(l)] = r;
    }
    for (int i = 0; i < WAVES; ++i) leaders &= leaders - 1;
  }
  __syncthreads();
  if (tid < a.T * WG_ROWS) {
    const int t = tid / WG_ROWS, r = tid % WG_ROWS;
    const int64_t at = static_cast<int64_t>(t) * a.d + base + r;
    float y = a.x[at];
    for (int i = 0; i < a.k; ++i)
      if (s_slot[t * a.k + i] >= 0) y = fmaf(a.w[t * a.k + i], part[t * a.k + i][r], y);
    if (a.shared_slot >= 0) y += part[MOE_MAX_DECODE_PAIRS + t][r];
    a.y[at] = y;
  }
}

template <int LPR, int ITER>
void launch_gate_up(const DecodeArgs& a, hipStream_t s) {
  constexpr int per = MD_UP_THREADS / 64 * MD_UP_ROWS * (64 / LPR);
  const dim3 grid((2 * a.f + per - 1) / per, a.T * a.k + (a.shared_slot >= 0 ? 1 : 0));
  if (grid.y > 0) mx_decode_gate_up_kernel<LPR, ITER><<<grid, MD_UP_THREADS, a.d * 4, s>>>(a);
}

template <int LPR, int ITER>
void launch_down(const DecodeArgs& a, hipStream_t s) {
  mx_decode_down_kernel<LPR, ITER><<<a.d / (MD_DOWN_ROWS * (64 / LPR)), MD_DOWN_THREADS, 0, s>>>(a);
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
  static_assert(4096 / 32 <= 64 * MD_MAX_ITER, "blocks of the longest row");
  if (nd <= 16)
    launch_gate_up<16, 1>(a, s);
  else if (nd <= 32)
    launch_gate_up<32, 1>(a, s);
  else if (nd <= 64)
    launch_gate_up<64, 1>(a, s);
  else
    launch_gate_up<64, 2>(a, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (nf <= 16)
    launch_down<16, 1>(a, s);
  else if (nf <= 32)
    launch_down<32, 1>(a, s);
  else if (nf <= 64)
    launch_down<64, 1>(a, s);
  else
    launch_down<64, 2>(a, s);
  return hipGetLastError();
}

}  // namespace bitffn
