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
//
// Bound: the reads of the weights (17/32 byte per value); what is above it is
// latency, so whatever does not depend on a load is asked for before it: x before
// the slots, the last step's weights and x before the rows, the next expert's rows
// before the present ones are used.  10 of 128 experts and the shared one, d = 2048,
// F = 768, the same ones again and again (so from the last-level cache): one
// token 6.2 + 4.8 us (27.6 MB: 2.5 TB/s), four tokens over 34 experts
// 14.4 + 11.9 us (86 MB: 3.3 TB/s).  The matrix cores were tried in place
// of the vector unit (activations as three bfloat16 parts): 10.7 + 13.6 and
// 22.4 + 30.0 us, for the parts' traffic through LDS.
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
typedef float df4 __attribute__((ext_vector_type(4)));

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
  uint32_t over_k;     // ceil(2^16 / k): p / k = p over_k / 2^16 for p, k <= 64
};

__host__ __device__ constexpr int md_swz(int b) { return (b & 7) ^ ((b >> 3) & 1); }

// Lane p < T k: the slot of pair p, -1 if it is none.
__device__ __forceinline__ int lane_slot(const DecodeArgs& a) {
  const int lane = threadIdx.x & 63;
  const int s = lane < a.T * a.k ? a.slot[lane] : -1;
  return s >= 0 && s < a.n_mats ? s : -1;
}

// Token of pair p; row of h of pair p and of token t's shared expert.
__device__ __forceinline__ int token_of(const DecodeArgs& a, int p) {
  return static_cast<int>(static_cast<uint32_t>(p) * a.over_k >> 16);
}
__device__ __forceinline__ int h_row(const DecodeArgs& a, int p) { return p + token_of(a, p); }
__device__ __forceinline__ int h_shared(const DecodeArgs& a, int t) { return t * (a.k + 1) + a.k; }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const uint8_t* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, bytes, 0x00020000);
}

// This lane's blocks l, l + LPR of rows row0 + ROWS g .. + ROWS - 1, g this
// lane's group in the wavefront.
template <int ROWS, int ITER>
struct Blocks {
  du4 c[ITER][ROWS];
  uint32_t s[ITER][ROWS];

  template <int LPR>
  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, int64_t row0, int nb) {
    const int lane = threadIdx.x & 63, l = lane % LPR, in_wave = lane / LPR * ROWS * nb;
    // buffers over the wavefront's rows: one address register for all loads of a block column
    const __amdgpu_buffer_rsrc_t cb = buffer(codes + row0 * nb * 16, 64 / LPR * ROWS * nb * 16);
    const __amdgpu_buffer_rsrc_t sb = buffer(scales + row0 * nb, 64 / LPR * ROWS * nb);
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
      // a lane past the row's end repeats its last block, and drops the sum
      const int at = in_wave + min(l + it * LPR, nb - 1);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        c[it][r] = __builtin_bit_cast(du4, __builtin_amdgcn_raw_buffer_load_b128(cb, at * 16, r * nb * 16, 2));
        s[it][r] = __builtin_amdgcn_raw_buffer_load_b8(sb, at, r * nb, 0);
      }
    }
  }

  // sum[r] += values 16 half .. 16 half + 15 of block it of row r times v
  __device__ __forceinline__ void dot(int it, int half, const df4 (&v)[4], float (&sum)[ROWS]) const {
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      uint32_t scale = s[it][r];
      opaque(scale);   // no wait for it before the activations are asked for
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float f[8];
        uint32_t word = c[it][r][2 * half + q];
        opaque(word);   // its values are formed here, not kept over the loop of tokens
        mx_values8(word, scale, f);
        const df4 x = v[2 * q], y = v[2 * q + 1];
        sum[r] = fmaf(f[0], x.x, sum[r]);
        sum[r] = fmaf(f[1], x.y, sum[r]);
        sum[r] = fmaf(f[2], x.z, sum[r]);
        sum[r] = fmaf(f[3], x.w, sum[r]);
        sum[r] = fmaf(f[4], y.x, sum[r]);
        sum[r] = fmaf(f[5], y.y, sum[r]);
        sum[r] = fmaf(f[6], y.z, sum[r]);
        sum[r] = fmaf(f[7], y.w, sum[r]);
      }
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
  constexpr int PER = (LPR * ITER * 8 + MD_UP_THREADS - 1) / MD_UP_THREADS;   // 16-byte pieces of x per thread
  __shared__ df4 s_x[LPR * ITER * 8];   // a token's x, 8 pieces per block
  const int tid = threadIdx.x, lane = tid & 63, l = lane % LPR, n = a.T * a.k;
  // the shared expert works for every token and comes first, so that its workgroups
  // are not the last to end (four tokens: 18.1 -> 15.0 us)
  const int p = a.shared_slot < 0 ? blockIdx.y : blockIdx.y == 0 ? n : blockIdx.y - 1;
  const int nb = a.d / 32, nf = a.f / 32;
  const auto fetch = [&](int t, df4 (&x)[PER]) {
    const df4* from = reinterpret_cast<const df4*>(a.x + t * a.d);
#pragma unroll
    for (int u = 0; u < PER; ++u) x[u] = from[static_cast<uint32_t>(min(tid + u * MD_UP_THREADS, 8 * nb - 1))];
  };
  const auto put = [&](const df4 (&x)[PER]) {   // places past the row get its last piece and are not read
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int i = min(tid + u * MD_UP_THREADS, LPR * ITER * 8 - 1);
      s_x[(i & ~7) | ((i & 7) ^ md_swz(i >> 3))] = x[u];
    }
  };
  // the first of the tokens worked for is the pair's own: asked for before the slots are known
  df4 x[PER];
  fetch(p < n ? token_of(a, p) : 0, x);
  const int slots = lane_slot(a);
  const int s = p < n ? __builtin_amdgcn_readlane(slots, p) : a.shared_slot;
  if (s < 0) return;
  // the pairs (bits) or tokens (shared expert) that this workgroup works for
  uint64_t todo = p < n ? __ballot(slots == s) : (1ull << a.T) - 1;
  if (p < n && __ffsll(static_cast<unsigned long long>(todo)) - 1 != p) return;   // an earlier pair's workgroup does it
  const int wave0 = __builtin_amdgcn_readfirstlane((static_cast<int>(blockIdx.x) * WAVES + (tid >> 6)) * (MD_UP_ROWS * SUB));
  const bool rows = wave0 < 2 * a.f;   // 2f is a multiple of 64: all of a wavefront's rows or none
  Blocks<MD_UP_ROWS, ITER> w;
  w.template load<LPR>(a.gc, a.gs, static_cast<int64_t>(s) * 2 * a.f + (rows ? wave0 : 0), nb);
  put(x);
  __builtin_amdgcn_sched_barrier(0);   // x is put there before the weights arrive
  for (;;) {
    const int q = __ffsll(static_cast<unsigned long long>(todo)) - 1;
    __syncthreads();
    float sum[MD_UP_ROWS] = {};
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
      const int b = l + it * LPR, bc = min(b, nb - 1);
      float before[MD_UP_ROWS];
#pragma unroll
      for (int r = 0; r < MD_UP_ROWS; ++r) before[r] = sum[r];
#pragma unroll
      for (int half = 0; half < 2; ++half) {   // half a block's activations at a time: 90 registers, five wavefronts a SIMD
        df4 v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = s_x[8 * bc + ((4 * half + c) ^ md_swz(bc))];
        w.dot(it, half, v, sum);
      }
#pragma unroll
      for (int r = 0; r < MD_UP_ROWS; ++r) sum[r] = b < nb ? sum[r] : before[r];
    }
    const float g = reduce_rows<MD_UP_ROWS, LPR>(sum, l);
    const float u = from8(g);   // the odd row of the pair
    if (rows && l < 4) {        // bits 0 and 1 name the even row
      const int j = (wave0 + MD_UP_ROWS * (lane / LPR) + reduced_row<MD_UP_ROWS>(l)) / 2;
      float* __restrict__ h = a.h + (p < n ? h_row(a, q) : h_shared(a, q)) * a.f;
      h[((j % 32u / 4) * nf + j / 32u) * 4 + j % 4u] = silu(g) * u;
    }
    todo &= todo - 1;
    if (!todo) return;
    const int next = __ffsll(static_cast<unsigned long long>(todo)) - 1;
    df4 y[PER];
    fetch(p < n ? token_of(a, next) : next, y);
    __syncthreads();   // the token before has been read
    put(y);
  }
}

template <int LPR, int ITER>
__global__ __launch_bounds__(MD_DOWN_THREADS) void mx_decode_down_kernel(DecodeArgs a) {
  constexpr int SUB = 64 / LPR, WAVES = MD_DOWN_THREADS / 64, WG_ROWS = MD_DOWN_ROWS * SUB;
  __shared__ float part[MOE_MAX_DECODE_PAIRS + MOE_MAX_DECODE_T][WG_ROWS];
  __shared__ int s_slot[MOE_MAX_DECODE_PAIRS];
  __shared__ float s_weight[MOE_MAX_DECODE_PAIRS];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = lane % LPR;
  const int n = a.T * a.k, base = static_cast<int>(blockIdx.x) * WG_ROWS, nf = a.f / 32;
  constexpr bool AHEAD = ITER == 1;   // there are registers for two jobs' rows
  const int slots = lane_slot(a);
  // what the last step needs, asked for before the rows
  const float weight = wave == 0 && lane < n ? a.w[lane] : 0.0f;
  const int64_t out = static_cast<int64_t>(tid / WG_ROWS) * a.d + base + tid % WG_ROWS;   // of y, of the first threads
  const float residual = tid < a.T * WG_ROWS ? a.x[out] : 0.0f;
  if (wave == 0) s_slot[lane] = slots, s_weight[lane] = weight;
  // the pairs that do the work of all pairs with their slot
  bool first = slots >= 0;
  if (a.T > 1)
    for (int q = 0; q < n; ++q)
      if (__builtin_amdgcn_readlane(slots, q) == slots && q < lane) first = false;
  uint64_t leaders = __ballot(first);
  const int jobs = __popcll(leaders) + (a.shared_slot >= 0 ? 1 : 0);
  for (int i = 0; i < wave; ++i) leaders &= leaders - 1;
  // Expert of the job named by the lowest bit of leaders, the shared one if there is none.
  const auto expert = [&]() {
    const int p = leaders ? __ffsll(static_cast<unsigned long long>(leaders)) - 1 : 0;
    return leaders ? __builtin_amdgcn_readlane(slots, p) : a.shared_slot;
  };
  typedef Blocks<MD_DOWN_ROWS, ITER> Rows;
  const auto load = [&](Rows& w) {
    w.template load<LPR>(a.dc, a.ds, static_cast<int64_t>(expert()) * a.d + base, nf);
  };
  // The job's pairs; then leaders names this wavefront's next job.
  struct Job {
    bool routed;
    uint64_t todo;
  };
  const auto take = [&]() {
    Job job = {leaders != 0, 0};
    job.todo = !job.routed ? (1ull << a.T) - 1 : a.T > 1 ? __ballot(slots == expert()) : leaders & -leaders;
    for (int i = 0; i < WAVES; ++i) leaders &= leaders - 1;
    return job;
  };
  const auto work = [&](const Rows& w, const Job& job) {
    for (uint64_t todo = job.todo; todo; todo &= todo - 1) {
      const int q = __ffsll(static_cast<unsigned long long>(todo)) - 1;
      const df4* h = reinterpret_cast<const df4*>(a.h + (job.routed ? h_row(a, q) : h_shared(a, q)) * a.f);
      float sum[MD_DOWN_ROWS] = {};
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        const int b = l + it * LPR;
        const uint32_t bc = min(b, nf - 1);
        float before[MD_DOWN_ROWS];
#pragma unroll
        for (int r = 0; r < MD_DOWN_ROWS; ++r) before[r] = sum[r];
        df4 v[2][4];
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c / 4][c % 4] = (h + c * nf)[bc];
        w.dot(it, 0, v[0], sum);
        w.dot(it, 1, v[1], sum);
#pragma unroll
        for (int r = 0; r < MD_DOWN_ROWS; ++r) sum[r] = b < nf ? sum[r] : before[r];
      }
      const float r = reduce_rows<MD_DOWN_ROWS, LPR>(sum, l);
      if (l < 4)
        part[job.routed ? q : MOE_MAX_DECODE_PAIRS + q][MD_DOWN_ROWS * (lane / LPR) + reduced_row<MD_DOWN_ROWS>(l)] = r;
    }
  };
  Rows w;
  if constexpr (AHEAD) {   // the next job's rows on their way
    Rows u;
    if (wave < jobs) load(w);
    for (int j = wave; j < jobs; j += 2 * WAVES) {
      const Job first = take();
      if (j + WAVES < jobs) load(u);
      work(w, first);
      if (j + WAVES >= jobs) break;
      const Job second = take();
      if (j + 2 * WAVES < jobs) load(w);
      work(u, second);
    }
  } else {
    for (int j = wave; j < jobs; j += WAVES) {
      load(w);
      work(w, take());
    }
  }
  __syncthreads();
  if (tid < a.T * WG_ROWS) {
    const int t = tid / WG_ROWS, r = tid % WG_ROWS;
    float y = residual;
#pragma unroll 4
    for (int i = 0; i < a.k; ++i) {
      const float next = fmaf(s_weight[t * a.k + i], part[t * a.k + i][r], y);
      y = s_slot[t * a.k + i] >= 0 ? next : y;
    }
    if (a.shared_slot >= 0) y += part[MOE_MAX_DECODE_PAIRS + t][r];
    a.y[out] = y;
  }
}

template <int LPR, int ITER>
void launch_gate_up(const DecodeArgs& a, hipStream_t s) {
  constexpr int per = MD_UP_THREADS / 64 * MD_UP_ROWS * (64 / LPR);
  const dim3 grid((2 * a.f + per - 1) / per, a.T * a.k + (a.shared_slot >= 0 ? 1 : 0));
  if (grid.y > 0) mx_decode_gate_up_kernel<LPR, ITER><<<grid, MD_UP_THREADS, 0, s>>>(a);
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
  a.over_k = k ? (65536 + k - 1) / k : 0;
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
