// Verification of drafted tokens: how many are accepted, and the token that
// follows, drawn by inverting the cumulative sum of r, what is left of the
// target's probabilities.
//
// A row is cut into chunks of 1,024 values, one per wavefront.  Short rows (16
// chunks) are one launch, a workgroup per request that keeps its values in
// registers: sums of the chunks, the chunk whose sums pass the border, the value
// in it.  Long rows are two launches, since one CU reads 1 MB in about 70 us:
// all sums first, over the whole card, then per request the chunk, which is read
// again, and the value.  Each wavefront of the first launch judges the drafts for
// itself (two dependent reads) rather than wait for a launch that does.  Should
// nothing be left of p, p itself is drawn from: its sums are formed beside r's.
#include "moe_internal.h"
#include "row_device.h"

namespace bitffn {
namespace {

constexpr int kLane = 16;               // values of a lane
constexpr int kChunk = 64 * kLane;
constexpr int kShortWaves = 16;         // chunks of a row that one workgroup takes
constexpr int kSumWaves = 4;            // chunks per workgroup of the first launch
constexpr int kPickThreads = 256;

struct VerifyArgs {
  const void* p;
  const void* q;
  const int32_t* draft;
  const int32_t* n_draft;
  const float* u_accept;
  const float* u_sample;
  int32_t* tokens;
  int32_t* n_accepted;
  double* sums;     // [2][B][chunks]: r's, then p's own
  int B, n, V, chunks;
  int b0;           // first request of a launch of the sums
};

__device__ __forceinline__ float prob(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float prob(const uint16_t* p, int64_t i) { return bf16_bits_to_float(p[i]); }

// The row a request draws from: p less q (a row, or the draft `gone` alone).
template <typename PT>
struct Rest {
  const PT* p;
  const PT* q;
  int gone;
  __device__ __forceinline__ bool less() const { return q || gone >= 0; }
};

__device__ __forceinline__ int drafts_given(const VerifyArgs& a, int64_t b) {
  return a.n_draft ? min(max(a.n_draft[b], 0), a.n) : a.n;
}

template <typename PT>
__device__ __forceinline__ Rest<PT> rest_of(const VerifyArgs& a, int64_t b, int m, bool all, int x) {
  Rest<PT> r;
  r.p = static_cast<const PT*>(a.p) + (b * (a.n + 1) + m) * a.V;
  r.q = a.q && !all ? static_cast<const PT*>(a.q) + (b * a.n + m) * a.V : nullptr;
  r.gone = !a.q && !all ? x : -1;
  return r;
}

// Lane i judges draft i; u * q < p in 64 bits, where the product is exact.
// Returns the number accepted (the same in all lanes); x: the lane's draft.
template <typename PT>
__device__ __forceinline__ int judge(const VerifyArgs& a, int64_t b, int given, int& x) {
  const int lane = threadIdx.x & 63;
  bool ok = false;
  x = -1;
  if (lane < given) {
    x = a.draft[b * a.n + lane];
    if (x >= 0 && x < a.V) {
      const float px = prob(static_cast<const PT*>(a.p) + (b * (a.n + 1) + lane) * a.V, x);
      const float qx = a.q ? prob(static_cast<const PT*>(a.q) + (b * a.n + lane) * a.V, x) : 1.0f;
      ok = static_cast<double>(a.u_accept[b * a.n + lane]) * qx < static_cast<double>(px);
    }
  }
  return __builtin_ctzll(~__ballot(ok));   // MOE_MAX_DRAFTS = 63: lane 63 accepts nothing
}

// Four consecutive values.  Rows start at any element, and a wide load needs no
// more alignment than its elements.
__device__ __forceinline__ void load4(const float* p, float (&f)[4]) {
  typedef float f4 __attribute__((ext_vector_type(4), aligned(4)));
  const f4 w = *reinterpret_cast<const f4*>(p);
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = w[j];
}
__device__ __forceinline__ void load4(const uint16_t* p, float (&f)[4]) {
  typedef uint32_t u2 __attribute__((ext_vector_type(2), aligned(2)));
  const u2 w = *reinterpret_cast<const u2*>(p);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    f[j] = __builtin_bit_cast(float, j % 2 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
}

__device__ __forceinline__ double counted(double r) { return r > 0.0 && r < INFINITY ? r : 0.0; }

// Lane's values of a chunk, p and q: 4 at v0 + 4 lane, 4 at 256 further, ...
template <typename PT>
struct ChunkValues {
  float p[kLane / 4][4], q[kLane / 4][4];
  int v0;

  __device__ __forceinline__ void load(const Rest<PT>& r, int chunk, int V) {
    v0 = chunk * kChunk + 4 * (threadIdx.x & 63);
    if ((chunk + 1) * kChunk <= V) {   // uniform: no lane's load depends on a comparison
#pragma unroll
      for (int g = 0; g < kLane / 4; ++g) load4(r.p + v0 + 256 * g, p[g]);
      if (r.q) {
#pragma unroll
        for (int g = 0; g < kLane / 4; ++g) load4(r.q + v0 + 256 * g, q[g]);
      }
      return;
    }
#pragma unroll
    for (int g = 0; g < kLane / 4; ++g)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int v = v0 + 256 * g + j;
        p[g][j] = v < V ? prob(r.p, v) : 0.0f;
        q[g][j] = r.q && v < V ? prob(r.q, v) : 0.0f;
      }
  }
  __device__ __forceinline__ double left(const Rest<PT>& r, int g, int j) const {
    double v = p[g][j];
    if (r.q)
      v -= q[g][j];
    else if (v0 + 256 * g + j == r.gone)
      v = 0.0;
    return counted(v);
  }
};

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

// (sum of r, sum of p's own values) of a wavefront's chunk, in every lane.
template <typename PT>
__device__ __forceinline__ void chunk_sums(const ChunkValues<PT>& c, const Rest<PT>& r, double& rest,
                                           double& own) {
  rest = own = 0.0;
#pragma unroll
  for (int g = 0; g < kLane / 4; ++g)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      rest += c.left(r, g, j);
      own += counted(c.p[g][j]);
    }
  rest = wave_sum(rest);
  own = r.less() ? wave_sum(own) : rest;
}

// The first value of the chunk whose sum from `before` on passes `want`, else the
// last one above 0.  One wavefront; the chunk holds a value above 0.
template <typename PT>
__device__ __forceinline__ int pick_in_chunk(const ChunkValues<PT>& c, const Rest<PT>& r,
                                             double before, double want) {
  const int lane = threadIdx.x & 63;
  int last = -1;
#pragma unroll
  for (int g = 0; g < kLane / 4; ++g) {
    double s[4], sum = 0.0;
    int mine = -1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const double v = c.left(r, g, j);
      sum += v;
      s[j] = sum;
      if (v > 0.0) mine = c.v0 + 256 * g + j;
    }
    double scan = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const double up = __shfl_up(scan, off);
      if (lane >= off) scan += up;
    }
    double lower = __shfl_up(scan, 1);
    if (lane == 0) lower = 0.0;
    int at = -1;   // first value of this lane that passes the border
#pragma unroll
    for (int j = 3; j >= 0; --j)
      if (c.left(r, g, j) > 0.0 && before + (lower + s[j]) > want) at = c.v0 + 256 * g + j;
    const uint64_t hit = __ballot(at >= 0);
    if (hit) return __shfl(at, __builtin_ctzll(hit));
    const uint64_t some = __ballot(mine >= 0);
    if (some) last = __shfl(mine, 63 - __builtin_clzll(some));
    before += __shfl(scan, 63);
  }
  return last;
}

__device__ __forceinline__ double border(float u, double total) {
  return static_cast<double>(u < 0.0f ? 0.0f : u) * total;
}

__device__ __forceinline__ void put_accepted(const VerifyArgs& a, int64_t b, int m, int x) {
  const int lane = threadIdx.x & 63;   // n < 64; place m is the drawn token's
  if (lane <= a.n && lane != m) a.tokens[b * (a.n + 1) + lane] = lane < m ? x : -1;
  if (lane == 0) a.n_accepted[b] = m;
}

template <typename PT>
__global__ __launch_bounds__(64 * kShortWaves) void verify_short_kernel(VerifyArgs a) {
  __shared__ double s_sum[2][kShortWaves];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t b = blockIdx.x;
  const int given = drafts_given(a, b);
  const float u = a.u_sample[b];
  int x;
  const int m = judge<PT>(a, b, given, x);
  Rest<PT> r = rest_of<PT>(a, b, m, m >= given, __shfl(x, m));
  ChunkValues<PT> c;
  c.load(r, wave, a.V);
  double rest, own;
  chunk_sums(c, r, rest, own);
  if (lane == 0) {
    s_sum[0][wave] = rest;
    s_sum[1][wave] = own;
  }
  if (wave == 0) put_accepted(a, b, m, x);
  __syncthreads();
  double total = 0.0;
  for (int w = 0; w < a.chunks; ++w) total += s_sum[0][w];
  const int which = total > 0.0 ? 0 : 1;
  if (which) {
    r.q = nullptr;
    r.gone = -1;
    total = 0.0;
    for (int w = 0; w < a.chunks; ++w) total += s_sum[1][w];
  }
  const double want = border(u, total);
  // the first chunk that passes the border, else the last that adds anything
  int at = -1;
  double before = 0.0, sum = 0.0;
  for (int w = 0; w < a.chunks; ++w) {
    const double add = s_sum[which][w];
    if (add > 0.0) {
      at = w;
      before = sum;
    }
    sum += add;
    if (sum > want) break;
  }
  if (at == wave) {
    const int pick = pick_in_chunk(c, r, before, want);
    if (lane == 0) a.tokens[b * (a.n + 1) + m] = pick;
  } else if (at < 0 && threadIdx.x == 0) {
    a.tokens[b * (a.n + 1) + m] = -1;
  }
}

template <typename PT>
__global__ __launch_bounds__(64 * kSumWaves) void verify_sums_kernel(VerifyArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t b = a.b0 + blockIdx.y;
  const int chunk = blockIdx.x * kSumWaves + (threadIdx.x >> 6);
  if (chunk >= a.chunks) return;
  const int given = drafts_given(a, b);
  int x;
  const int m = judge<PT>(a, b, given, x);
  const Rest<PT> r = rest_of<PT>(a, b, m, m >= given, __shfl(x, m));
  ChunkValues<PT> c;
  c.load(r, chunk, a.V);
  double rest, own;
  chunk_sums(c, r, rest, own);
  if (lane == 0) {
    a.sums[b * a.chunks + chunk] = rest;
    a.sums[(a.B + b) * a.chunks + chunk] = own;
  }
  if (chunk == 0) put_accepted(a, b, m, x);
}

// Sums over the threads before this one (fixed order), and the total.
__device__ __forceinline__ double block_before(double mine, double* s_wave, double& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double scan = mine;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const double up = __shfl_up(scan, off);
    if (lane >= off) scan += up;
  }
  if (lane == 63) s_wave[wave] = scan;
  double lower = __shfl_up(scan, 1);
  if (lane == 0) lower = 0.0;
  __syncthreads();
  double before = 0.0;
  total = 0.0;
  for (int w = 0; w < kPickThreads / 64; ++w) {
    if (w == wave) before = total;
    total += s_wave[w];
  }
  return before + lower;
}

template <typename PT>
__global__ __launch_bounds__(kPickThreads) void verify_pick_kernel(VerifyArgs a) {
  __shared__ double s_wave[2][kPickThreads / 64];
  __shared__ int s_first, s_last;
  __shared__ double s_first_before, s_last_before;
  const int tid = threadIdx.x;
  const int64_t b = blockIdx.x;
  const int given = drafts_given(a, b);
  const int m = a.n_accepted[b];
  const float u = a.u_sample[b];
  const int x = m < given ? a.draft[b * a.n + m] : -1;
  Rest<PT> r = rest_of<PT>(a, b, m, m >= given, x);
  // each thread owns a run of consecutive chunks
  const int per = (a.chunks + kPickThreads - 1) / kPickThreads;
  const int c0 = min(a.chunks, tid * per), c1 = min(a.chunks, c0 + per);
  if (tid == 0) {
    s_first = 1 << 30;
    s_last = -1;
  }
  const double* sums = a.sums + b * a.chunks;
  double mine = 0.0, total;
  for (int c = c0; c < c1; ++c) mine += sums[c];
  double before = block_before(mine, s_wave[0], total);
  if (!(total > 0.0)) {   // uniform
    r.q = nullptr;
    r.gone = -1;
    sums += static_cast<int64_t>(a.B) * a.chunks;
    mine = 0.0;
    for (int c = c0; c < c1; ++c) mine += sums[c];
    before = block_before(mine, s_wave[1], total);
  }
  const double want = border(u, total);
  int first = 1 << 30, last = -1;
  double first_before = 0.0, last_before = 0.0, sum = before;
  for (int c = c0; c < c1; ++c) {
    const double add = sums[c];
    if (add > 0.0) {
      last = c;
      last_before = sum;
      if (first == 1 << 30 && sum + add > want) {
        first = c;
        first_before = sum;
      }
    }
    sum += add;
  }
  if (first < 1 << 30) atomicMin(&s_first, first);
  if (last >= 0) atomicMax(&s_last, last);
  __syncthreads();
  if (first < 1 << 30 && first == s_first) s_first_before = first_before;
  if (last >= 0 && last == s_last) s_last_before = last_before;
  __syncthreads();
  if (tid >= 64) return;
  const bool found = s_first < 1 << 30;
  const int at = found ? s_first : s_last;
  int pick = -1;
  if (at >= 0) {
    ChunkValues<PT> c;
    c.load(r, at, a.V);
    pick = pick_in_chunk(c, r, found ? s_first_before : s_last_before, want);
  }
  if (tid == 0) a.tokens[b * (a.n + 1) + m] = pick;
}

template <typename PT>
hipError_t launch_as(VerifyArgs a, void* ws, hipStream_t s) {
  if (a.chunks <= kShortWaves) {
    verify_short_kernel<PT><<<a.B, 64 * a.chunks, 0, s>>>(a);
    return hipGetLastError();
  }
  a.sums = static_cast<double*>(ws);
  constexpr int kMost = 32768;   // rows of a launch's grid
  for (; a.b0 < a.B; a.b0 += kMost)
    verify_sums_kernel<PT><<<dim3((a.chunks + kSumWaves - 1) / kSumWaves, min(kMost, a.B - a.b0)),
                             64 * kSumWaves, 0, s>>>(a);
  verify_pick_kernel<PT><<<a.B, kPickThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t verify_workspace_bytes(int B, int V) {
  const int64_t chunks = (static_cast<int64_t>(V) + kChunk - 1) / kChunk;
  if (chunks <= kShortWaves) return 0;
  return static_cast<size_t>(align256(2 * B * chunks * 8));
}

hipError_t launch_verify_drafts(const void* p, const void* q, int dtype, int B, int n, int V,
                                const int32_t* draft, const int32_t* n_draft,
                                const float* u_accept, const float* u_sample, int32_t* tokens,
                                int32_t* n_accepted, void* ws, hipStream_t s) {
  const VerifyArgs a{p, q, draft, n_draft, u_accept, u_sample, tokens, n_accepted, nullptr,
                     B, n, V, (V + kChunk - 1) / kChunk, 0};
  return dtype == MOE_DTYPE_F32 ? launch_as<float>(a, ws, s) : launch_as<uint16_t>(a, ws, s);
}

}  // namespace bitffn
