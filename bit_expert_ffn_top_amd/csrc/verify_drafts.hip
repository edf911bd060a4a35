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
// Measured (fp32, three drafts, 64 requests unless said): 131,072 values 11.3 + 4.2 us;
// most drafts are accepted there, and a request that keeps all of its drafts reads no
// row of q, so that is 42 MB, 8 us at a copy's rate: what is left is that chain of reads
// before the rows' own.  On both sides of the border, in a graph of calls: 16,384
// values in one launch 8.3 us, 16,385 in two 8.6; one request 5.8 and 7.2; bfloat16 8.3
// and 8.5, 6.3 and 6.8.  A call pays 4 us more for the second launch and its workspace.
#include "moe_internal.h"
#include "row_device.h"
#include "scan_device.h"

namespace bitffn {
namespace {

constexpr int kLane = 16;               // values of a lane
constexpr int kChunk = 64 * kLane;
constexpr int kShortWaves = 16;         // chunks of a row that one workgroup takes
constexpr int kSumWaves = 4;            // chunks per workgroup of the first launch

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

// The sum over the wavefront, the same for all lanes.
__device__ __forceinline__ double wave_sum(double v) { return lane_value(wave_scan_add(v), 63); }

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
  constexpr int G = kLane / 4;
  double s[G][4], scan[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < 4; ++j) s[g][j] = sum += c.left(r, g, j);
    scan[g] = wave_scan_add(sum);
  }
  int last = -1;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const double lower = before + lane_before(scan[g]);
    int at = -1, mine = -1;   // this lane's first value that passes the border; its last above 0
#pragma unroll
    for (int j = 3; j >= 0; --j) {
      if (!(c.left(r, g, j) > 0.0)) continue;
      if (lower + s[g][j] > want) at = c.v0 + 256 * g + j;
      mine = max(mine, c.v0 + 256 * g + j);
    }
    const uint64_t hit = __ballot(at >= 0);
    if (hit) return lane_value(at, __builtin_ctzll(hit));
    const uint64_t some = __ballot(mine >= 0);
    if (some) last = lane_value(mine, 63 - __builtin_clzll(some));
    before += lane_value(scan[g], 63);
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

// The chunk whose sums pass the border, or else the last that adds anything (-1:
// none does), and the sum before it.  Each lane owns a run of consecutive chunks,
// four of them in registers.
__device__ __forceinline__ int find_chunk(const double* sums, int chunks, float u, double& before,
                                          double& want) {
  constexpr int kHeld = 4;
  const int lane = threadIdx.x & 63;
  const int per = (chunks + 63) / 64;
  const int c0 = min(chunks, lane * per), c1 = min(chunks, c0 + per);
  double held[kHeld], mine = 0.0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) held[i] = c0 + i < c1 ? sums[c0 + i] : 0.0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) mine += held[i];
  for (int c = c0 + kHeld; c < c1; ++c) mine += sums[c];
  const double scan = wave_scan_add(mine);
  const double total = lane_value(scan, 63);
  want = border(u, total);
  int first = -1, last = -1;
  double first_before = 0.0, last_before = 0.0, sum = lane_before(scan);
  const auto look = [&](int c, double add) {
    if (add > 0.0) {
      last = c;
      last_before = sum;
      if (first < 0 && sum + add > want) {
        first = c;
        first_before = sum;
      }
    }
    sum += add;
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (c0 + i < c1) look(c0 + i, held[i]);
  for (int c = c0 + kHeld; c < c1; ++c) look(c, sums[c]);
  const uint64_t hit = __ballot(first >= 0), some = __ballot(last >= 0);
  if (hit) {
    const int who = __builtin_ctzll(hit);
    before = lane_value(first_before, who);
    return lane_value(first, who);
  }
  if (!some) return -1;
  const int who = 63 - __builtin_clzll(some);
  before = lane_value(last_before, who);
  return lane_value(last, who);
}

// One wavefront per request.
template <typename PT>
__global__ __launch_bounds__(64) void verify_pick_kernel(VerifyArgs a) {
  const int64_t b = blockIdx.x;
  const int given = drafts_given(a, b);
  const int m = __builtin_amdgcn_readfirstlane(a.n_accepted[b]);
  const float u = a.u_sample[b];
  double before = 0.0, want;
  int at = find_chunk(a.sums + b * a.chunks, a.chunks, u, before, want);
  const bool all = m >= given || at < 0;
  if (at < 0) at = find_chunk(a.sums + (a.B + b) * a.chunks, a.chunks, u, before, want);
  int pick = -1;
  if (at >= 0) {
    const Rest<PT> r = rest_of<PT>(a, b, m, all, all || a.q ? -1 : a.draft[b * a.n + m]);
    ChunkValues<PT> c;
    c.load(r, at, a.V);
    pick = pick_in_chunk(c, r, before, want);
  }
  if (threadIdx.x == 0) a.tokens[b * (a.n + 1) + m] = pick;
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
  verify_pick_kernel<PT><<<a.B, 64, 0, s>>>(a);
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
