// The router's auxiliary losses, per-expert counts and logit gradients
// (moe_route_balance, moe_route_backward).
//
// A wavefront holds one row of logits in registers (lane l the experts
// VEC l + 64 VEC c .. + VEC - 1), so the row is read once: maximum, sum of
// exponentials and the probabilities come from the registers.
//
// Forward, two launches (one where all rows fit one workgroup and there are
// few sequences): rows are cut into chunks of a fixed length; a workgroup
// sums the probabilities of its chunk's rows per sequence (every lane keeps
// its experts' sums over the wavefront's rows, the wavefronts meet in LDS in
// order) and counts the chosen experts in an LDS histogram.  Chunk c and
// sequence s meet in at most one run of rows, and along the rows c + s only
// grows, so c + s numbers the partial results without gaps to search.  The
// second launch adds a sequence's partials chunk by chunk; the workgroup that
// finishes a sequence last adds up its loss, in a fixed order: nothing depends on
// which that is.
// Backward, one launch: a wavefront takes runs of consecutive rows, the
// coefficients of their sequence in registers.
// Bound: HBM (the logits once; the gradient written once).  65,536 rows of 512
// experts, 16 sequences: forward 34 us (137 MB: 4.0 TB/s; the rows 28.6, the
// second launch 6.4), backward 60 us (276 MB: 4.6 TB/s); 131 rows of 60 experts,
// 5 sequences: 11 us, two launches' latency.  Not for very many sequences: a
// workgroup of the first launch takes its chunk's one after the other, and the
// second has one to four for each (those 65,536 rows as 32,768 sequences of two:
// 0.3 + 3.6 ms; 4,096 rows of 60 experts in 1,024 sequences: 10 + 6 us).
#include "moe_internal.h"

namespace bitffn {
namespace {

constexpr int RB_WAVES = 16;
constexpr int RB_THREADS = RB_WAVES * 64;
constexpr int RB_HALF = RB_WAVES / 2;
constexpr int RB_MAX_CHUNKS = 256;    // one workgroup per CU on the largest inputs
constexpr int RB_SINGLE_ROWS = 64;    // single launch: rows and sequences
constexpr int RB_SINGLE_SEQS = 4;
constexpr int RB_ETILE = 128;         // experts per workgroup of the second launch
constexpr int RB_SUBS = 8;
constexpr int RB_FOLD = 64;           // rows a wavefront adds up before they join its total

struct BalanceArgs {
  const float* logits;
  const int32_t* idx;
  const int32_t* seq;     // [S+1] or null
  const uint8_t* mask;    // [T] or null
  float* balance;
  float* z;
  int32_t* counts;
  float* prob_sum;
  int32_t* n_tokens;
  // workspace
  float* p_part;          // [chunks + S][E]
  int32_t* c_part;        // [chunks + S][E]
  double* z_part;         // [chunks + S]
  int32_t* n_part;        // [chunks + S]
  double* l_part;         // [S][etiles]
  uint32_t* done;         // [S]
  int T, E, k, S, chunk_rows, n_chunks, n_etiles;
};

__host__ __device__ __forceinline__ int balance_chunk_rows(int T) {
  const int unit = RB_WAVES * RB_MAX_CHUNKS;
  return RB_WAVES * ((T + unit - 1) / unit);
}

__device__ __forceinline__ int seq_bound(const int32_t* seq, int s, int S, int T) {
  if (seq == nullptr) return s <= 0 ? 0 : T;
  return min(max(seq[s], 0), T);
}

// The sequence of row t: the last s with bound(s) <= t (empty ones before it
// are passed over), -1 before the first; S where t lies past the last.  All 64
// lanes of a wavefront, which asks for 64 bounds at a time.
__device__ __forceinline__ int seq_of_row(const int32_t* seq, int S, int T, int t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = S + 1;   // bounds lo .. lo + n - 1 may be <= t, all before are
  while (n > 64) {
    const int step = (n + 63) / 64;
    const int at = lo + lane * step;
    const bool below = lane * step < n && seq_bound(seq, at, S, T) <= t;
    const int k = __popcll(__ballot(below));   // pivots 0 .. k - 1
    if (k == 0) return lo - 1;
    const int end = lo + n;
    lo += (k - 1) * step;
    n = min(step, end - lo);
  }
  const bool below = lane < n && seq_bound(seq, lo + lane, S, T) <= t;
  return __builtin_amdgcn_readfirstlane(lo + __popcll(__ballot(below)) - 1);
}

// Sum and maximum over a wavefront, the same in every lane: the rows of 16
// lanes by lane permutes inside the vector unit, then the four of them.
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = row16_sum_dpp(v);
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}
template <int CTRL>
__device__ __forceinline__ float max_dpp(float v) {
  return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                      0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false)));
}
__device__ __forceinline__ float wave_max(float v) {
  v = max_dpp<0xB1>(v);    // quad_perm [1,0,3,2]
  v = max_dpp<0x4E>(v);    // quad_perm [2,3,0,1]
  v = max_dpp<0x124>(v);   // row_ror:4
  v = max_dpp<0x128>(v);   // row_ror:8
  return fmaxf(fmaxf(lane_value(v, 0), lane_value(v, 16)), fmaxf(lane_value(v, 32), lane_value(v, 48)));
}

// Orders this wavefront's LDS accesses for its own lanes (one wavefront's LDS
// accesses take effect in program order; this keeps the compiler to it).
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ bool finite(float v) { return fabsf(v) < __builtin_huge_valf(); }

typedef float rf4 __attribute__((ext_vector_type(4)));

// One row in a wavefront's registers.
template <int VEC, int NC>
struct Row {
  float v[NC][VEC];

  __device__ __forceinline__ void load(const float* __restrict__ row, int E, int lane) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int e = VEC * (64 * c + lane);
      if constexpr (VEC == 4) {   // E is a multiple of 4
        const rf4 q = e < E ? __builtin_nontemporal_load(reinterpret_cast<const rf4*>(row + e))
                            : rf4{kNegInf, kNegInf, kNegInf, kNegInf};
        v[c][0] = q.x, v[c][1] = q.y, v[c][2] = q.z, v[c][3] = q.w;
      } else {
        v[c][0] = e < E ? row[e] : kNegInf;
      }
    }
  }

  // v becomes exp(v - max), returns their sum; lse = log of the sum of exp(v).
  // NaN as -inf; equal values, infinities too, differ by 0; absent experts 0.
  // The exponential is 2^((v - max) log2(e)).  The difference, its product and the
  // constant are rounded: a relative error of 2.2 |v - max| 2^-24, of which the
  // difference's 1.0 is there whatever follows, in terms that are e^(v - max)
  // small (of a probability never more than 2^-24); a product in two parts would
  // leave 1.0 and cost four instructions more per logit.
  __device__ __forceinline__ float exps(int E, int lane, float& lse) {
    float m = kNegInf;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        v[c][j] = fmaxf(v[c][j], kNegInf);   // the number of the two: NaN becomes -inf
        m = fmaxf(m, v[c][j]);
      }
    m = wave_max(m);
    float sum = 0.0f;
    if (finite(m)) {   // absent experts hold -inf, whose exponential is 0
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          v[c][j] = __builtin_amdgcn_exp2f((v[c][j] - m) * 1.44269504f);
          sum += v[c][j];
        }
    } else {           // only the logits equal to the infinite maximum count
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          v[c][j] = v[c][j] == m && VEC * (64 * c + lane) < E ? 1.0f : 0.0f;
          sum += v[c][j];
        }
    }
    sum = wave_sum(sum);
    lse = m + logf(sum);
    return sum;
  }
};

// The losses of a sequence from its sums.
__device__ __forceinline__ void write_losses(const BalanceArgs& a, int s, int n, double cp, double zs) {
  const double dn = n;
  a.balance[s] = n > 0 ? static_cast<float>(cp * a.E / (dn * dn * a.k)) : 0.0f;
  a.z[s] = n > 0 ? static_cast<float>(zs / dn) : 0.0f;
  a.n_tokens[s] = n;
}

// SINGLE: one workgroup does everything.  FOLD: a wavefront may have more than
// RB_FOLD rows.
template <int VEC, int NC, bool SINGLE, bool FOLD>
__global__ __launch_bounds__(RB_THREADS) void balance_rows_kernel(BalanceArgs a) {
  extern __shared__ float lds[];
  float* s_p = lds;                                                 // [RB_HALF][E]
  int32_t* s_c = reinterpret_cast<int32_t*>(lds + RB_HALF * a.E);   // [E]
  __shared__ double s_z[RB_WAVES];
  __shared__ int s_n[RB_WAVES];
  __shared__ double s_l[RB_WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int E = a.E, chunk = blockIdx.x;
  if (!SINGLE)   // the second launch's tickets
    for (int s = chunk * RB_THREADS + tid; s < a.S; s += a.n_chunks * RB_THREADS) a.done[s] = 0;
  const int t0 = chunk * a.chunk_rows, t1 = min(a.T, t0 + a.chunk_rows);
  // first sequence that can hold a row of the chunk
  int s = SINGLE ? 0 : max(seq_of_row(a.seq, a.S, a.T, t0), 0);
  for (; s < a.S; ++s) {
    const int b0 = max(seq_bound(a.seq, s, a.S, a.T), t0);
    const int b1 = min(seq_bound(a.seq, s + 1, a.S, a.T), t1);
    if (!SINGLE) {
      if (b0 >= t1) break;
      if (b0 >= b1) continue;
    }
    for (int e = tid; e < E; e += RB_THREADS) s_c[e] = 0;
    // Probabilities in fp32: RB_FOLD rows at a time, whose sums join a total, so
    // that a sum's error does not grow with the rows (16.8 million equal rows of
    // 37 experts: 936 units of 2^-24 without, 9 with).  Squares of lse in 64 bits: one a row,
    // and the sum of those whose mean is finite may not be.
    float acc[NC][VEC] = {}, total[NC][VEC] = {};
    double zs = 0.0;
    int n = 0;
    // the next row is on its way while one is worked on
    Row<VEC, NC> r, ahead;
    bool part = false;
    if (b0 + wave < b1) {
      ahead.load(a.logits + static_cast<int64_t>(b0 + wave) * E, E, lane);
      part = !a.mask || a.mask[b0 + wave] != 0;
    }
    __syncthreads();   // the histogram is clear
    const int64_t p0 = static_cast<int64_t>(b0) * a.k;
    const int np = max(b1 - b0, 0) * a.k;
    for (int p = tid; p < np; p += RB_THREADS) {
      if (a.mask && !a.mask[b0 + p / a.k]) continue;
      const int e = a.idx[p0 + p];
      if (e >= 0 && e < E) atomicAdd(&s_c[e], 1);
    }
    for (int t = b0 + wave; t < b1; t += RB_WAVES) {
      r = ahead;
      const bool now = part;
      if (t + RB_WAVES < b1) {
        ahead.load(a.logits + static_cast<int64_t>(t + RB_WAVES) * E, E, lane);
        part = !a.mask || a.mask[t + RB_WAVES] != 0;
      }
      if (!now) continue;
      float lse;
      const float inv = 1.0f / r.exps(E, lane, lse);
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[c][j] = fmaf(r.v[c][j], inv, acc[c][j]);
      zs += finite(lse) ? static_cast<double>(lse) * lse : 0.0;
      ++n;
      if constexpr (FOLD) {
        if (n % RB_FOLD == 0) {
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < VEC; ++j) total[c][j] += acc[c][j], acc[c][j] = 0.0f;
        }
      }
    }
    if constexpr (FOLD) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[c][j] += total[c][j];
    }
    // wavefronts 8..15 hand their sums to 0..7, whose sums then meet below
    // (half the LDS of all sixteen at once: two workgroups fit a CU)
#pragma unroll
    for (int h = 1; h >= 0; --h) {
      if ((wave >= RB_HALF) == (h == 1)) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const int e = VEC * (64 * c + lane) + j;
            float* at = s_p + (wave % RB_HALF) * E + e;
            if (e < E) *at = h == 1 ? acc[c][j] : acc[c][j] + *at;
          }
      }
      if (h == 1) __syncthreads();
    }
    if (lane == 0) {
      s_z[wave] = zs;
      s_n[wave] = n;
    }
    __syncthreads();
    double cp = 0.0;
    const int64_t at = SINGLE ? static_cast<int64_t>(s) * E : static_cast<int64_t>(chunk + s) * E;
    for (int e = tid; e < E; e += RB_THREADS) {
      float p = 0.0f;
#pragma unroll
      for (int w = 0; w < RB_HALF; ++w) p += s_p[w * E + e];
      const int c = s_c[e];
      (SINGLE ? a.prob_sum : a.p_part)[at + e] = p;
      (SINGLE ? a.counts : a.c_part)[at + e] = c;
      cp += static_cast<double>(c) * p;
    }
    if (SINGLE) {
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) cp += __shfl_xor(cp, off, 64);
      if (lane == 0) s_l[wave] = cp;
      __syncthreads();
    }
    if (tid == 0) {
      double zz = 0.0;
      int nn = 0;
      for (int w = 0; w < RB_WAVES; ++w) {
        zz += s_z[w];
        nn += s_n[w];
      }
      if (SINGLE) {
        double l = 0.0;
        for (int w = 0; w < RB_WAVES; ++w) l += s_l[w];
        write_losses(a, s, nn, l, zz);
      } else {
        a.z_part[chunk + s] = zz;
        a.n_part[chunk + s] = nn;
      }
    }
    __syncthreads();   // s_p, s_c and the rest are free again
  }
}

__global__ __launch_bounds__(RB_ETILE * RB_SUBS) void balance_reduce_kernel(BalanceArgs a) {
  __shared__ float s_p[RB_SUBS][RB_ETILE];
  __shared__ int32_t s_c[RB_SUBS][RB_ETILE];
  __shared__ double s_l[RB_ETILE / 64];
  const int tile = static_cast<int>(blockIdx.x) % a.n_etiles, s = static_cast<int>(blockIdx.x) / a.n_etiles;
  const int tid = threadIdx.x, el = tid % RB_ETILE, sub = tid / RB_ETILE;
  const int e = tile * RB_ETILE + el;
  const int b0 = seq_bound(a.seq, s, a.S, a.T), b1 = seq_bound(a.seq, s + 1, a.S, a.T);
  const int c0 = b0 / a.chunk_rows, c1 = b1 > b0 ? (b1 - 1) / a.chunk_rows + 1 : c0;
  // the sequence's z and row count (lanes over its chunks), in the first
  // wavefront of every workgroup: whichever needs them has them at hand
  double zs = 0.0;
  int n = 0;
  if (tid < 64) {
    for (int q = c0 + tid; q < c1; q += 64) {
      zs += a.z_part[q + s];
      n += a.n_part[q + s];
    }
  }
  float p = 0.0f;
  int32_t c = 0;
  if (e < a.E) {
#pragma unroll 8
    for (int q = c0 + sub; q < c1; q += RB_SUBS) {
      const int64_t at = static_cast<int64_t>(q + s) * a.E + e;
      p += a.p_part[at];
      c += a.c_part[at];
    }
  }
  s_p[sub][el] = p;
  s_c[sub][el] = c;
  __syncthreads();
  if (sub == 0) {   // whole wavefronts
    for (int i = 1; i < RB_SUBS; ++i) {
      p += s_p[i][el];
      c += s_c[i][el];
    }
    double cp = 0.0;
    if (e < a.E) {
      const int64_t at = static_cast<int64_t>(s) * a.E + e;
      a.prob_sum[at] = p;
      a.counts[at] = c;
      cp = static_cast<double>(c) * p;
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) cp += __shfl_xor(cp, off, 64);
    if (tid % 64 == 0) s_l[tid / 64] = cp;
  }
  __syncthreads();
  if (tid >= 64) return;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    zs += __shfl_xor(zs, off, 64);
    n += __shfl_xor(n, off, 64);
  }
  double l = 0.0;
  for (int i = 0; i < RB_ETILE / 64; ++i) l += s_l[i];
  if (a.n_etiles > 1) {
    double* part = a.l_part + static_cast<int64_t>(s) * a.n_etiles;
    uint32_t before = 0;
    if (tid == 0) {
      __hip_atomic_store(&part[tile], l, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      before = __hip_atomic_fetch_add(&a.done[s], 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (__builtin_amdgcn_readfirstlane(before) + 1 != static_cast<uint32_t>(a.n_etiles)) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    l = tid < a.n_etiles ? __hip_atomic_load(&part[tid], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) l += __shfl_xor(l, off, 64);
  }
  if (tid == 0) write_losses(a, s, n, l, zs);
}

// ---------------------------------------------------------------------------

constexpr int RW_WAVES = 4;
constexpr int RW_THREADS = RW_WAVES * 64;

struct BackwardArgs {
  const float* logits;
  const int32_t* idx;
  const int32_t* seq;
  const uint8_t* mask;
  const int32_t* counts;
  const int32_t* n_tokens;
  const float* g_balance;
  const float* g_z;
  const float* w;
  const float* dw;
  float* dlogits;
  int T, E, k, S, rows;   // rows: consecutive rows per wavefront
};

struct Pair {   // lane i: pair i of a row
  int e;
  float w, dw;
};

template <int VEC, int NC>
__global__ __launch_bounds__(RW_THREADS) void balance_backward_kernel(BackwardArgs a) {
  extern __shared__ float lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int E = a.E;
  // this wavefront's scratch: the row's routing terms and who owns each
  float* s_v = lds + wave * 2 * E;
  int32_t* s_o = reinterpret_cast<int32_t*>(s_v + E);
  const bool routed = a.w != nullptr;
  for (int e = lane; e < E; e += 64) s_v[e] = 0.0f;
  wave_lds_sync();
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * RW_WAVES + wave) * a.rows;
  if (first >= a.T) return;
  const int t0 = static_cast<int>(first), t1 = min(a.T, t0 + a.rows);
  int s = seq_of_row(a.seq, a.S, a.T, t0);
  int s_end = s < 0 ? seq_bound(a.seq, 0, a.S, a.T) : s < a.S ? seq_bound(a.seq, s + 1, a.S, a.T) : a.T;
  float cc[NC][VEC] = {};   // counts of the sequence less their mean
  float kb = 0.0f, kz = 0.0f;
  int loaded = -2;
  // the next row and its pairs are on their way while one is worked on
  Row<VEC, NC> ahead;
  Pair next = {};
  bool part_next = false;
  const bool reads = a.g_balance || a.g_z;
  const auto request = [&](int t) {
    part_next = !a.mask || a.mask[t] != 0;
    if (reads) ahead.load(a.logits + static_cast<int64_t>(t) * E, E, lane);
    if (routed && lane < a.k) {
      const int64_t at = static_cast<int64_t>(t) * a.k + lane;
      next = Pair{a.idx[at], a.w[at], a.dw[at]};
    }
  };
  request(t0);
  for (int t = t0; t < t1; ++t) {
    while (t >= s_end && s < a.S) {
      ++s;
      s_end = s < a.S ? seq_bound(a.seq, s + 1, a.S, a.T) : a.T;
    }
    Row<VEC, NC> r = ahead;
    const Pair pair = next;
    const bool part = s >= 0 && s < a.S && part_next;
    if (t + 1 < t1) request(t + 1);
    float* __restrict__ out = a.dlogits + static_cast<int64_t>(t) * E;
    float d[NC][VEC] = {};
    if (part) {
      if (s != loaded) {
        loaded = s;
        const int n = a.n_tokens ? a.n_tokens[s] : 0;
        const float fn = static_cast<float>(n);
        kb = a.g_balance && n > 0
                 ? static_cast<float>(static_cast<double>(a.g_balance[s]) * E / (static_cast<double>(n) * n * a.k))
                 : 0.0f;
        kz = a.g_z && n > 0 ? 2.0f * a.g_z[s] / fn : 0.0f;
        // p sums to 1, so a constant off every count changes nothing but the
        // cancellation between the two terms
        const int mean = static_cast<int>(static_cast<int64_t>(n) * a.k / E);
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const int e = VEC * (64 * c + lane) + j;
            cc[c][j] = a.g_balance && e < E ? static_cast<float>(a.counts[static_cast<int64_t>(s) * E + e] - mean) : 0.0f;
          }
      }
      if (kb != 0.0f || kz != 0.0f) {
        float lse;
        const float inv = 1.0f / r.exps(E, lane, lse);
        float dot = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int j = 0; j < VEC; ++j) dot = fmaf(cc[c][j], r.v[c][j], dot);
        dot = wave_sum(dot) * inv;
        const float lz = finite(lse) ? kz * lse : 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int j = 0; j < VEC; ++j) d[c][j] = r.v[c][j] * inv * fmaf(kb, cc[c][j] - dot, lz);
      }
      if (routed) {
        const bool mine = lane < a.k;
        const int e = mine ? pair.e : -1;
        const float dot = wave_sum(mine ? pair.w * pair.dw : 0.0f);
        float v = pair.w * (pair.dw - dot);
        const bool ok = mine && e >= 0 && e < E;
        // equal ids in the row: the lane that reads back its own number adds
        // up all of them in order
        if (ok) s_o[e] = lane;
        wave_lds_sync();
        const int owner = ok ? s_o[e] : lane;
        if (__ballot(owner != lane)) {
          float sum = 0.0f;
          for (int i = 0; i < a.k; ++i) {
            const int ei = __builtin_amdgcn_readlane(e, i);
            const float vi = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), i));
            if (ei == e) sum += vi;
          }
          v = sum;
        }
        if (ok && owner == lane) s_v[e] = v;
        wave_lds_sync();
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const int q = VEC * (64 * c + lane) + j;
            if (q < E) d[c][j] += s_v[q];
          }
        wave_lds_sync();
        if (ok) s_v[e] = 0.0f;
        wave_lds_sync();
      }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int e = VEC * (64 * c + lane);
      if (e < E) {
        if constexpr (VEC == 4)
          __builtin_nontemporal_store(rf4{d[c][0], d[c][1], d[c][2], d[c][3]}, reinterpret_cast<rf4*>(out + e));
        else
          out[e] = d[c][0];
      }
    }
  }
}

// One launch and no workspace for few rows: a call takes 16 us instead of 20.5,
// which the host bounds.  Not for more: 256 rows of 64 experts in 8 sequences would
// keep the one workgroup busy for 29 us (two launches: 7.9).
bool balance_single(int T, int S) { return T <= RB_SINGLE_ROWS && S <= RB_SINGLE_SEQS; }

struct BalanceSpace {
  int chunk_rows, n_chunks, n_etiles;
  int64_t p, c, z, n, l, done, total;
};

BalanceSpace balance_space(int T, int E, int S) {
  BalanceSpace b;
  b.chunk_rows = balance_chunk_rows(T > 0 ? T : 1);
  b.n_chunks = (T + b.chunk_rows - 1) / b.chunk_rows;
  if (b.n_chunks < 1) b.n_chunks = 1;
  b.n_etiles = (E + RB_ETILE - 1) / RB_ETILE;
  const int64_t np = static_cast<int64_t>(b.n_chunks) + S;
  b.p = 0;
  b.c = b.p + align256(np * E * 4);
  b.z = b.c + align256(np * E * 4);
  b.n = b.z + align256(np * 8);
  b.l = b.n + align256(np * 4);
  b.done = b.l + align256(static_cast<int64_t>(S) * b.n_etiles * 8);
  b.total = b.done + align256(static_cast<int64_t>(S) * 4);
  return b;
}

template <int VEC, int NC>
hipError_t run_forward(BalanceArgs& a, hipStream_t st) {
  const size_t lds = static_cast<size_t>(RB_HALF + 1) * a.E * 4;
  if (balance_single(a.T, a.S)) {
    a.chunk_rows = RB_SINGLE_ROWS;
    balance_rows_kernel<VEC, NC, true, false><<<1, RB_THREADS, lds, st>>>(a);
    return hipGetLastError();
  }
  if (a.chunk_rows > RB_WAVES * RB_FOLD)   // more than 262,144 rows
    balance_rows_kernel<VEC, NC, false, true><<<a.n_chunks, RB_THREADS, lds, st>>>(a);
  else
    balance_rows_kernel<VEC, NC, false, false><<<a.n_chunks, RB_THREADS, lds, st>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  balance_reduce_kernel<<<static_cast<unsigned>(a.S) * a.n_etiles, RB_ETILE * RB_SUBS, 0, st>>>(a);
  return hipGetLastError();
}

template <int VEC, int NC>
hipError_t run_backward(const BackwardArgs& a, hipStream_t st) {
  const size_t lds = static_cast<size_t>(RW_WAVES) * 2 * a.E * 4;
  const int64_t per = static_cast<int64_t>(RW_WAVES) * a.rows;
  balance_backward_kernel<VEC, NC>
      <<<static_cast<unsigned>((a.T + per - 1) / per), RW_THREADS, lds, st>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t route_balance_workspace_bytes(int T, int E, int S) {
  if (balance_single(T, S)) return 0;
  return static_cast<size_t>(balance_space(T, E, S).total);
}

hipError_t launch_route_balance(const float* logits, const int32_t* idx, int T, int E, int k,
                                const int32_t* seq, int S, const uint8_t* mask, float* balance,
                                float* z, int32_t* counts, float* prob_sum, int32_t* n_tokens,
                                void* ws, hipStream_t s) {
  const BalanceSpace b = balance_space(T, E, S);
  char* p = static_cast<char*>(ws);
  BalanceArgs a{logits, idx, seq, mask, balance, z, counts, prob_sum, n_tokens,
                reinterpret_cast<float*>(p + b.p), reinterpret_cast<int32_t*>(p + b.c),
                reinterpret_cast<double*>(p + b.z), reinterpret_cast<int32_t*>(p + b.n),
                reinterpret_cast<double*>(p + b.l), reinterpret_cast<uint32_t*>(p + b.done),
                T, E, k, S, b.chunk_rows, b.n_chunks, b.n_etiles};
  if (E % 4 == 0) {
    if (E <= 256) return run_forward<4, 1>(a, s);
    if (E <= 512) return run_forward<4, 2>(a, s);
    return run_forward<4, 4>(a, s);
  }
  if (E <= 64) return run_forward<1, 1>(a, s);
  if (E <= 256) return run_forward<1, 4>(a, s);
  return run_forward<1, 16>(a, s);
}

hipError_t launch_route_backward(const float* logits, const int32_t* idx, int T, int E, int k,
                                 const int32_t* seq, int S, const uint8_t* mask,
                                 const int32_t* counts, const int32_t* n_tokens,
                                 const float* g_balance, const float* g_z, const float* w,
                                 const float* dw, float* dlogits, hipStream_t s) {
  // runs of rows only where there are many more rows than wavefronts fit
  const int rows = T >= 65536 ? 8 : T >= 16384 ? 4 : 1;
  const BackwardArgs a{logits, idx, seq, mask, counts, n_tokens, g_balance, g_z, w, dw, dlogits,
                       T, E, k, S, rows};
  if (E % 4 == 0) {
    if (E <= 256) return run_backward<4, 1>(a, s);
    if (E <= 512) return run_backward<4, 2>(a, s);
    return run_backward<4, 4>(a, s);
  }
  if (E <= 64) return run_backward<1, 1>(a, s);
  if (E <= 256) return run_backward<1, 4>(a, s);
  return run_backward<1, 16>(a, s);
}

}  // namespace bitffn
