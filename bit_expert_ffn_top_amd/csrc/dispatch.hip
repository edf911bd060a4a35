// Tokens to the experts and back: the pairs' rows in group order, the weighted
// sum of them in the tokens' order, and the gradients of both:
//   rows[pos] = x[t]          dx[t] = sum_i drows[pos]
//   y[t] = base[t] + sum_i w rows[pos]
//   drows[pos] = w dy[t]      dw = <dy[t], rows[pos]>
// Nothing is computed to speak of; HBM bounds all of it where there are many
// tokens, launches and dependent loads where there are few.  A chunk of 8,192
// tokens x 10 pairs of 2,048 bfloat16 columns (335 MB of rows): dispatch 4.8 us for
// the counts + 72 us (5.0 TB/s), its gradient and the combine 62 and 64 us (5.9 and
// 6.2 TB/s), the combine's gradients 143 us (4.9 TB/s).  Rows are streamed past the
// caches in both directions: they are more than these hold (plain stores and loads:
// dispatch 94 us, combine 84 us).
#include <algorithm>

#include "moe_internal.h"
#include "row_device.h"
#include "scan_device.h"

namespace bitffn {
namespace {

constexpr int kMaxE = MOE_MAX_EXPERTS;
constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxOwn = 1024;   // pairs of one workgroup's tokens (16 of MOE_MAX_TOPK)
// Many pairs are counted in parts: fewer are less to add up for each workgroup,
// more are less to count again before its own tokens (81,920 pairs in parts of
// 640: 84 us, 1,280: 80.2, 2,560: 79.7, 5,120: 81.7, 10,240: 87.8).
constexpr int kPartPairs = 2560;
constexpr int kMaxParts = 128;

struct DispatchArgs {
  const void* x;
  const int32_t* idx;
  void* rows;
  int32_t* offsets;
  int32_t* pair_pos;
  uint16_t* counts;   // [parts][counts_row(E)]: pairs of each expert in a part
  int T, k, E;
  int nv;             // vectors of a row
  int tokens;         // of a workgroup
  int parts;
  int part_tokens;    // of a part, and its workgroups
  int subs;
};

__host__ __device__ inline int counts_row(int E) { return (E + 7) & ~7; }

__device__ __forceinline__ bool is_expert(int e, int E) { return e >= 0 && e < E; }

// The ids of pairs p0 + thread, + 256, .. below p1: eight loads at a time, so that
// a workgroup waits for memory once for 2,048 of them.  -1 for ids of no expert.
template <typename F>
__device__ __forceinline__ void each_id(const int32_t* __restrict__ idx, int p0, int p1, int E, F f) {
  constexpr int kBatch = 8;
  for (int p = p0 + static_cast<int>(threadIdx.x); p < p1; p += kBatch * kThreads) {
    int e[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) e[i] = idx[min(p + i * kThreads, p1 - 1)];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (p + i * kThreads < p1) f(p + i * kThreads, is_expert(e[i], E) ? e[i] : -1);
  }
}

// Pairs of every expert in one part of the tokens.
__global__ __launch_bounds__(kThreads) void dispatch_count_kernel(DispatchArgs a) {
  __shared__ int32_t s_count[kMaxE];
  const int row = counts_row(a.E);
  for (int e = threadIdx.x; e < row; e += kThreads) s_count[e] = 0;
  __syncthreads();
  const int t0 = min(a.T, static_cast<int>(blockIdx.x) * a.part_tokens);
  const int t1 = min(a.T, t0 + a.part_tokens);
  each_id(a.idx, t0 * a.k, t1 * a.k, a.E, [&](int, int e) {
    if (e >= 0) atomicAdd(&s_count[e], 1);
  });
  __syncthreads();
  for (int e = threadIdx.x; e < row; e += kThreads)
    a.counts[static_cast<int>(blockIdx.x) * row + e] = static_cast<uint16_t>(s_count[e]);
}

// The row of a pair = pairs of smaller experts + earlier pairs of its expert.
// Every workgroup finds both for its own tokens, so no launch waits for a sort.
// Few pairs: it counts all of them in LDS.  Many (COUNTED): it adds up the parts
// that an earlier launch counted, and counts what its own part holds before its
// tokens.  Ranks among its own pairs are counted directly, which keeps equal ids
// of a token in order.  Then it reads its tokens' rows once and writes each to
// its k places.  64 tokens x 10 pairs: 5.4 us, most of it the chain of counting,
// scanning and ranking.
template <typename V, bool COUNTED>   // V: the part of a row that one lane moves
__global__ __launch_bounds__(kThreads) void dispatch_kernel(DispatchArgs a) {
  __shared__ int32_t s_total[kMaxE];
  __shared__ int32_t s_before[kMaxE];   // then each expert's row for the next own pair
  __shared__ int32_t s_wave[kWaves];
  __shared__ __align__(16) int32_t s_own[kMaxOwn];
  __shared__ int32_t s_pos[kMaxOwn];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int E = a.E, k = a.k;
  int t0, t1, part = 0;
  if (COUNTED) {
    part = blockIdx.x / a.subs;
    const int sub = blockIdx.x - part * a.subs;
    t0 = min(a.T, part * a.part_tokens + sub * a.tokens);
    t1 = min(min(a.T, t0 + a.tokens), (part + 1) * a.part_tokens);
  } else {
    t0 = blockIdx.x * a.tokens;
    t1 = min(a.T, t0 + a.tokens);
  }
  const int p0 = t0 * k, own = (t1 - t0) * k;
  for (int e = tid; e < kMaxE; e += kThreads) s_total[e] = s_before[e] = 0;
  for (int q = own + tid; q < (own + 3) / 4 * 4; q += kThreads) s_own[q] = -1;
  each_id(a.idx, p0, p0 + own, E, [&](int p, int e) { s_own[p - p0] = e; });
  __syncthreads();
  if (COUNTED) {
    // eight experts' counts per load, the parts dealt to groups of threads
    const int vecs = counts_row(E) / 8, groups = kThreads / vecs;
    const int g = tid / vecs, j = tid - g * vecs;
    if (g < groups) {
      int total[8], before[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) total[i] = before[i] = 0;
      const uint4* src = reinterpret_cast<const uint4*>(a.counts) + j;
      constexpr int kBatch = 8;
      for (int c = g; c < a.parts; c += kBatch * groups) {
        uint4 v[kBatch];
#pragma unroll
        for (int n = 0; n < kBatch; ++n) v[n] = src[min(c + n * groups, a.parts - 1) * vecs];
#pragma unroll
        for (int n = 0; n < kBatch; ++n) {
          const int at = c + n * groups;
          const uint32_t w[4] = {v[n].x, v[n].y, v[n].z, v[n].w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int m = i % 2 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu;
            total[i] += at < a.parts ? m : 0;
            before[i] += at < part ? m : 0;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (total[i]) atomicAdd(&s_total[8 * j + i], total[i]);
        if (before[i]) atomicAdd(&s_before[8 * j + i], before[i]);
      }
    }
    each_id(a.idx, part * a.part_tokens * k, p0, E, [&](int, int e) {
      if (e >= 0) atomicAdd(&s_before[e], 1);
    });
  } else {
    each_id(a.idx, 0, a.T * k, E, [&](int p, int e) {
      if (e >= 0) {
        atomicAdd(&s_total[e], 1);
        if (p < p0) atomicAdd(&s_before[e], 1);
      }
    });
  }
  __syncthreads();
  // the experts' first rows: an exclusive scan, four experts per thread
  constexpr int kPer = kMaxE / kThreads;
  int c[kPer], sum = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    c[j] = sum;
    sum += s_total[tid * kPer + j];
  }
  const int scan = wave_scan_add(sum);
  if (lane == 63) s_wave[wave] = scan;
  __syncthreads();
  int first = scan - sum;
  for (int w = 0; w < wave; ++w) first += s_wave[w];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = tid * kPer + j;
    s_before[e] += first + c[j];
    if (blockIdx.x == 0 && e < E) a.offsets[e] = first + c[j];
  }
  if (blockIdx.x == 0 && tid == kThreads - 1) a.offsets[E] = first + sum;
  __syncthreads();
  for (int q = tid; q < own; q += kThreads) {
    const int e = s_own[q];
    int at = -1;
    if (e >= 0) {
      at = s_before[e];
#pragma unroll 4
      for (int r = 0; r < q; r += 4) {   // four at a time; those past q do not count
        const int4 o = *reinterpret_cast<const int4*>(&s_own[r]);
        at += (o.x == e) + (r + 1 < q && o.y == e) + (r + 2 < q && o.z == e) + (r + 3 < q && o.w == e);
      }
    }
    s_pos[q] = at;
    a.pair_pos[p0 + q] = at;
  }
  __syncthreads();
  const V* x = static_cast<const V*>(a.x) + static_cast<int64_t>(t0) * a.nv;
  V* rows = static_cast<V*>(a.rows);
  const int items = (t1 - t0) * a.nv;
  for (int i = tid; i < items; i += kThreads) {
    const V v = x[i];
    const int t = i / a.nv, j = i - t * a.nv;
    for (int q = t * k; q < t * k + k; ++q) {
      const int at = s_pos[q];
      if (at >= 0) __builtin_nontemporal_store(v, &rows[static_cast<int64_t>(at) * a.nv + j]);
    }
  }
}

__device__ __forceinline__ bool has_row(int p, int R) { return p >= 0 && p < R; }

// One thread per N consecutive columns of one token (the last one of a row may
// have half of them), the k terms in i order.
template <typename RT, typename YT, int N>
__global__ __launch_bounds__(kThreads) void combine_rows_kernel(
    const RT* __restrict__ rows, int R, int T, int d, int k, const int32_t* __restrict__ pair_pos,
    const float* __restrict__ w, const void* base, int base_dtype, YT* y) {
  const int dn = (d + N - 1) / N;
  const int64_t gid = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (gid >= static_cast<int64_t>(T) * dn) return;
  const int t = static_cast<int>(gid / dn);
  const int c = static_cast<int>(gid - static_cast<int64_t>(t) * dn) * N;
  const int64_t at = static_cast<int64_t>(t) * d + c;
  const bool half = c + N > d;
  float acc[N];
#pragma unroll
  for (int j = 0; j < N; ++j) acc[j] = 0.0f;
  if (base && base_dtype == MOE_DTYPE_F32) {
    RowPart<float, N> b;
    b.load(static_cast<const float*>(base) + at, half);
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = b.get(j);
  } else if (base) {
    RowPart<uint16_t, N> b;
    b.load(static_cast<const uint16_t*>(base) + at, half);
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = b.get(j);
  }
  // the terms in batches: all places of a batch, then all its rows (one that is
  // missing re-reads one that is there, so that no load waits for a comparison).  More
  // terms at a time are more registers, which cost where there are few terms; few at a
  // time are waits (2048 bfloat16 columns, batches of 4, 8, 10 and 16 terms: 8,192
  // tokens x 2 23, 23, 24 and 31 us, x 10 65, 65, 64 and 64, x 24 142, 142, 141 and 139;
  // 64 tokens x 2 2.9, 3.1, 3.2 and 3.7, x 10 5.4, 5.2, 4.2 and 4.8)
  constexpr int KC = 10;
  const int64_t q0 = static_cast<int64_t>(t) * k;
  for (int i0 = 0; i0 < k; i0 += KC) {
    int p[KC];
    float wi[KC];
    RowPart<RT, N> r[KC];
    int any = -1;
#pragma unroll
    for (int j = 0; j < KC; ++j) {
      const int64_t q = q0 + min(i0 + j, k - 1);
      p[j] = i0 + j < k ? pair_pos[q] : -1;
      wi[j] = w ? w[q] : 1.0f;
    }
#pragma unroll
    for (int j = KC - 1; j >= 0; --j) any = has_row(p[j], R) ? p[j] : any;
    if (any < 0) continue;
#pragma unroll
    for (int j = 0; j < KC; ++j)
      if (i0 + j < k)   // uniform
        r[j].template load<true>(rows + static_cast<int64_t>(has_row(p[j], R) ? p[j] : any) * d + c, half);
#pragma unroll
    for (int j = 0; j < KC; ++j) {
      if (!has_row(p[j], R)) continue;
#pragma unroll
      for (int n = 0; n < N; ++n) acc[n] = fmaf(wi[j], r[j].get(n), acc[n]);
    }
  }
  RowPart<YT, N> out;
  out.set(acc);
  out.template store<true>(y + at, half);
}

constexpr int kBackWaves = 16;

// One workgroup per token, one wavefront per pair at a time: the product with
// dy for dw, and dy times the weight for drows.  NC > 0: a row has at most NC
// parts per lane, and dy's stay in registers; 0: rows of any length.
template <typename GT, typename RT, int N, int NC>
__global__ __launch_bounds__(64 * kBackWaves) void combine_backward_kernel(
    const GT* __restrict__ dy, const RT* __restrict__ rows, int R, int d, int k,
    const int32_t* __restrict__ pair_pos, const float* __restrict__ w, RT* __restrict__ drows,
    float* __restrict__ dw) {
  constexpr int H = NC > 0 ? NC : 1;
  const int lane = threadIdx.x & 63;
  const int64_t t = blockIdx.x;
  const int c0 = lane * N;
  RowPart<GT, N> g[H];
  if (NC > 0) {
#pragma unroll
    for (int j = 0; j < H; ++j)
      if (c0 + 64 * N * j < d) g[j].load(dy + t * d + c0 + 64 * N * j, c0 + 64 * N * j + N > d);
  }
  for (int i = threadIdx.x >> 6; i < k; i += blockDim.x >> 6) {
    const int64_t q = t * k + i;
    const int p = pair_pos[q];
    float sum = 0.0f;
    if (has_row(p, R)) {
      const float wi = w ? w[q] : 1.0f;
      const int64_t row = static_cast<int64_t>(p) * d;
      for (int b = c0; b < d; b += 64 * N * H) {
        RowPart<RT, N> r[H];
        if (dw) {
#pragma unroll
          for (int j = 0; j < H; ++j)
            if (b + 64 * N * j < d) r[j].load(rows + row + b + 64 * N * j, b + 64 * N * j + N > d);
        }
#pragma unroll
        for (int j = 0; j < H; ++j) {
          const int c = b + 64 * N * j;
          if (c >= d) break;
          if (NC == 0) g[j].load(dy + t * d + c, c + N > d);
          if (drows) {
            float f[N];
#pragma unroll
            for (int n = 0; n < N; ++n) f[n] = wi * g[j].get(n);
            RowPart<RT, N> out;
            out.set(f);
            out.template store<true>(drows + row + c, c + N > d);
          }
          if (dw) {
#pragma unroll
            for (int n = 0; n < N; ++n) sum = fmaf(g[j].get(n), r[j].get(n), sum);
          }
        }
      }
    }
    if (dw) {
      sum = row16_sum_dpp(sum);
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (lane == 0) dw[q] = sum;
    }
  }
}

// A lane's part of a row: 16 bytes of the narrower type.
template <typename A, typename B>
constexpr int part_of() {
  return sizeof(A) == 4 && sizeof(B) == 4 ? 4 : 8;
}

template <typename RT, typename YT>
hipError_t combine_rows_as(const void* rows, int64_t R, int T, int d, int k,
                           const int32_t* pair_pos, const float* w, const void* base,
                           int base_dtype, void* y, hipStream_t s) {
  constexpr int N = part_of<RT, YT>();
  const int per = (d + N - 1) / N;
  // a launch has fewer than 2^32 threads (std::min: min alone may be that of 32 bits)
  const int most = static_cast<int>(std::min(int64_t{T}, (int64_t{1} << 31) / per));
  const int64_t base_bytes = static_cast<int64_t>(d) * (base_dtype == MOE_DTYPE_F32 ? 4 : 2);
  for (int t = 0; t < T; t += most) {
    const int n = min(most, T - t);
    const int64_t blocks = (static_cast<int64_t>(n) * per + kThreads - 1) / kThreads;
    combine_rows_kernel<RT, YT, N><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(
        static_cast<const RT*>(rows), static_cast<int>(R), n, d, k, pair_pos + int64_t{t} * k,
        w ? w + int64_t{t} * k : nullptr, base ? static_cast<const char*>(base) + t * base_bytes : nullptr,
        base_dtype, static_cast<YT*>(y) + int64_t{t} * d);
  }
  return hipGetLastError();
}

template <typename GT, typename RT>
hipError_t combine_backward_as(const void* dy, const void* rows, int64_t R, int T, int d, int k,
                               const int32_t* pair_pos, const float* w, void* drows, float* dw,
                               hipStream_t s) {
  // few tokens: a wavefront for every pair; many: four per token, which share dy
  // (64 tokens x 10 pairs 4.1 against 6.4 us, 400 9.2 against 9.4, 8,192 163 against 143)
  const int waves = T <= 512 ? min(k, kBackWaves) : min(k, 4);
  const auto go = [&](auto kernel) {
    kernel<<<T, 64 * waves, 0, s>>>(static_cast<const GT*>(dy), static_cast<const RT*>(rows),
                                  static_cast<int>(R), d, k, pair_pos, w, static_cast<RT*>(drows),
                                  dw);
  };
  // A lane keeps up to 32 values of dy, eight parts of four or four of eight: twice as
  // many spill, with 128 registers for each of 1,024 threads (4,096 tokens x 8, 4096
  // bfloat16 columns: 170 us with 64 values, 124 with none; kept against not, 2048
  // columns: bfloat16 61 against 69 us, fp32 114 against 123).
  constexpr int W = part_of<GT, RT>();
  constexpr bool kEight = W == 4;
  if (d <= 64 * W)
    go(combine_backward_kernel<GT, RT, W, 1>);
  else if (d <= 256 * W)
    go(combine_backward_kernel<GT, RT, W, 4>);
  else if (kEight && d <= 512 * W)
    go(combine_backward_kernel<GT, RT, W, kEight ? 8 : 4>);
  else
    go(combine_backward_kernel<GT, RT, W, 0>);
  return hipGetLastError();
}

}  // namespace

namespace {

// Pairs up to which every workgroup counts all of them (512 bfloat16 columns, one
// launch against two: 4,000 pairs 7.6 against 11.6 us, 8,000 9.8 against 12.0,
// 16,000 15.6 against 12.7).
constexpr int kFewPairs = 8192;

// Parts of at most 32,768 pairs (T <= 65536), so that counts have 16 bits.
int count_parts(int T, int k) {
  return max(1, min(kMaxParts, (T * k + kPartPairs - 1) / kPartPairs));
}

template <typename V>
void dispatch_as(DispatchArgs a, hipStream_t s) {
  if (!a.counts) {
    a.tokens = max(1, min((a.T + 511) / 512, kMaxOwn / a.k));
    dispatch_kernel<V, false><<<max(1, (a.T + a.tokens - 1) / a.tokens), kThreads, 0, s>>>(a);
    return;
  }
  a.parts = count_parts(a.T, a.k);
  a.part_tokens = (a.T + a.parts - 1) / a.parts;
  a.tokens = min(16, (a.T + 1023) / 1024);   // 1,024 workgroups, four per CU, until tokens are many
  a.subs = (a.part_tokens + a.tokens - 1) / a.tokens;
  dispatch_count_kernel<<<a.parts, kThreads, 0, s>>>(a);
  dispatch_kernel<V, true><<<a.parts * a.subs, kThreads, 0, s>>>(a);
}

}  // namespace

size_t dispatch_workspace_bytes(int T, int k, int E) {
  if (T * k <= kFewPairs) return 0;
  return static_cast<size_t>(align256(int64_t{count_parts(T, k)} * counts_row(E) * 2));
}

hipError_t launch_dispatch(const void* x, int dtype, int T, int d, const int32_t* idx, int k, int E,
                           void* rows, int32_t* offsets, int32_t* pair_pos, void* ws,
                           hipStream_t s) {
  const int bytes = d * (dtype == MOE_DTYPE_F32 ? 4 : 2);
  DispatchArgs a{x, idx, rows, offsets, pair_pos, nullptr, T, k, E, 0, 0, 0, 0, 0};
  if (dispatch_workspace_bytes(T, k, E) > 0) a.counts = static_cast<uint16_t*>(ws);
  if (bytes % 16 == 0) {
    a.nv = bytes / 16;
    dispatch_as<nu4>(a, s);
  } else {
    a.nv = bytes / 8;
    dispatch_as<nu2>(a, s);
  }
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
