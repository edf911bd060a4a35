// Products of microscaled 4-bit operands (moe_mxfp4_linear, moe_mxfp4_gate_up):
// y[r][n] = sum_j A[src(r)][j] W_g[n][j], on v_mfma_scale_f32_16x16x128_f8f6f4
// with both operands in the 4-bit format.
//
// Of the 128 columns that one instruction takes, lane l holds the 32 of column
// group l / 16 for row l % 16: one block of the format, 16 bytes of codes and
// one scale byte, so a wavefront's operand is 16 rows of 64 bytes as they lie
// in memory and the scales need no arithmetic.  Weights are the first operand:
// element i of lane l is then output column 4 (l / 16) + i of its 16 for token
// l % 16, four consecutive columns of one token, and a gate and its up value
// sit in neighbouring registers.
//
// Columns are summed in whatever order suits the loads, the same for every
// row: in a chunk of 256 columns lane group q takes blocks 2q and 2q + 1, so
// two instructions use 32 contiguous bytes of each lane and whole 128-byte
// lines.
#include "moe_internal.h"
#include "mx_device.h"

namespace bitffn {
namespace {

typedef int mi4 __attribute__((ext_vector_type(4)));
typedef int mi8 __attribute__((ext_vector_type(8)));
typedef float mf4 __attribute__((ext_vector_type(4)));

constexpr int ML_THREADS = 256;   // four wavefronts
constexpr uint32_t kOne = 127;    // scale byte of 2^0

struct LinearArgs {
  const uint8_t* ac;       // A codes, scales
  const uint8_t* as;
  const uint8_t* wc;       // W codes, scales
  const uint8_t* ws;
  const int32_t* offsets;  // [G+1] or null
  const int32_t* row_src;  // [R] or null
  void* y;
  int64_t R, a_rows;
  int G, N, K, src_div;
};

// What a wavefront works on: rows r0 .. r0 + rows - 1 of group g.
struct RowTile {
  int g;
  int rows;
  int64_t r0;
};

// Tile number `tile` of the row tiles of all groups in order (tile_m rows
// each, the last of a group shorter).  All threads of the workgroup take part;
// rows = 0 past the last tile.  Each thread counts the tiles of its own run of
// groups; the runs are scanned over the workgroup, and the thread whose run
// holds the tile says where it lies.
__device__ __forceinline__ RowTile find_row_tile(const LinearArgs& a, int tile, int tile_m) {
  if (a.offsets == nullptr) {
    const int64_t r0 = static_cast<int64_t>(tile) * tile_m;
    return RowTile{0, static_cast<int>(min(static_cast<int64_t>(tile_m), max(a.R - r0, int64_t{0}))), r0};
  }
  __shared__ int s_wave[ML_THREADS / 64];
  __shared__ int s_g, s_rows, s_r0;
  const int tid = threadIdx.x, lane = tid & 63;
  constexpr int kPer = (MOE_MAX_EXPERTS + ML_THREADS - 1) / ML_THREADS;
  const int R = static_cast<int>(a.R);
  int bound[kPer + 1], nt[kPer], mine = 0;
#pragma unroll
  for (int i = 0; i <= kPer; ++i) {
    const int v = a.offsets[min(tid * kPer + i, a.G)];
    bound[i] = min(max(v, 0), R);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    nt[i] = (max(bound[i + 1] - bound[i], 0) + tile_m - 1) / tile_m;
    mine += nt[i];
  }
  int scan = mine;   // inclusive over the wavefront
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int v = __shfl_up(scan, off, 64);
    if (lane >= off) scan += v;
  }
  if (lane == 63) s_wave[tid >> 6] = scan;
  if (tid == 0) s_rows = 0;
  __syncthreads();
  int at = scan - mine;
  for (int w = 0; w < (tid >> 6); ++w) at += s_wave[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (tile >= at && tile < at + nt[i]) {   // one thread, one i
      const int r0 = bound[i] + (tile - at) * tile_m;
      s_g = tid * kPer + i;
      s_r0 = r0;
      s_rows = min(tile_m, bound[i + 1] - r0);
    }
    at += nt[i];
  }
  __syncthreads();
  return RowTile{s_g, s_rows, s_r0};
}

// A's row for output row r, and whether it exists.
__device__ __forceinline__ int64_t source_row(const LinearArgs& a, int64_t r, bool& ok) {
  const int64_t s = a.row_src ? static_cast<int64_t>(a.row_src[r]) / a.src_div : r;
  ok = s >= 0 && s < a.a_rows && (!a.row_src || a.row_src[r] >= 0);
  return ok ? s : 0;
}

__device__ __forceinline__ mf4 mfma_fp4(mi4 w, mi4 x, mf4 c, uint32_t sw, uint32_t sx) {
  const mi8 a = {w.x, w.y, w.z, w.w, 0, 0, 0, 0};
  const mi8 b = {x.x, x.y, x.z, x.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, 0, static_cast<int>(sw), 0,
                                                          static_cast<int>(sx));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 bf2;
  const bf2 v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return __builtin_bit_cast(uint32_t, v);
}

// Output columns n .. n + 3 of row r.  Plain: four values.  GATED: columns
// (gate, up, gate, up), two values at n / 2.
template <bool GATED, bool BF16>
__device__ __forceinline__ void store_out(const LinearArgs& a, int64_t r, int n, mf4 v) {
  if constexpr (GATED) {
    const int64_t at = r * (a.N / 2) + n / 2;
    const float h0 = silu(v[0]) * v[1], h1 = silu(v[2]) * v[3];
    if constexpr (BF16)
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.y) + at) = pack_bf16(h0, h1);
    else
      *reinterpret_cast<float2*>(static_cast<float*>(a.y) + at) = make_float2(h0, h1);
  } else {
    const int64_t at = r * a.N + n;
    if constexpr (BF16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + at) =
          make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(a.y) + at) = make_float4(v[0], v[1], v[2], v[3]);
  }
}

// Few rows per group: a wavefront takes 16 weight rows and MT tiles of 16
// tokens, everything straight from memory.  SPLIT wavefronts share one
// 16-row tile, each with its share of the 256-column chunks (chunk c belongs
// to wavefront c % SPLIT), and their sums meet in LDS in wavefront order.
template <int MT, int SPLIT, bool GATED, bool BF16>
__global__ __launch_bounds__(ML_THREADS) void mx_linear_rows_kernel(LinearArgs a) {
  constexpr int WAVES = ML_THREADS / 64;
  constexpr int TILES = WAVES / SPLIT;       // 16-row weight tiles per workgroup
  const int n_wg = (a.N + 16 * TILES - 1) / (16 * TILES);
  const RowTile t = find_row_tile(a, static_cast<int>(blockIdx.x) / n_wg, 16 * MT);
  if (t.rows <= 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int n0 = (static_cast<int>(blockIdx.x) % n_wg * TILES + wave / SPLIT) * 16;
  const bool here = n0 < a.N;                // the last workgroup may have tiles to spare
  const int nb = a.K / 32;                   // blocks of a row
  const int64_t crow = a.K / 2;
  const int64_t wrow = static_cast<int64_t>(t.g) * a.N + min(n0, a.N - 16) + r;
  const uint8_t* __restrict__ wc = a.wc + wrow * crow;
  const uint8_t* __restrict__ ws = a.ws + wrow * nb;
  const uint8_t* xc[MT];
  const uint8_t* xs[MT];
  bool ok[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int local = 16 * m + r;
    const int64_t s = source_row(a, t.r0 + min(local, t.rows - 1), ok[m]);
    xc[m] = a.ac + s * crow;
    xs[m] = a.as + s * nb;
  }
  mf4 acc[MT] = {};
  const int chunks = (nb + 7) / 8;
  for (int c = wave % SPLIT; c < chunks; c += SPLIT) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int b = 8 * c + 2 * q + j;
      const bool in = b < nb;
      const int bc = in ? b : nb - 1;        // a block past the row: zeros with scale 1
      mi4 w = *reinterpret_cast<const mi4*>(wc + 16 * bc);
      const uint32_t sw = in ? ws[bc] : kOne;
      if (!in) w = mi4{0, 0, 0, 0};
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const mi4 x = *reinterpret_cast<const mi4*>(xc[m] + 16 * bc);
        const uint32_t sx = in ? xs[m][bc] : kOne;
        acc[m] = mfma_fp4(w, x, acc[m], sw, sx);
      }
    }
  }
  if constexpr (SPLIT > 1) {
    __shared__ mf4 part[TILES][SPLIT - 1][MT][64];
    const int ti = wave / SPLIT, si = wave % SPLIT;
    if (si > 0) {
#pragma unroll
      for (int m = 0; m < MT; ++m) part[ti][si - 1][m][lane] = acc[m];
    }
    __syncthreads();
    if (si > 0) return;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < SPLIT - 1; ++i) acc[m] += part[ti][i][m][lane];
  }
  if (!here) return;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int local = 16 * m + r;
    if (local < t.rows)
      store_out<GATED, BF16>(a, t.r0 + local, n0 + 4 * q, ok[m] ? acc[m] : mf4{0, 0, 0, 0});
  }
}

template <bool GATED, bool BF16>
void launch_rows(const LinearArgs& a, hipStream_t s) {
  constexpr int MT = 4, SPLIT = 4;
  const int64_t full = (a.R + 16 * MT - 1) / (16 * MT);
  const int64_t tiles = a.offsets ? (a.R / (16 * MT)) + min(static_cast<int64_t>(a.G), a.R) : full;
  const unsigned grid = static_cast<unsigned>(tiles * ((a.N + 15) / 16));
  mx_linear_rows_kernel<MT, SPLIT, GATED, BF16><<<grid, ML_THREADS, 0, s>>>(a);
}

}  // namespace

hipError_t launch_mx_linear(const moe_mxfp4& A, const moe_mxfp4& W, const int32_t* offsets,
                            const int32_t* row_src, int src_div, int64_t R, void* y, int y_dtype,
                            bool gated, hipStream_t s) {
  LinearArgs a;
  a.ac = static_cast<const uint8_t*>(A.codes);
  a.as = static_cast<const uint8_t*>(A.scales);
  a.wc = static_cast<const uint8_t*>(W.codes);
  a.ws = static_cast<const uint8_t*>(W.scales);
  a.offsets = offsets;
  a.row_src = row_src;
  a.y = y;
  a.R = R;
  a.a_rows = A.rows;
  a.G = W.n_mats;
  a.N = W.rows;
  a.K = W.cols;
  a.src_div = src_div;
  const bool bf16 = y_dtype == MOE_DTYPE_BF16;
  if (gated)
    bf16 ? launch_rows<true, true>(a, s) : launch_rows<true, false>(a, s);
  else
    bf16 ? launch_rows<false, true>(a, s) : launch_rows<false, false>(a, s);
  return hipGetLastError();
}

}  // namespace bitffn
