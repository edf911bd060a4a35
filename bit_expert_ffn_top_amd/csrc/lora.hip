// Low-rank adapters of many requests beside a projection that they share:
//   y[t] = base[t] + scale[m] * B_m (A_m x[t]),   m the adapter of t's request
//
// A workgroup takes 16 or 32 consecutive rows of one request (a row alone where
// every row is a request) and a slice of the output columns, in one launch: the
// product with A needs all of x before B can start, but A is small (64 KB at rank
// 16 and 2048 columns), so that a slice's repeating it costs less than a second
// launch.  Both products are on the matrix cores, with the adapter's rows as the
// first operand, so that a lane of the result holds consecutive ranks or columns
// of one token:
//   h = A x    the eight wavefronts split the columns; their sums meet in LDS in
//              a fixed order
//   y = B h    the wavefronts split the slice's columns
// fp32 values enter as sums of bfloat16 parts: x as three (exact but for its
// smallest values), h as two where the results are bfloat16 (off by 2^-16 of it,
// where they round by 2^-8) and three where they are fp32.  A row has the same
// bits whatever other rows there are.
#include "moe_internal.h"
#include "row_device.h"
#include "scan_device.h"

namespace bitffn {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kGroup = 64;   // output columns that a wavefront takes at a time

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));

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
  int slice;   // output columns of a workgroup, a multiple of kGroup
};

__device__ __forceinline__ nf4 mfma(nu4 a, nu4 b, nf4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b),
                                                 c, 0, 0, 0);
}

// Eight consecutive values of x as bfloat16 parts.
template <typename XT>
struct XPart;

template <>
struct XPart<uint16_t> {
  static constexpr int kParts = 1;
  nu4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const nu4*>(p); }
  __device__ __forceinline__ void split(nu4 (&out)[1]) const { out[0] = v; }
};

// The high halves of two words.
__device__ __forceinline__ uint32_t high_halves(float lo, float hi) {
  return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, hi), __builtin_bit_cast(uint32_t, lo), 0x07060302u);
}

template <>
struct XPart<float> {
  static constexpr int kParts = 3;
  nf4 v[2];
  __device__ __forceinline__ void load(const float* p) {
    v[0] = reinterpret_cast<const nf4*>(p)[0];
    v[1] = reinterpret_cast<const nf4*>(p)[1];
  }
  // Each part takes the highest eight bits that are left: 24 in all.
  __device__ __forceinline__ void split(nu4 (&out)[3]) const {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = v[i / 4][i % 4];
#pragma unroll
    for (int part = 0; part < 3; ++part) {
#pragma unroll
      for (int i = 0; i < 4; ++i) out[part][i] = high_halves(r[2 * i], r[2 * i + 1]);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        r[i] -= __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, r[i]) & 0xFFFF0000u);
    }
  }
};

// Rows [row0, row1) and request of one tile of `rows` rows; false if there are
// fewer tiles.  A request's rows end at the largest bound so far, clamped to the
// rows there are.  Every wavefront searches for itself, eight bounds per lane.
__device__ __forceinline__ bool find_tile(const LoraArgs& g, int tile, int rows, int& row0, int& row1,
                                          int& request) {
  if (!g.seq) {
    row0 = request = tile;
    row1 = tile + 1;
    return tile < g.T;
  }
  constexpr int kPer = 8;
  const int lane = threadIdx.x & 63;
  int low = min(max(g.seq[0], 0), g.T);   // largest bound so far
  int before = 0;                         // tiles of the requests so far
  for (int s0 = 0; s0 < g.n_seq; s0 += 64 * kPer) {
    int end[kPer], top = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int s = s0 + lane * kPer + j;
      end[j] = s < g.n_seq ? min(max(g.seq[s + 1], 0), g.T) : 0;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) end[j] = top = max(top, end[j]);
    const int upto = wave_scan_max(top);
    const int start = max(low, lane_before(upto));
    int tiles = 0, at = start;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      end[j] = max(end[j], start);
      tiles += (end[j] - at + rows - 1) / rows;
      at = end[j];
    }
    const int sum = before + wave_scan_add(tiles);
    const uint64_t past = __ballot(sum > tile);
    if (past) {
      const int who = __builtin_ctzll(past);
      int left = tile - (sum - tiles), r0 = 0, r1 = 0, req = 0;
      at = start;
      bool found = false;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int n = (end[j] - at + rows - 1) / rows;
        if (!found && left < n) {
          found = true;
          r0 = at + left * rows;
          r1 = min(end[j], r0 + rows);
          req = s0 + lane * kPer + j;
        }
        if (!found) left -= n;
        at = end[j];
      }
      row0 = lane_value(r0, who);
      row1 = lane_value(r1, who);
      request = lane_value(req, who);
      return true;
    }
    before = lane_value(sum, 63);
    low = max(low, lane_value(upto, 63));
  }
  return false;
}

// MT: 16-rank tiles (rank <= 16 MT); NT: 16-row tiles.
template <typename XT, typename YT, int MT, int NT>
__global__ __launch_bounds__(kThreads) void lora_kernel(LoraArgs g) {
  constexpr int XP = XPart<XT>::kParts;
  constexpr int HP = sizeof(YT) == 4 ? 3 : 2;   // parts of h
  constexpr int RS = (MT + 1) / 2;              // 32-rank steps of the second product
  constexpr int kPartRow = 16 * MT + 4;         // LDS rows, padded against bank conflicts
  constexpr int kHRow = 32 * RS + 8;
  __shared__ __align__(16) float s_part[kWaves][16 * NT][kPartRow];
  __shared__ __align__(16) uint16_t s_h[HP][16 * NT][kHRow];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l16 = lane & 15, quad = lane >> 4;
  int row0, row1, request;
  if (!find_tile(g, blockIdx.x, 16 * NT, row0, row1, request)) return;
  const int m = g.adapter[request];
  const int n0 = blockIdx.y * g.slice, n1 = min(g.d_out, n0 + g.slice);
  const YT* base = static_cast<const YT*>(g.base);
  YT* y = static_cast<YT*>(g.y);
  if (m < 0 || m >= g.n_adapters) {   // no adapter
    if (y == base) return;
    const int parts = (n1 - n0) / 8;
    for (int i = tid; i < (row1 - row0) * parts; i += kThreads) {
      const int t = i / parts;
      const int64_t at = static_cast<int64_t>(row0 + t) * g.d_out + n0 + 8 * (i - t * parts);
      RowPart<YT, 8> v;
      v.load(base + at);
      v.store(y + at);
    }
    return;
  }
  const float scale = g.scale ? g.scale[m] : 1.0f;

  // h = A x: lane (l16, quad) reads 8 columns of row l16 of each operand
  {
    const uint16_t* a = g.a + static_cast<int64_t>(m) * g.rank * g.d_in + 8 * quad;
    const XT* x = static_cast<const XT*>(g.x) + 8 * quad;
    const uint16_t* ar[MT];
    const XT* xr[NT];
#pragma unroll
    for (int i = 0; i < MT; ++i) ar[i] = a + static_cast<int64_t>(min(16 * i + l16, g.rank - 1)) * g.d_in;
#pragma unroll
    for (int i = 0; i < NT; ++i) xr[i] = x + static_cast<int64_t>(min(row0 + 16 * i + l16, row1 - 1)) * g.d_in;
    nf4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = nf4{0.0f, 0.0f, 0.0f, 0.0f};
    const int steps = g.d_in / 32, per = (steps + kWaves - 1) / kWaves;
    const int k0 = min(steps, wave * per), k1 = min(steps, k0 + per);
    constexpr int U = MT * NT <= 2 ? 8 : MT * NT <= 4 ? 4 : 2;
    for (int k = k0; k < k1; k += U) {
      nu4 av[U][MT];
      XPart<XT> xv[U][NT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = 32 * min(k + u, k1 - 1);
#pragma unroll
        for (int i = 0; i < MT; ++i) av[u][i] = *reinterpret_cast<const nu4*>(ar[i] + c);
#pragma unroll
        for (int j = 0; j < NT; ++j) xv[u][j].load(xr[j] + c);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (k + u < k1) {   // uniform
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            nu4 xp[XP];
            xv[u][j].split(xp);
#pragma unroll
            for (int part = 0; part < XP; ++part)
#pragma unroll
              for (int i = 0; i < MT; ++i) acc[i][j] = mfma(av[u][i], xp[part], acc[i][j]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        *reinterpret_cast<nf4*>(&s_part[wave][16 * j + l16][16 * i + 4 * quad]) = acc[i][j];
  }
  __syncthreads();
  for (int i = tid; i < 16 * NT * 32 * RS; i += kThreads) {
    const int t = i / (32 * RS), r = i - t * (32 * RS);
    float h = 0.0f;
    if (r < g.rank) {
#pragma unroll
      for (int w = 0; w < kWaves; ++w) h += s_part[w][t][r];
      h *= scale;
    }
#pragma unroll
    for (int part = 0; part < HP; ++part) {
      const uint32_t p = pack_bf16(h, 0.0f) & 0xFFFFu;
      s_h[part][t][r] = static_cast<uint16_t>(p);
      const float v = bf16_bits_to_float(p);
      h = __builtin_isfinite(v) ? h - v : 0.0f;   // an infinity has no rest
    }
  }
  __syncthreads();

  // y = base + B h: rows of B are dealt to the two results of 32 columns so that
  // a lane holds columns 8 quad .. 8 quad + 7 of token l16
  nu4 hv[HP][RS][NT];
#pragma unroll
  for (int part = 0; part < HP; ++part)
#pragma unroll
    for (int s = 0; s < RS; ++s)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        hv[part][s][j] = *reinterpret_cast<const nu4*>(&s_h[part][16 * j + l16][32 * s + 8 * quad]);
  const uint16_t* b = g.b + static_cast<int64_t>(m) * g.d_out * g.rank;
  const int column = 8 * (l16 >> 2) + (l16 & 3);   // of this lane's row of B, the second result's 4 further
  const int groups = (n1 - n0 + kGroup - 1) / kGroup, per = (groups + kWaves - 1) / kWaves;
  for (int k = wave * per; k < min(groups, (wave + 1) * per); ++k) {
    const int c0 = n0 + k * kGroup;
#pragma unroll
    for (int blk = 0; blk < kGroup / 32; ++blk) {
      const int c = c0 + 32 * blk;
      if (c >= n1) break;   // uniform
      nu4 bv[2][RS];
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int s = 0; s < RS; ++s) {
          const int r = 32 * s + 8 * quad;
          const int64_t at = static_cast<int64_t>(min(c + column + 4 * half, g.d_out - 1)) * g.rank;
          const nu4 v = *reinterpret_cast<const nu4*>(b + at + min(r, g.rank - 8));
          bv[half][s] = r < g.rank ? v : nu4{0, 0, 0, 0};
        }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int t = row0 + 16 * j + l16;
        const bool there = t < row1 && c + 8 * quad < n1;
        const int64_t at = static_cast<int64_t>(t) * g.d_out + c + 8 * quad;
        RowPart<YT, 8> v;
        if (there) v.load(base + at);
        nf4 acc[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          acc[half] = nf4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int s = 0; s < RS; ++s)
#pragma unroll
            for (int part = 0; part < HP; ++part)
              acc[half] = mfma(bv[half][s], hv[part][s][j], acc[half]);
        }
        if (there) {
          float f[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = v.get(i) + acc[i / 4][i % 4];
          v.set(f);
          v.store(y + at);
        }
      }
    }
  }
}

template <typename XT, typename YT, int NT>
void launch_tiles(LoraArgs g, hipStream_t s) {
  const int rows = 16 * NT;
  // ceil(n / rows) summed over the requests is at most this
  const int64_t tiles = g.seq ? (g.T + static_cast<int64_t>(rows - 1) * min(g.n_seq, g.T)) / rows : g.T;
  const int groups = (g.d_out + kGroup - 1) / kGroup;
  const int slices = static_cast<int>(max(int64_t{1}, min(int64_t{(groups + kWaves - 1) / kWaves}, 512 / tiles)));
  g.slice = (groups + slices - 1) / slices * kGroup;
  const dim3 grid(static_cast<unsigned>(tiles), (g.d_out + g.slice - 1) / g.slice);
  if (g.rank <= 16)
    lora_kernel<XT, YT, 1, NT><<<grid, kThreads, 0, s>>>(g);
  else if (g.rank <= 32)
    lora_kernel<XT, YT, 2, NT><<<grid, kThreads, 0, s>>>(g);
  else if (g.rank <= 64)
    lora_kernel<XT, YT, 4, NT><<<grid, kThreads, 0, s>>>(g);
  else
    lora_kernel<XT, YT, 8, NT><<<grid, kThreads, 0, s>>>(g);
}

template <typename XT, typename YT>
hipError_t launch_as(const LoraArgs& g, hipStream_t s) {
  launch_tiles<XT, YT, 1>(g, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lora(const void* base, const void* x, int x_dtype, int64_t T, int d_in, int d_out,
                       const uint16_t* a, const uint16_t* b, int n_adapters, int rank,
                       const int32_t* seq, int n_seq, const int32_t* adapter, const float* scale,
                       void* y, int y_dtype, hipStream_t s) {
  const LoraArgs g{base, x, a, b, seq, adapter, scale, y, static_cast<int>(T),
                   d_in, d_out, n_adapters, rank, n_seq, 0};
  const bool xf = x_dtype == MOE_DTYPE_F32, yf = y_dtype == MOE_DTYPE_F32;
  const auto f = xf ? (yf ? launch_as<float, float> : launch_as<float, uint16_t>)
                    : (yf ? launch_as<uint16_t, float> : launch_as<uint16_t, uint16_t>);
  return f(g, s);
}

}  // namespace bitffn
