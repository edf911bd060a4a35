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
typedef uint32_t mu2 __attribute__((ext_vector_type(2)));
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
  int G, N, K;
  // row_src[r] / src_div = row_src[r] * div_mul >> div_shift, exact below 2^31
  uint32_t div_mul;
  int div_shift;
};

// What a wavefront works on: rows r0 .. r0 + rows - 1 of group g.
struct RowTile {
  int g;
  int rows;
  int64_t r0;
  bool whole;   // all rows of the group
};

// Number `at` of the row tiles that XCD `xcd` takes (xcd < 0: of all), which is
// an eighth of the row tiles of all groups, in order: neighbouring tiles mostly
// belong to one group, and what they share meets in one L2.  tile_m rows each,
// the last of a group shorter.  All threads of the workgroup take part; rows = 0
// past the last tile.  Each thread counts the tiles of its own run of groups;
// the runs are scanned over the workgroup, and the thread whose run holds the
// tile says where it lies.
__device__ __forceinline__ RowTile find_row_tile(const LinearArgs& a, int xcd, int at_tile, int tile_m) {
  const auto number = [&](int total) {   // of the tile among all, -1 if there is none
    if (xcd < 0) return at_tile;
    const int share = (total + 7) / 8;
    return at_tile < share ? xcd * share + at_tile : -1;
  };
  if (a.offsets == nullptr) {
    const int tile = number(static_cast<int>((a.R + tile_m - 1) / tile_m));
    if (tile < 0) return RowTile{0, 0, 0, true};
    const int64_t r0 = static_cast<int64_t>(tile) * tile_m;
    return RowTile{0, static_cast<int>(min(static_cast<int64_t>(tile_m), max(a.R - r0, int64_t{0}))), r0,
                   a.R <= tile_m};
  }
  __shared__ int s_wave[ML_THREADS / 64], s_top[ML_THREADS / 64], s_bad[ML_THREADS / 64];
  __shared__ int s_g, s_rows, s_r0, s_whole;
  const int tid = threadIdx.x, lane = tid & 63;
  constexpr int kPer = (MOE_MAX_EXPERTS + ML_THREADS - 1) / ML_THREADS;
  const int R = static_cast<int>(a.R);
  int bound[kPer + 1], nt[kPer], mine = 0;
#pragma unroll
  for (int i = 0; i <= kPer; ++i) {
    const int v = a.offsets[min(tid * kPer + i, a.G)];
    bound[i] = min(max(v, 0), R);
  }
  const auto count = [&]() {   // this thread's tiles; their scan over the wavefront, inclusive
    mine = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      bad |= bound[i + 1] < bound[i];
      nt[i] = (max(bound[i + 1] - bound[i], 0) + tile_m - 1) / tile_m;
      mine += nt[i];
    }
    int scan = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int v = __shfl_up(scan, off, 64);
      if (lane >= off) scan += v;
    }
    bad = __any(bad);
    if (lane == 63) s_wave[tid >> 6] = scan, s_bad[tid >> 6] = bad;
    return scan;
  };
  int scan = count();
  if (tid == 0) s_rows = 0;
  __syncthreads();
  bool bad = false;
#pragma unroll
  for (int w = 0; w < ML_THREADS / 64; ++w) bad |= s_bad[w] != 0;
  if (bad) {   // a bound below an earlier one counts as that one: no row is in two groups
    __syncthreads();
    int top = bound[0];
#pragma unroll
    for (int i = 1; i <= kPer; ++i) top = max(top, bound[i]);
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) top = max(top, __shfl_up(top, off, 64));   // lane < off: its own
    if (lane == 63) s_top[tid >> 6] = top;
    __syncthreads();
    int before = __shfl_up(top, 1, 64);
    if (lane == 0) before = 0;
    for (int w = 0; w < tid >> 6; ++w) before = max(before, s_top[w]);
#pragma unroll
    for (int i = 0; i <= kPer; ++i) bound[i] = before = max(before, bound[i]);
    scan = count();
    __syncthreads();
  }
  int at = scan - mine, total = 0;
#pragma unroll
  for (int w = 0; w < ML_THREADS / 64; ++w) {
    at += w < (tid >> 6) ? s_wave[w] : 0;
    total += s_wave[w];
  }
  const int tile = number(total);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (tile >= at && tile < at + nt[i]) {   // one thread, one i
      const int r0 = bound[i] + (tile - at) * tile_m;
      s_g = tid * kPer + i;
      s_r0 = r0;
      s_rows = min(tile_m, bound[i + 1] - r0);
      s_whole = nt[i] == 1;
    }
    at += nt[i];
  }
  __syncthreads();
  // the same in every thread: kept in scalar registers
  return RowTile{__builtin_amdgcn_readfirstlane(s_g), __builtin_amdgcn_readfirstlane(s_rows),
                 __builtin_amdgcn_readfirstlane(s_r0), __builtin_amdgcn_readfirstlane(s_whole) != 0};
}

// A's row for output row r; 0 and ok = false if there is none.
__device__ __forceinline__ int source_row(const LinearArgs& a, int64_t r, bool& ok) {
  if (!a.row_src) {
    ok = true;   // R is at most A's rows
    return static_cast<int>(r);
  }
  const int v = a.row_src[r];
  const uint32_t s = static_cast<uint32_t>(static_cast<uint64_t>(static_cast<uint32_t>(v)) * a.div_mul >> a.div_shift);
  ok = v >= 0 && s < static_cast<uint32_t>(a.a_rows);
  return ok ? static_cast<int>(s) : 0;
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

// silu(z) = z / (1 + e^-z).  The product with log2(e) is carried in two parts,
// so the exponential is good to about 2 units in the last place for every z;
// the hardware's exponential and reciprocal are each good to 1.  Past +-126
// the exponential is 0 or infinite either way.
__device__ __forceinline__ float silu_hw(float z) {
  const float c = __builtin_amdgcn_fmed3f(z, -126.0f, 126.0f);
  const float t = -c * 1.44269502f;                                  // log2(e), rounded
  const float lo = fmaf(-c, 1.44269502f, -t) - c * 1.92596303e-8f;   // what both roundings lost
  const float e = __builtin_amdgcn_exp2f(t) * fmaf(lo, 0.693147182f, 1.0f);
  return z * __builtin_amdgcn_rcpf(1.0f + e);
}

// Four consecutive output columns of a row, put at p in LDS.  GATED: the columns
// are (gate, up, gate, up) and two values are put there.
template <bool GATED, bool BF16>
__device__ __forceinline__ void put_out(__attribute__((address_space(3))) uint8_t* p, mf4 v) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  if constexpr (GATED) {
    const float h0 = silu_hw(v[0]) * v[1], h1 = silu_hw(v[2]) * v[3];
    if constexpr (BF16)
      *(__attribute__((address_space(3))) uint32_t*)p = pack_bf16(h0, h1);
    else
      *(__attribute__((address_space(3))) f2*)p = f2{h0, h1};
  } else if constexpr (BF16) {
    *(__attribute__((address_space(3))) mu2*)p = mu2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
  } else {
    *(__attribute__((address_space(3))) mf4*)p = v;
  }
}

// The same, stored at p in memory.
template <bool GATED, bool BF16>
__device__ __forceinline__ void store_out(uint8_t* p, mf4 v) {
  if constexpr (GATED) {
    const float h0 = silu_hw(v[0]) * v[1], h1 = silu_hw(v[2]) * v[3];
    if constexpr (BF16)
      *reinterpret_cast<uint32_t*>(p) = pack_bf16(h0, h1);
    else
      *reinterpret_cast<float2*>(p) = make_float2(h0, h1);
  } else if constexpr (BF16) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
}

// Place of 16-byte piece p of row r of 128 bytes in LDS: p ^ mg_swz(r).
__host__ __device__ constexpr int mg_swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// Keeps the compiler to the program order of this wavefront's LDS accesses
// (which is the order in which they take effect).
__device__ __forceinline__ void mg_wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Few rows per group: a wavefront takes 16 weight rows and up to 4 tiles of 16
// tokens.  SPLIT wavefronts share one 16-row tile, each with its share of the
// 256-column chunks (chunk c belongs to wavefront c % SPLIT), and their sums meet
// in LDS in wavefront order.  Every chunk of 16 rows is read as it lies, 8 rows
// of 128 bytes per instruction, the next one while this one is multiplied, and
// passes through a piece of LDS of the wavefront's own to the lanes that
// multiply it: read where they want it, 16 bytes a row, it costs the path from
// the caches 64 bytes for each 16.
// Bound: HBM (the weights) and, with little of them, latency.  37 tokens x 4 over
// 60 experts of 1040 x 704: 7.1 us for 23 MB (3.2 TB/s; every token tile
// multiplied, operands read where they are wanted: 11.9 us); one row to each of
// 30 experts of 2048 x 4096: 35 us for 134 MB (3.8 TB/s).
constexpr int MR_TILES = 4;
constexpr int MR_PIECE = 16 * 128 + 16 * 8;   // LDS of 16 rows of a chunk: codes, scales

// 16 rows of a chunk: 16-byte piece lane % 8 of rows lane / 8 and 8 more, and two
// scales of row lane / 4.  rows: where the first, the second and the scales' row
// begin.
struct MrRows {
  mi4 c[2];
  uint32_t s;

  template <bool STREAM>
  __device__ __forceinline__ void load(const uint8_t* c0, const uint8_t* c1, const uint8_t* sc, int nb, int chunk) {
    const int lane = threadIdx.x & 63;
    const int piece = min(8 * chunk + (lane & 7), nb - 1);   // past a row: its last, not used
    const mi4* p0 = reinterpret_cast<const mi4*>(c0 + 16 * piece);
    const mi4* p1 = reinterpret_cast<const mi4*>(c1 + 16 * piece);
    c[0] = STREAM ? __builtin_nontemporal_load(p0) : *p0;
    c[1] = STREAM ? __builtin_nontemporal_load(p1) : *p1;
    const int b = 8 * chunk + 2 * (lane & 3);
    if (nb % 2 == 0)
      s = *reinterpret_cast<const uint16_t*>(sc + min(b, nb - 2));
    else
      s = sc[min(b, nb - 1)] | sc[min(b + 1, nb - 1)] << 8;
  }

  __device__ __forceinline__ void put(uint8_t* to) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = 8 * j + (lane >> 3);
      *reinterpret_cast<mi4*>(to + 128 * row + 16 * ((lane & 7) ^ mg_swz(row))) = c[j];
    }
    *reinterpret_cast<uint16_t*>(to + 16 * 128 + 2 * lane) = static_cast<uint16_t>(s);
  }
};

// What lane l multiplies: blocks 2 (l / 16) and the next of row l % 16.
struct MrOperand {
  mi4 c[2];
  uint32_t s[2];

  __device__ __forceinline__ void get(const uint8_t* from, int nb, int chunk, bool weights) {
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const uint32_t both = *reinterpret_cast<const uint16_t*>(from + 16 * 128 + 8 * r + 2 * q);
    s[0] = both & 0xFFu;
    s[1] = both >> 8;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      c[j] = *reinterpret_cast<const mi4*>(from + 128 * r + 16 * ((2 * q + j) ^ mg_swz(r)));
      if (8 * chunk + 2 * q + j >= nb) {   // past the row: zeros with scale 1
        s[j] = kOne;
        if (weights) c[j] = mi4{0, 0, 0, 0};
      }
    }
  }
};

struct MrAt {
  const uint8_t* c0;
  const uint8_t* c1;
  const uint8_t* s;
};

// The sums of M token tiles over chunks first, first + step, .., AHEAD of them
// on their way.
template <int M, int AHEAD, bool STREAM>
__device__ __forceinline__ void mr_sums(mf4 (&acc)[MR_TILES], const MrAt& w, const MrAt (&x)[MR_TILES],
                                        uint8_t* lds, int nb, int first, int step) {
  const int chunks = (nb + 7) / 8;
  MrRows nw[AHEAD], nx[AHEAD][M];
  const auto load = [&](int d, int c) {
    if (c >= chunks) return;
    nw[d].template load<STREAM>(w.c0, w.c1, w.s, nb, c);
#pragma unroll
    for (int m = 0; m < M; ++m) nx[d][m].template load<false>(x[m].c0, x[m].c1, x[m].s, nb, c);
  };
#pragma unroll
  for (int d = 0; d < AHEAD; ++d) load(d, first + d * step);
  for (int c0 = first; c0 < chunks; c0 += AHEAD * step) {
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) {
      const int c = c0 + d * step;
      if (c >= chunks) break;
      mg_wave_sync();
      nw[d].put(lds);
      MrOperand ow, ox;
#pragma unroll
      for (int m = 0; m < M; ++m) {
        nx[d][m].put(lds + MR_PIECE);
        if (m + 1 == M) load(d, c + AHEAD * step);
        mg_wave_sync();
        if (m == 0) ow.get(lds, nb, c, true);
        ox.get(lds + MR_PIECE, nb, c, false);
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[m] = mfma_fp4(ow.c[j], ox.c[j], acc[m], ow.s[j], ox.s[j]);
        mg_wave_sync();
      }
    }
  }
}

template <int SPLIT, bool GATED, bool BF16>
__global__ __launch_bounds__(ML_THREADS) void mx_linear_rows_kernel(LinearArgs a, int64_t first) {
  constexpr int WAVES = ML_THREADS / 64;
  constexpr int TILES = WAVES / SPLIT;       // 16-row weight tiles per workgroup
  constexpr int kPart = SPLIT > 1 ? TILES * (SPLIT - 1) * MR_TILES * 64 * static_cast<int>(sizeof(mf4)) : 0;
  __shared__ __align__(16) uint8_t lds[kPart > WAVES * 2 * MR_PIECE ? kPart : WAVES * 2 * MR_PIECE];
  const int n_wg = (a.N + 16 * TILES - 1) / (16 * TILES);
  const int64_t at_wg = first + blockIdx.x;
  const RowTile t = find_row_tile(a, -1, static_cast<int>(at_wg / n_wg), 16 * MR_TILES);
  if (t.rows <= 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int n0 = (static_cast<int>(at_wg % n_wg) * TILES + wave / SPLIT) * 16;
  const bool here = n0 < a.N;                // the last workgroup may have tiles to spare
  const int nb = a.K / 32;                   // blocks of a row
  const int64_t crow = a.K / 2;
  const int64_t wrow = static_cast<int64_t>(t.g) * a.N + min(n0, a.N - 16);
  const MrAt w = {a.wc + (wrow + (lane >> 3)) * crow, a.wc + (wrow + 8 + (lane >> 3)) * crow,
                  a.ws + (wrow + (lane >> 2)) * nb};
  // lane i: the source of the tile's row i, complemented where it has none
  static_assert(16 * MR_TILES == 64, "a row of the tile per lane");
  bool ok;
  const int s = source_row(a, t.r0 + min(lane, t.rows - 1), ok);
  const int src = ok ? s : ~s;
  MrAt x[MR_TILES];
#pragma unroll
  for (int m = 0; m < MR_TILES; ++m) {
    const auto row = [&](int i) {            // widened: offsets may pass 2^32
      const int v = __shfl(src, 16 * m + i, 64);
      return static_cast<int64_t>(v < 0 ? ~v : v);
    };
    x[m] = MrAt{a.ac + row(lane >> 3) * crow, a.ac + row(8 + (lane >> 3)) * crow, a.as + row(lane >> 2) * nb};
  }
  mf4 acc[MR_TILES] = {};
  uint8_t* mine = lds + 2 * MR_PIECE * wave;
  // weights that only this tile reads stream past the caches (16 experts of
  // 4096 x 4096, a row each: 57 -> 34 us)
  if (!t.whole)
    mr_sums<MR_TILES, 1, false>(acc, w, x, mine, nb, wave % SPLIT, SPLIT);
  else if (t.rows <= 16)
    mr_sums<1, 4, true>(acc, w, x, mine, nb, wave % SPLIT, SPLIT);
  else if (t.rows <= 32)
    mr_sums<2, 2, true>(acc, w, x, mine, nb, wave % SPLIT, SPLIT);
  else
    mr_sums<MR_TILES, 1, true>(acc, w, x, mine, nb, wave % SPLIT, SPLIT);
  if constexpr (SPLIT > 1) {
    mf4* part = reinterpret_cast<mf4*>(lds);   // [TILES][SPLIT - 1][MR_TILES][64]
    const int ti = wave / SPLIT, si = wave % SPLIT;
    __syncthreads();
    if (si > 0) {
#pragma unroll
      for (int m = 0; m < MR_TILES; ++m) part[((ti * (SPLIT - 1) + si - 1) * MR_TILES + m) * 64 + lane] = acc[m];
    }
    __syncthreads();
    if (si > 0) return;
#pragma unroll
    for (int m = 0; m < MR_TILES; ++m)
#pragma unroll
      for (int i = 0; i < SPLIT - 1; ++i) acc[m] += part[((ti * (SPLIT - 1) + i) * MR_TILES + m) * 64 + lane];
  }
  if (!here) return;
#pragma unroll
  for (int m = 0; m < MR_TILES; ++m) {
    const int local = 16 * m + r;
    const bool has = __shfl(src, local, 64) >= 0;
    if (local < t.rows) {
      const int col = n0 + 4 * q;
      const int64_t at = (t.r0 + local) * (GATED ? a.N / 2 : a.N) + (GATED ? col / 2 : col);
      store_out<GATED, BF16>(static_cast<uint8_t*>(a.y) + at * (BF16 ? 2 : 4), has ? acc[m] : mf4{0, 0, 0, 0});
    }
  }
}

// Many rows per group.  A workgroup takes MG_ROWS weight rows and up to 16 CAP
// tokens of one group; each of its four wavefronts owns 64 of the weight rows
// (four MFMA tiles) for all the tokens, 256 columns per step: the more weight
// rows a wavefront has, the fewer times the tokens are read from LDS, which is
// the busiest part where groups are full.
//
// The MFMA wants row l % 16 in lane l, so a load straight into its operands
// would touch 64 places with 16 bytes each, and the path from the caches, which
// takes 64 contiguous bytes of four neighbouring lanes at a time, would be the
// bound (gate/up of 81,920 rows: 437 us so, 336 as below).  Everything is
// therefore loaded as it lies, 8 rows of 128 bytes per instruction, and changes
// lanes in LDS, 16-byte piece p of row r at position p ^ swz(r), which spreads
// the 16 rows that a read of one piece touches over all banks:
//   the tokens' codes, which all wavefronts share, by loads that write LDS
//     directly;
//   a wavefront's weights through its registers and a piece of LDS of its own,
//     without a barrier;
//   scales, four steps at a time, through registers;
// each requested one step ahead.
// The products of 2, 4, 6 or 8 token tiles are code of their own.
//
// Measured: gate/up of 81,920 rows over 512 experts, 1536 x 2048, bf16 out:
// 281 us a call, 1.8 PFLOP/s and 3.5 TB/s, the matrix cores busy 23% of the time;
// down, 2048 x 768, fp32 out: 298 us, 3.8 TB/s (671 MB of them stores), busy 10%;
// 640 rows over some 365 of those gate/up experts: 77 us, 8 TB/s, part of it from
// the last-level cache.  Rows of 704 or 2016 columns, whose scales come by bytes:
// 449 and 621 us where 768 and 2048 take 283 and 281.
// What is left, by the compiled code and the counters: two wavefronts per SIMD
// (256 registers each) of which each step waits for the next step's tokens
// before it asks for the next weights, because the compiler cannot tell the LDS
// that those loads write from the LDS it reads next; and registers that spill,
// 23 to 50 of them where a row is a multiple of 128 columns, 185 to 230 where it
// is not, which go to memory (8192 x 2048 x 768, bf16: 58 MB written for 34 MB of
// results) and whose reloads wait for the stores of a slice before them.
constexpr int MG_TILES = 4;              // of 16 weight rows per wavefront
constexpr int MG_ROWS = 4 * 16 * MG_TILES;
constexpr int MG_STEP = 256;             // columns per step
constexpr int MG_CHUNK = 4;              // steps per load of scales, 32 bytes of a row
constexpr uint32_t MG_OUT = 0x80000000u; // an offset outside every buffer: reads zeros, no traffic

typedef __amdgpu_buffer_rsrc_t MgRsrc;
typedef __attribute__((address_space(3))) uint8_t LdsByte;
typedef __attribute__((address_space(3))) mi4 LdsInt4;
typedef __attribute__((address_space(3))) mf4 LdsFloat4;
typedef __attribute__((address_space(3))) uint16_t LdsU16;

__device__ __forceinline__ MgRsrc mg_rsrc(const uint8_t* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0,
                                           static_cast<int>(static_cast<uint32_t>(bytes)), 0x00020000);
}

// Buffers (a read past one gives zeros) and this lane's byte offsets in them.
// Every offset is formed in full before the load: of a load's two offsets only
// the vector one is checked against the buffer's end.
struct MgLane {
  MgRsrc ac, as, wc, ws;
  uint32_t av[8];        // A codes: the row pieces this lane moves to LDS
  uint32_t asv;          // A scales: half a chunk of row tid / 2
  uint32_t wv;           // weights: piece lane % 8 of the wavefront's row lane / 8
  uint32_t wsv, ws32;    // weight scales: half a chunk of the wavefront's row lane / 2; 32 rows
  uint32_t w8;           // 8 rows of weights
  uint32_t wslice, wsslice;   // one slice of weight rows: codes, scales
  int nb, steps, slices, wave;
  bool stream;           // nobody else reads these weights: they need not stay in the caches
};

// 16 scale bytes as loaded, G at a time: 8 or 4 where that divides the blocks of
// a row, else 1, so that a load is aligned and lies wholly inside or outside the
// buffer.
template <int G>
struct MgScales {
  uint32_t v[G == 1 ? 16 : 4];
};

template <int G>
__device__ __forceinline__ void mg_load_s(MgScales<G>& s, MgRsrc rs, uint32_t at, int chunk) {
  at += chunk * (8 * MG_CHUNK);
  if constexpr (G == 8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const auto q = __builtin_amdgcn_raw_buffer_load_b64(rs, at + 8 * i, 0, 0);
      s.v[2 * i] = q[0];
      s.v[2 * i + 1] = q[1];
    }
  } else if constexpr (G == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s.v[i] = __builtin_amdgcn_raw_buffer_load_b32(rs, at + 4 * i, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) s.v[i] = __builtin_amdgcn_raw_buffer_load_b8(rs, at + i, 0, 0);
  }
}

// To LDS; b0 is the first block's number, a block past the row gets scale 1
// (its codes are zeros in the weights).
template <int G>
__device__ __forceinline__ void mg_put_s(const MgScales<G>& s, LdsByte* to, int b0, int nb) {
  mi4 v;
  if constexpr (G == 1) {
    v = mi4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      v[i >> 2] |= static_cast<int>((b0 + i < nb ? s.v[i] : kOne) << (8 * (i & 3)));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = static_cast<int>(G == 8 || b0 + 4 * i < nb ? s.v[i] : 0x01010101u * kOne);
  }
  *(LdsInt4*)to = v;
}

// This wavefront's weight rows of step c of a slice, 8 rows per instruction.
__device__ __forceinline__ void mg_load_w(mi4 (&w)[2 * MG_TILES], const MgLane& l, int slice, int c) {
  const uint32_t v = slice < l.slices ? l.wv + slice * l.wslice + c * 128 : MG_OUT;
  if (l.stream) {   // cache policy 2: nontemporal
#pragma unroll
    for (int j = 0; j < 2 * MG_TILES; ++j)
      w[j] = __builtin_bit_cast(mi4, __builtin_amdgcn_raw_buffer_load_b128(l.wc, v + j * l.w8, 0, 2));
  } else {
#pragma unroll
    for (int j = 0; j < 2 * MG_TILES; ++j)
      w[j] = __builtin_bit_cast(mi4, __builtin_amdgcn_raw_buffer_load_b128(l.wc, v + j * l.w8, 0, 0));
  }
}

// The codes of step c's tokens: 8 rows per instruction, the four wavefronts in
// turn (rows past the tile have offsets outside the buffer).
template <int NT>
__device__ __forceinline__ void mg_load_a(const MgLane& l, LdsByte* buf, int c) {
#pragma unroll
  for (int j = 0; j < (NT + 1) / 2; ++j)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        l.ac, (__attribute__((address_space(3))) void*)(buf + (4 * j + l.wave) * 1024), 16,
        l.av[j] + c * 128, 0, 0, 0);
}

// This lane's byte offsets of its two pieces of a tile's row, and of the row's
// scale bytes.
struct MgRead {
  int k0, k1, s;
};

// The operands of N tiles of 16 rows (weights or tokens).
template <int N>
struct MgTiles {
  mi4 x[N][2];
  int s[N];
};

__device__ __forceinline__ MgTiles<1> mg_read(const LdsByte* buf, const LdsByte* sbuf, const MgRead& at, int i) {
  MgTiles<1> x;
  x.x[0][0] = *(const LdsInt4*)(buf + at.k0 + 2048 * i);
  x.x[0][1] = *(const LdsInt4*)(buf + at.k1 + 2048 * i);
  x.s[0] = *(const LdsU16*)(sbuf + at.s + 16 * 8 * MG_CHUNK * i);
  return x;
}

template <int HALF>
__device__ __forceinline__ mf4 mg_mfma(mi4 w, mi4 x, mf4 c, int sw, int sx) {
  const mi8 a = {w.x, w.y, w.z, w.w, 0, 0, 0, 0};
  const mi8 b = {x.x, x.y, x.z, x.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, HALF, sw, HALF, sx);
}

// One step, a token tile at a time, the next on its way from LDS.  The sums
// are opaque afterwards: the compiler would move products past the barrier, to
// where their sums are used next.
template <int NT>
__device__ __forceinline__ void mg_multiply(mf4 (&acc)[NT][MG_TILES], const MgTiles<MG_TILES>& w,
                                            MgTiles<1> x, const LdsByte* buf, const LdsByte* sbuf,
                                            const MgRead& at) {
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    MgTiles<1> next = x;
    if (i + 1 < NT) next = mg_read(buf, sbuf, at, i + 1);
#pragma unroll
    for (int t = 0; t < MG_TILES; ++t)
      acc[i][t] = mg_mfma<0>(w.x[t][0], x.x[0][0], acc[i][t], w.s[t], x.s[0]);
#pragma unroll
    for (int t = 0; t < MG_TILES; ++t)
      acc[i][t] = mg_mfma<1>(w.x[t][1], x.x[0][1], acc[i][t], w.s[t], x.s[0]);
    x = next;
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int t = 0; t < MG_TILES; ++t) opaque(acc[i][t]);
}

// At most N of this wavefront's loads are still on their way (they arrive in
// order) and its LDS writes are done; then all wavefronts meet.
template <int N>
__device__ __forceinline__ void mg_barrier() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));   // vmcnt(N) lgkmcnt(0)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

template <int CAP>
struct MgShared {
  LdsByte* a[2];    // tokens' codes, 2048 bytes per tile
  LdsByte* w;       // this wavefront's: a weight tile, or results
  LdsByte* sa;      // tokens' scales: two chunks, 32 bytes per row
  LdsByte* sw;      // this wavefront's weight scales: two chunks
  static constexpr int kSa = CAP * 16 * 8 * MG_CHUNK;
  static constexpr int kSw = 16 * MG_TILES * 8 * MG_CHUNK;
  static constexpr int kW = 4096;
};

// The weights of step c from the registers through LDS into MFMA operands, a
// tile of 16 rows at a time; p: which half of the scales' LDS holds the step's
// chunk.
template <int G, int CAP>
__device__ __forceinline__ MgTiles<MG_TILES> mg_turn_w(mi4 (&w)[2 * MG_TILES], const MgShared<CAP>& m,
                                                       const MgLane& l, const MgRead& at, int p, int c) {
  const int lane = threadIdx.x & 63;
  if constexpr (G != 8) {   // a piece past the row belongs to the next one
    if (8 * c + (lane & 7) >= l.nb) {
#pragma unroll
      for (int j = 0; j < 2 * MG_TILES; ++j) w[j] = mi4{0, 0, 0, 0};
    }
  }
  const LdsByte* sbuf = m.sw + p * MgShared<CAP>::kSw + 8 * (c % MG_CHUNK);
  MgTiles<MG_TILES> x;
#pragma unroll
  for (int u = 0; u < MG_TILES; ++u) {
    mg_wave_sync();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = 8 * j + (lane >> 3);
      *(LdsInt4*)(m.w + 128 * row + 16 * ((lane & 7) ^ mg_swz(row))) = w[2 * u + j];
    }
    mg_wave_sync();
    x.x[u][0] = *(const LdsInt4*)(m.w + at.k0);
    x.x[u][1] = *(const LdsInt4*)(m.w + at.k1);
    x.s[u] = *(const LdsU16*)(sbuf + at.s + 16 * 8 * MG_CHUNK * u);
  }
  return x;
}

template <int CAP>
__device__ __forceinline__ const LdsByte* mg_scales_at(const MgShared<CAP>& m, int p, int c) {
  return m.sa + p * MgShared<CAP>::kSa + 8 * (c % MG_CHUNK);
}

// A chunk's scales on their way: of half a token row, and of half of two
// weight rows, 32 apart.
template <int G>
struct MgChunk {
  MgScales<G> a, w[2];
};

template <int G>
__device__ __forceinline__ void mg_load_chunk(MgChunk<G>& s, const MgLane& l, int slice, int chunk) {
  mg_load_s<G>(s.a, l.as, l.asv, chunk);
#pragma unroll
  for (int i = 0; i < 2; ++i) mg_load_s<G>(s.w[i], l.ws, l.wsv + slice * l.wsslice + i * l.ws32, chunk);
}

// Into half p of their LDS.
template <int CAP, int G>
__device__ __forceinline__ void mg_put_chunk(const MgShared<CAP>& m, const MgLane& l, const MgChunk<G>& s,
                                             int p, int chunk) {
  const int tid = threadIdx.x, lane = tid & 63, b0 = chunk * (8 * MG_CHUNK) + 16 * (tid & 1);
  if (tid < 32 * CAP) mg_put_s<G>(s.a, m.sa + p * MgShared<CAP>::kSa + 16 * tid, b0, l.nb);
#pragma unroll
  for (int i = 0; i < 2; ++i) mg_put_s<G>(s.w[i], m.sw + p * MgShared<CAP>::kSw + 16 * (lane + 64 * i), b0, l.nb);
}

// Where the products are: step c of a slice, its scales in half p.
struct MgAt {
  int slice, c, p;
};

// One step: its weights are in w, its tokens in m.a[B].  The tokens of the next
// step (of the next slice's first one, after the last) go into the other
// buffer, which the step before has left, its weights into w once this step's
// have left it.  At the first step of a chunk the next chunk's scales are
// requested, at its last they move on to LDS.  LAST: nothing follows.
template <int CAP, int NT, int G, int B, bool LAST>
__device__ __forceinline__ void mg_step(mf4 (&acc)[NT][MG_TILES], const MgShared<CAP>& m, const MgLane& l,
                                        const MgRead& at, MgAt& pos, mi4 (&w)[2 * MG_TILES], MgChunk<G>& sc) {
  const LdsByte* sbuf = mg_scales_at(m, pos.p, pos.c);
  if constexpr (LAST) {
    const MgTiles<MG_TILES> wp = mg_turn_w<G, CAP>(w, m, l, at, pos.p, pos.c);
    mg_multiply<NT>(acc, wp, mg_read(m.a[B], sbuf, at, 0), m.a[B], sbuf, at);
    return;
  }
  const bool ends = pos.c + 1 == l.steps;   // of the slice
  const int chunk = pos.c / MG_CHUNK;
  const bool chunk_ends = ends || pos.c % MG_CHUNK == MG_CHUNK - 1;
  const bool next_slice = ends || (chunk + 1) * MG_CHUNK >= l.steps;   // holds the next chunk
  const int next_chunk = next_slice ? 0 : chunk + 1;
  if (pos.c % MG_CHUNK == 0 && (!next_slice || pos.slice + 1 < l.slices)) {
    mg_load_chunk<G>(sc, l, pos.slice + (next_slice ? 1 : 0), next_chunk);
  }
  const int nc = ends ? 0 : pos.c + 1;
  mg_load_a<NT>(l, m.a[1 - B], nc);
  const MgTiles<MG_TILES> wp = mg_turn_w<G, CAP>(w, m, l, at, pos.p, pos.c);
  const MgTiles<1> x = mg_read(m.a[B], sbuf, at, 0);
  mg_load_w(w, l, pos.slice + (ends ? 1 : 0), nc);
  mg_multiply<NT>(acc, wp, x, m.a[B], sbuf, at);
  if (chunk_ends) mg_put_chunk<CAP, G>(m, l, sc, 1 - pos.p, next_chunk);
  pos.slice += ends ? 1 : 0;
  pos.c = nc;
  pos.p = chunk_ends ? 1 - pos.p : pos.p;
  mg_barrier<2 * MG_TILES>();   // newer than the next step's tokens: its weights
}

// The results of a slice: two tiles of 16 tokens at a time through this
// wavefront's piece of LDS, so that neighbouring lanes store neighbouring
// bytes, kPer lanes to a token; kPass weight tiles of it at a time, as fit.
// Leaves the sums zero.
template <int CAP, int NT, bool GATED, bool BF16>
__device__ __forceinline__ void mg_store(const LinearArgs& a, const RowTile& t, mf4 (&acc)[NT][MG_TILES],
                                         const MgShared<CAP>& m, int n0, const int* s_src) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  constexpr int kSize = BF16 ? 2 : 4, kHalf = GATED ? 2 : 1;
  constexpr int kPass = GATED || BF16 ? MG_TILES : MG_TILES / 2;
  constexpr int kRow = 16 * kPass / kHalf * kSize;   // bytes of a token
  static_assert(2 * 16 * kRow <= MgShared<CAP>::kW && NT % 2 == 0, "a wavefront's piece of LDS");
  constexpr int kPer = kRow / 16;
  const int width = a.N / kHalf;
#pragma unroll
  for (int i = 0; i < NT; i += 2) {
#pragma unroll
    for (int p = 0; p < MG_TILES / kPass; ++p) {
      const int col = (n0 + 16 * kPass * p) / kHalf;
      uint8_t* __restrict__ y = static_cast<uint8_t*>(a.y) + (t.r0 * width + col) * kSize;
      mg_wave_sync();
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bool has = s_src[16 * (i + u) + r] >= 0;
#pragma unroll
        for (int w = 0; w < kPass; ++w) {
          put_out<GATED, BF16>(m.w + (16 * u + r) * kRow + (16 * w + 4 * q) / kHalf * kSize,
                               has ? acc[i + u][kPass * p + w] : mf4{0, 0, 0, 0});
          acc[i + u][kPass * p + w] = mf4{0, 0, 0, 0};
        }
      }
      mg_wave_sync();
#pragma unroll
      for (int e = lane; e < 32 * kPer; e += 64) {
        const int row = 16 * i + e / kPer, piece = e % kPer;
        const mi4 v = *(const LdsInt4*)(m.w + 16 * e);
        if (row < t.rows && col + piece * (16 / kSize) < width)
          __builtin_nontemporal_store(v, reinterpret_cast<mi4*>(y + static_cast<uint32_t>(row * width) * kSize + 16 * piece));
      }
    }
  }
}

// NT: token tiles, at least the tile's rows.
template <int CAP, int NT, int G, bool GATED, bool BF16>
__device__ __forceinline__ void mg_tile(const LinearArgs& a, const RowTile& t, MgLane& l, int n0,
                                        const MgShared<CAP>& m, int* s_src) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int r = lane & 15, q = lane >> 4;
  mi4 w[2 * MG_TILES];
  MgChunk<G> sc;
  MgAt pos = {0, 0, 0};
  mg_load_w(w, l, 0, 0);
  // thread tid looks up tile row tid's source; the others take it from LDS
  if (tid < 16 * CAP) {
    bool ok = false;
    int src = -1;
    if (tid < t.rows) src = source_row(a, t.r0 + tid, ok);
    s_src[tid] = ok ? src : ~src;   // ~src >= 0 only past the tile's rows
  }
  __syncthreads();
  // the row pieces this lane moves: tile row 8 (4 j + wave) + lane / 8
#pragma unroll
  for (int j = 0; j < (NT + 1) / 2; ++j) {
    const int row = 8 * (4 * j + l.wave) + (lane >> 3);
    const int v = s_src[row];
    l.av[j] = row < t.rows ? static_cast<uint32_t>(v < 0 ? ~v : v) * (a.K / 2) + 16 * ((lane & 7) ^ mg_swz(row & 15))
                           : MG_OUT;
  }
  {
    const int row = tid >> 1;
    const int v = row < 16 * CAP ? s_src[row] : 0;
    l.asv = row < t.rows && row < 16 * CAP ? static_cast<uint32_t>(v < 0 ? ~v : v) * l.nb + 16 * (tid & 1) : MG_OUT;
  }
  const MgRead at = {r * 128 + 16 * ((2 * q) ^ mg_swz(r)), r * 128 + 16 * ((2 * q + 1) ^ mg_swz(r)),
                     r * (8 * MG_CHUNK) + 2 * q};
  mf4 acc[NT][MG_TILES] = {};
  mg_load_chunk<G>(sc, l, 0, 0);
  mg_load_a<NT>(l, m.a[0], 0);
  mg_put_chunk<CAP, G>(m, l, sc, 0, 0);
  mg_barrier<0>();
  const int total = l.slices * l.steps;
  int done = 0;   // slices stored
  for (int v = 0; v + 2 <= total; v += 2) {
    mg_step<CAP, NT, G, 0, false>(acc, m, l, at, pos, w, sc);
    if (pos.slice > done) mg_store<CAP, NT, GATED, BF16>(a, t, acc, m, n0 + MG_ROWS * done++, s_src);
    mg_step<CAP, NT, G, 1, false>(acc, m, l, at, pos, w, sc);
    if (pos.slice > done) mg_store<CAP, NT, GATED, BF16>(a, t, acc, m, n0 + MG_ROWS * done++, s_src);
  }
  if (total & 1) mg_step<CAP, NT, G, 0, true>(acc, m, l, at, pos, w, sc);
  __builtin_amdgcn_s_waitcnt(0x0F70);   // a load still on its way to LDS may not outlive the workgroup
  if (done < l.slices) mg_store<CAP, NT, GATED, BF16>(a, t, acc, m, n0 + MG_ROWS * done, s_src);
}

// slices: of MG_ROWS weight rows, one after the other, per workgroup.
template <int CAP, int G, bool GATED, bool BF16>
__global__ __launch_bounds__(ML_THREADS, 2) void mx_linear_groups_kernel(LinearArgs a,
                                                                                       int slices) {
  typedef MgShared<CAP> M;
  __shared__ __align__(16) uint8_t s_a0[CAP * 2048], s_a1[CAP * 2048];
  __shared__ __align__(16) uint8_t s_w[4 * M::kW];
  __shared__ __align__(16) uint8_t s_sa[2 * M::kSa], s_sw[4 * 2 * M::kSw];
  __shared__ int s_src[CAP * 16];   // each row's source, complemented where it has none
  // workgroups go to the 8 XCDs in turn; an XCD takes all slices of a tile, so
  // that the tile's token rows meet in its L2, then the next tile's
  const int n_slices = (a.N + MG_ROWS - 1) / MG_ROWS, n_wg = (n_slices + slices - 1) / slices;
  const int i = static_cast<int>(blockIdx.x) >> 3;
  const RowTile t = find_row_tile(a, static_cast<int>(blockIdx.x) & 7, i / n_wg, 16 * CAP);
  if (t.rows <= 0) return;
  const int s0 = i % n_wg * slices, n0 = s0 * MG_ROWS;
  const int lane = threadIdx.x & 63;
  const int nb = a.K / 32, crow = a.K / 2;
  MgLane l;
  l.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  l.nb = nb;
  l.steps = (a.K + MG_STEP - 1) / MG_STEP;
  l.slices = min(slices, n_slices - s0);
  l.stream = t.whole;
  l.ac = mg_rsrc(a.ac, a.a_rows * crow);
  l.as = mg_rsrc(a.as, a.a_rows * nb);
  const int64_t wrow = static_cast<int64_t>(t.g) * a.N;
  l.wc = mg_rsrc(a.wc + wrow * crow, static_cast<int64_t>(a.N) * crow);
  l.ws = mg_rsrc(a.ws + wrow * nb, static_cast<int64_t>(a.N) * nb);
  const int wave0 = n0 + 16 * MG_TILES * l.wave;   // the wavefront's first weight row
  l.wv = static_cast<uint32_t>((wave0 + (lane >> 3)) * crow + 16 * (lane & 7));
  l.wsv = static_cast<uint32_t>((wave0 + (lane >> 1)) * nb + 16 * (lane & 1));
  l.ws32 = 32 * nb;
  l.w8 = 8 * crow;
  l.wslice = MG_ROWS * crow;
  l.wsslice = MG_ROWS * nb;
  const M m = {{(LdsByte*)s_a0, (LdsByte*)s_a1}, (LdsByte*)s_w + M::kW * l.wave, (LdsByte*)s_sa,
               (LdsByte*)s_sw + 2 * M::kSw * l.wave};
  const int nt = (t.rows + 15) / 16;
  if constexpr (CAP >= 8) {
    if (nt > 6) return mg_tile<CAP, 8, G, GATED, BF16>(a, t, l, wave0, m, s_src);
    if (nt > 4) return mg_tile<CAP, 6, G, GATED, BF16>(a, t, l, wave0, m, s_src);
  }
  if (nt > 2) return mg_tile<CAP, 4, G, GATED, BF16>(a, t, l, wave0, m, s_src);
  mg_tile<CAP, 2, G, GATED, BF16>(a, t, l, wave0, m, s_src);
}

template <int CAP, bool GATED, bool BF16>
void launch_groups(const LinearArgs& a, hipStream_t s) {
  const int64_t m = 16 * CAP;
  const int64_t tiles = a.offsets ? a.R / m + min(static_cast<int64_t>(a.G), a.R) : (a.R + m - 1) / m;
  const int64_t n_slices = (a.N + MG_ROWS - 1) / MG_ROWS;
  // A workgroup's start (its tile, its rows' sources, the first loads) costs as
  // much as a third of a slice of 2,048 columns; two slices share it
  // where enough workgroups are left to even out the end (four: slower, the
  // token rows of the workgroups under way no longer fit the L2s).
  const int64_t want = int64_t{8} * device_cus();
  const int slices = static_cast<int>(min(max(tiles * n_slices / want, int64_t{1}), min(int64_t{2}, n_slices)));
  const unsigned grid = static_cast<unsigned>((tiles + 7) / 8 * 8 * ((n_slices + slices - 1) / slices));
  const int nb = a.K / 32;
  if (nb % 8 == 0)
    mx_linear_groups_kernel<CAP, 8, GATED, BF16><<<grid, ML_THREADS, 0, s>>>(a, slices);
  else if (nb % 4 == 0)
    mx_linear_groups_kernel<CAP, 4, GATED, BF16><<<grid, ML_THREADS, 0, s>>>(a, slices);
  else
    mx_linear_groups_kernel<CAP, 1, GATED, BF16><<<grid, ML_THREADS, 0, s>>>(a, slices);
}

constexpr int64_t kMaxBlocks = (int64_t{1} << 32) / ML_THREADS - 8;   // of a launch: 32 bits of threads

template <int SPLIT, bool GATED, bool BF16>
void launch_rows(const LinearArgs& a, int64_t tiles, hipStream_t s) {
  constexpr int per = 16 * (ML_THREADS / 64) / SPLIT;
  const int64_t n = tiles * ((a.N + per - 1) / per);
  for (int64_t first = 0; first < n; first += kMaxBlocks)
    mx_linear_rows_kernel<SPLIT, GATED, BF16><<<static_cast<unsigned>(min(n - first, kMaxBlocks)), ML_THREADS, 0, s>>>(a, first);
}

template <bool GATED, bool BF16>
void launch_rows(const LinearArgs& a, hipStream_t s) {
  constexpr int m = 16 * MR_TILES;
  const int64_t tiles = a.offsets ? a.R / m + min(static_cast<int64_t>(a.G), a.R) : (a.R + m - 1) / m;
  // A wavefront per 16 weight rows where that makes a workgroup for every CU, else
  // four that share the columns (one and four wavefronts, cold weights: 64 rows x
  // 8192 x 2048 in 128 workgroups 13.8 and 9.3 us; 40 rows over 8 experts of
  // 2048 x 768 in 256 8.2 and 10.2; a row to each of 16 experts of 4096 x 4096 in
  // 1024 34 and 40).
  if (tiles * (a.N / 64) >= device_cus())
    launch_rows<1, GATED, BF16>(a, tiles, s);
  else
    launch_rows<4, GATED, BF16>(a, tiles, s);
}

template <bool GATED, bool BF16>
void launch_product(const LinearArgs& a, hipStream_t s) {
  // The kernel for full tiles where it has two workgroups for every CU; its
  // offsets into A have 32 bits.  Full tiles and few rows, cold operands: 2048
  // rows x 2048 x 768 (128 workgroups) 18.3 and 15.2 us; 400 rows over 60 experts
  // of 1536 x 2048 (378) 28.4 and 28.6; 8192 rows x 2048 x 768 (512) 30 and 42; 640
  // rows over 400 experts (2430, tiles mostly empty) 134 and 135.
  const int64_t wgs = (a.offsets ? a.R / 128 + min(static_cast<int64_t>(a.G), a.R) : (a.R + 127) / 128) *
                      ((a.N + MG_ROWS - 1) / MG_ROWS);
  if (wgs >= 2 * device_cus() && a.a_rows * (a.K / 2) < int64_t{MG_OUT})
    launch_groups<8, GATED, BF16>(a, s);
  else
    launch_rows<GATED, BF16>(a, s);
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
  // with l = ceil(log2 d): ceil(2^(31+l) / d) < 2^32, and the error of the
  // rounded-up factor stays below 1 / d for every dividend below 2^31
  int l = 0;
  while ((int64_t{1} << l) < src_div) ++l;
  a.div_shift = 31 + l;
  a.div_mul = static_cast<uint32_t>(((uint64_t{1} << a.div_shift) + src_div - 1) / src_div);
  const bool bf16 = y_dtype == MOE_DTYPE_BF16;
  if (gated)
    bf16 ? launch_product<true, true>(a, s) : launch_product<true, false>(a, s);
  else
    bf16 ? launch_product<false, true>(a, s) : launch_product<false, false>(a, s);
  return hipGetLastError();
}

}  // namespace bitffn
