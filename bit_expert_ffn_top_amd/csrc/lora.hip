// Low-rank adapters of many requests beside a projection that they share:
//   y[t] = base[t] + scale[m] * B_m (A_m x[t]),   m the adapter of t's request
//
// Both products are on the matrix cores, with the adapter's rows as the first
// operand:
//   h = A x    16 or 32 consecutive rows of one request, or as many of one adapter
//              gathered from many requests; the eight wavefronts of a workgroup
//              split the columns, and their sums meet in LDS in a fixed order
//   y = B h    64 columns per wavefront
// Few rows: both in one launch.  A workgroup repeats h for its slice of y's
// columns; A is small (64 KB at rank 16 and 2048 columns), and a second launch
// would cost more.  Many rows: two launches, with h in the workspace in the order
// in which the second one's lanes read it.
// Operands are read as their rows lie and change lanes in LDS: read directly, an
// operand's layout has 16 bytes of each of 16 rows in a quarter of a wavefront,
// sixteen cache lines where four would do (8,192 rows at rank 64, two launches: 50 us
// where this took 28).  y leaves the same way.
// Measured (2,048 columns in and out, bfloat16): 8,192 rows of eight requests, rank
// 64, 101 MB of x, base and y: 12.3 + 16.7 us each launch alone, 27 in a graph of calls
// (as the variants below are compared), 20 at a copy's rate; what is left is each
// workgroup's chain of loads, LDS and products.  64 rows with an adapter each, rank 16,
// 1,536 columns out: 6.5 us, one fp32 row 7.1, that chain alone.
// fp32 values, x and h, enter as sums of three bfloat16 parts, exact but for the
// smallest values.  (With two parts of h for bfloat16 y the prompts above took 26
// instead of 27 us, but columns of B that cancel show what is lost.)  A row has the
// same bits whatever other rows there are.
#include <algorithm>

#include "moe_internal.h"
#include "row_device.h"
#include "scan_device.h"

namespace bitffn {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kGroup = 64;   // output columns that belong together

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
  int slice;     // output columns of a workgroup, a multiple of kGroup
  int together;  // rows of one adapter share a workgroup
  int4* tiles;   // in the workspace (many rows)
  int* lists;
  nu4* h;
  int n_tiles;
};

__device__ __forceinline__ nf4 mfma(nu4 a, nu4 b, nf4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b),
                                                 c, 0, 0, 0);
}

// Eight consecutive values of x, as they lie in LDS, or of h as bfloat16 parts.
template <typename T>
struct Parts;

template <>
struct Parts<uint16_t> {
  static constexpr int kParts = 1;
  static __device__ __forceinline__ void split(const nu4 (&v)[1], nu4 (&out)[1]) { out[0] = v[0]; }
};

// The high halves of two words.
__device__ __forceinline__ uint32_t high_halves(uint32_t lo, uint32_t hi) {
  return __builtin_amdgcn_perm(hi, lo, 0x07060302u);
}

template <>
struct Parts<float> {
  static constexpr int kParts = 3;
  // Each part takes the highest eight bits that are left: 24 in all.  An infinity is
  // whole in its first part and leaves nothing (a difference would be NaN); a NaN
  // whose high half is an infinity's leaves one.
  static __device__ __forceinline__ void split(const nu4 (&v)[2], nu4 (&out)[3]) {
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = v[i / 4][i % 4];
#pragma unroll
    for (int part = 0; part < 3; ++part) {
#pragma unroll
      for (int i = 0; i < 4; ++i) out[part][i] = high_halves(r[2 * i], r[2 * i + 1]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = __builtin_bit_cast(float, r[i]);
        const float left = v - __builtin_bit_cast(float, r[i] & 0xFFFF0000u);
        // what is left of a finite value is finite
        r[i] = __builtin_bit_cast(uint32_t, part == 0 && __builtin_isinf(v) ? 0.0f : left);
      }
    }
  }
};

// Rows [row0, row1) and request of one tile of `rows` rows; false if there are
// fewer tiles.  A request's rows end at the largest bound so far, clamped to the
// rows there are.  Every wavefront searches for itself, kPer bounds per lane.
template <int kPer>
__device__ __forceinline__ bool search_tile(const LoraArgs& g, int tile, int rows, int& row0, int& row1,
                                            int& request) {
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

__device__ __forceinline__ bool find_tile(const LoraArgs& g, int tile, int rows, int& row0, int& row1,
                                          int& request) {
  if (!g.seq) {
    row0 = request = tile;
    row1 = tile + 1;
    return tile < g.T;
  }
  return g.n_seq <= 64 ? search_tile<1>(g, tile, rows, row0, row1, request)
                       : search_tile<8>(g, tile, rows, row0, row1, request);
}

// The rows of a tile: row0 and those after it, or (LISTED) those that a list in
// LDS has, counted from row0.
template <bool LISTED>
struct Rows {
  int row0, n;
  const int* list;
  __device__ __forceinline__ int after(int i) const { return LISTED ? list[i] : i; }   // i < n
  // The same with the last one in place of those that are missing.
  __device__ __forceinline__ int held(int i) const { return after(min(i, n - 1)); }
  // The rows from the i-th on (there may be none).
  __device__ __forceinline__ Rows from(int i) const {
    return LISTED ? Rows{row0, n - i, list + i} : Rows{row0 + i, n - i, nullptr};
  }
};

// Tile `tile` of the requests' rows sorted by adapter, ROWS of one adapter (the
// last ones of each may be fewer; rows without one come last), found by the whole
// workgroup: it counts every adapter's rows in LDS, scans their tiles, and gathers
// the rows.  Each wavefront looks through an eighth of the requests.
template <int ROWS>
struct TogetherShared {
  int count[MOE_MAX_EXPERTS + 1];
  int wave[2][kWaves];
  int who, nth;    // the tile's adapter, and which of its tiles it is
  int list[ROWS];
};

// Requests of a wavefront whose adapters and bounds are asked for at a time; if it
// has no more, they are kept (8,192 rows that are requests, rank 64, 48 adapters, two
// launches: one at a time 48.3 us, four 44.9, eight 44.7, sixteen, then kept, 43.6; 512
// of them in one launch, with two 16.3 and with eight 17.6).
template <int BATCH>
struct Requests {
  int id[BATCH], bound[BATCH];
};

// f(bucket, first row, number of rows), one request per lane, for the requests
// [s0, s1), in order, until it is false; requests from s1 on have no rows.  low: the
// largest bound before s0.  kept: q has them.
template <int BATCH, typename F>
__device__ __forceinline__ void for_requests(const LoraArgs& g, Requests<BATCH>& q, bool kept, int s0, int s1,
                                             int low, F f) {
  const int lane = threadIdx.x & 63;
  for (int s = s0; s < s1; s += 64 * BATCH) {
    if (!kept) {
#pragma unroll
      for (int j = 0; j < BATCH; ++j) q.id[j] = g.adapter[min(s + 64 * j + lane, g.n_seq - 1)];
      if (g.seq) {
#pragma unroll
        for (int j = 0; j < BATCH; ++j) q.bound[j] = g.seq[min(s + 64 * j + lane, g.n_seq - 1) + 1];
      }
    }
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      const int r = s + 64 * j + lane;
      if (s + 64 * j >= s1) return;   // uniform
      int start = r, n = r < s1;
      if (g.seq) {
        const int upto = wave_scan_max(r < s1 ? min(max(q.bound[j], 0), g.T) : 0);
        start = max(low, lane_before(upto));
        n = max(low, upto) - start;
        low = max(low, lane_value(upto, 63));
      }
      if (!f(q.id[j] >= 0 && q.id[j] < g.n_adapters ? q.id[j] : g.n_adapters, start, n)) return;   // uniform
    }
  }
}

template <int ROWS, int BATCH = ROWS == 16 ? 2 : 16>
__device__ __forceinline__ bool find_together(const LoraArgs& g, int tile, TogetherShared<ROWS>& sh, int& m,
                                              int& rows) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int buckets = g.n_adapters + 1;
  for (int b = tid; b < buckets; b += kThreads) sh.count[b] = 0;
  if (tid == 0) sh.who = -1;
  const int part = ((g.n_seq + kWaves - 1) / kWaves + 63) / 64 * 64;   // requests of a wavefront
  const int s0 = min(g.n_seq, wave * part), s1 = min(g.n_seq, s0 + part);
  int low = 0;   // the largest bound before the wavefront's requests
  if (g.seq) {
    int top = 0;
    for (int s = s0 + lane; s < s1; s += 64) top = max(top, min(max(g.seq[s + 1], 0), g.T));
    top = lane_value(wave_scan_max(top), 63);
    if (lane == 0) sh.wave[0][wave] = top;
    low = min(max(g.seq[0], 0), g.T);
  }
  __syncthreads();
  if (g.seq)
    for (int w = 0; w < wave; ++w) low = max(low, sh.wave[0][w]);
  Requests<BATCH> q;
  const bool keep = part <= 64 * BATCH;
  for_requests(g, q, false, s0, s1, low, [&](int b, int, int n) {
    if (n > 0) atomicAdd(&sh.count[b], n);
    return true;
  });
  __syncthreads();
  constexpr int kPer = (MOE_MAX_EXPERTS + kThreads) / kThreads;   // buckets of a thread
  int tiles[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * kPer + i;
    tiles[i] = b < buckets ? (sh.count[b] + ROWS - 1) / ROWS : 0;
    sum += tiles[i];
  }
  const int scan = wave_scan_add(sum);
  if (lane == 63) sh.wave[1][wave] = scan;
  __syncthreads();
  int left = tile - (scan - sum);
  for (int w = 0; w < wave; ++w) left -= sh.wave[1][w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (left >= 0 && left < tiles[i]) {
      sh.who = tid * kPer + i;
      sh.nth = left;
    }
    left -= tiles[i];
  }
  __syncthreads();
  const int who = sh.who;
  if (who < 0) return false;   // uniform
  int mine = 0;
  for_requests(g, q, keep, s0, s1, low, [&](int b, int, int n) {
    mine += b == who ? n : 0;
    return true;
  });
  mine = lane_value(wave_scan_add(mine), 63);
  if (lane == 0) sh.wave[0][wave] = mine;   // last read before two barriers
  __syncthreads();
  int at = -ROWS * sh.nth;   // place of the next row found among the tile's
  for (int w = 0; w < wave; ++w) at += sh.wave[0][w];
  for_requests(g, q, keep, s0, s1, low, [&](int b, int start, int n) {
    if (b != who) n = 0;
    const int end = at + wave_scan_add(n), first = end - n;
    for (int place = max(first, 0); place < min(end, ROWS); ++place) sh.list[place] = start + place - first;
    at = lane_value(end, 63);
    return at < ROWS;
  });
  rows = min(ROWS, sh.count[who] - ROWS * sh.nth);
  __syncthreads();
  m = who < g.n_adapters ? who : -1;
  return true;
}

// Rows of a tile without an adapter: columns [n0, n1) of base, by a workgroup or a
// wavefront.
template <typename YT, bool LISTED>
__device__ __forceinline__ void copy_base(const LoraArgs& g, const Rows<LISTED>& rows, int n0, int n1, int threads) {
  const YT* base = static_cast<const YT*>(g.base);
  YT* y = static_cast<YT*>(g.y);
  if (y == base) return;
  const int parts = (n1 - n0) / 8;
  for (int i = threadIdx.x % threads; i < rows.n * parts; i += threads) {
    const int t = i / parts;
    const int64_t at = static_cast<int64_t>(rows.row0 + rows.after(t)) * g.d_out + n0 + 8 * (i - t * parts);
    RowPart<YT, 8> v;
    v.load(base + at);
    v.store(y + at);
  }
}

// 16 rows of 128 bytes of a matrix: a lane holds chunk lane % 8 (16 bytes) of rows
// lane / 8 and lane / 8 + 8.  In LDS a row's chunks are exchanged by its number, so
// that eight lanes that read one chunk of eight rows meet no bank twice.
constexpr int kUnitBytes = 2048;

struct UnitRows {
  uint32_t at[2];   // the lane's rows and chunk, bytes from the matrix's start
  template <bool LISTED>
  __device__ __forceinline__ void set(const Rows<LISTED>& rows, int row, uint32_t row_bytes) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int h = 0; h < 2; ++h) at[h] = rows.held(row + (lane >> 3) + 8 * h) * row_bytes + 16 * (lane & 7);
  }
};

// Order between the LDS accesses of one wavefront's lanes, which take effect as
// they are issued: for the compiler only.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ void put_unit(char* lds, const nu4 (&v)[2]) {
  const int lane = threadIdx.x & 63, row = lane >> 3;
#pragma unroll
  for (int h = 0; h < 2; ++h)   // rows 8 apart have one exchange
    *reinterpret_cast<nu4*>(lds + 128 * (row + 8 * h) + 16 * ((lane & 7) ^ row)) = v[h];
}

__device__ __forceinline__ nu4 get_chunk(const char* lds, int row, int chunk) {
  return *reinterpret_cast<const nu4*>(lds + 128 * row + 16 * (chunk ^ (row & 7)));
}

// Shared memory of one wavefront, in its three uses: x, then A, then the sums (A beside
// x would leave fp32 one workgroup per CU: 8,192 rows that are requests, rank 16, 48
// adapters, 305 workgroups, 76 us instead of 58).
template <typename XT, int MT, int NT>
struct Down {
  static constexpr int kUnits = sizeof(XT) / 2;   // of x, for 64 columns
  static constexpr int kRanks = MT < 4 ? MT : 4;  // 16-rank tiles of a pass
  static constexpr int kPartRow = 16 * kRanks + 4;
  static constexpr int kStage = std::max(NT * kUnits, 2) * kUnitBytes;
  static constexpr int kPart = 16 * NT * kPartRow * 4;
  static constexpr int kBytes = kStage > kPart ? kStage : kPart;
  // 64-column units asked for at a time
  static constexpr int kAhead = kRanks * NT <= 1 ? 4 : kRanks * NT <= 2 ? 2 : 1;
};

// A wavefront's share of h = A x for 16 NT rows and the ranks from 64 pass on,
// left in its part of LDS: [row][rank].
template <typename XT, int MT, int NT, bool LISTED>
__device__ __forceinline__ void down_product(const LoraArgs& g, int m, const Rows<LISTED>& rows, int pass,
                                             char* lds) {
  using D = Down<XT, MT, NT>;
  constexpr int MP = D::kRanks, XU = D::kUnits, XP = Parts<XT>::kParts, U = D::kAhead;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, quad = lane >> 4;
  const char* a = reinterpret_cast<const char*>(g.a + static_cast<int64_t>(m) * g.rank * g.d_in);
  const char* x = reinterpret_cast<const char*>(static_cast<const XT*>(g.x) + static_cast<int64_t>(rows.row0) * g.d_in);
  UnitRows ar[MP], xr[NT];
#pragma unroll
  for (int i = 0; i < MP; ++i) ar[i].set(Rows<false>{0, g.rank, nullptr}, 64 * pass + 16 * i, g.d_in * 2);
#pragma unroll
  for (int j = 0; j < NT; ++j) xr[j].set(rows, 16 * j, g.d_in * sizeof(XT));
  nf4 acc[MP][NT];
#pragma unroll
  for (int i = 0; i < MP; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = nf4{0.0f, 0.0f, 0.0f, 0.0f};
  const int units = (g.d_in + 63) / 64;
  for (int u0 = wave; u0 < units; u0 += kWaves * U) {
    nu4 av[U][MP][2], xv[U][NT][XU][2];
#pragma unroll
    for (int n = 0; n < U; ++n) {
      const int u = min(u0 + kWaves * n, units - 1);
      // the last unit of bfloat16 rows may end after 32 columns
      const uint32_t c = 128 * u, back = c + 16 * (lane & 7) >= static_cast<uint32_t>(g.d_in) * 2 ? 64 : 0;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int w = 0; w < XU; ++w)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t cx = XU == 1 ? c - back : min(256 * u + 128 * w, g.d_in * 4 - 128);
            xv[n][j][w][h] = *reinterpret_cast<const nu4*>(x + (xr[j].at[h] + cx));
          }
#pragma unroll
      for (int i = 0; i < MP; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) av[n][i][h] = *reinterpret_cast<const nu4*>(a + (ar[i].at[h] + (c - back)));
    }
#pragma unroll
    for (int n = 0; n < U; ++n) {
      const int u = u0 + kWaves * n;
      if (u >= units) break;   // uniform
      wave_order();
      const bool whole = 64 * u + 32 < g.d_in;
      nu4 xp[2][NT][XP];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int w = 0; w < XU; ++w) put_unit(lds + (j * XU + w) * kUnitBytes, xv[n][j][w]);
        wave_order();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          nu4 v[XU];
#pragma unroll
          for (int w = 0; w < XU; ++w)
            v[w] = XU == 1 ? get_chunk(lds + j * kUnitBytes, l16, 4 * s + quad)
                           : get_chunk(lds + (j * XU + s) * kUnitBytes, l16, 2 * quad + w);
          Parts<XT>::split(v, xp[s][j]);
        }
      }
#pragma unroll
      for (int i = 0; i < MP; ++i) {
        char* at = lds + (i & 1) * kUnitBytes;   // x has been read
        wave_order();
        put_unit(at, av[n][i]);
        wave_order();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (s == 1 && !whole) break;   // uniform
          const nu4 af = get_chunk(at, l16, 4 * s + quad);
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int p = 0; p < XP; ++p) acc[i][j] = mfma(af, xp[s][j][p], acc[i][j]);
        }
      }
    }
  }
  wave_order();
  float* part = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int i = 0; i < MP; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
      *reinterpret_cast<nf4*>(part + (16 * j + l16) * D::kPartRow + 16 * i + 4 * quad) = acc[i][j];
}

constexpr int kHParts = Parts<float>::kParts;

// Eight ranks (64 pass + 32 step + 8 quad ..) of token t: the wavefronts' sums in
// order, scaled; zeros past the adapter's rank.
template <typename D, int STRIDE>   // STRIDE: from one wavefront's sums to the next one's
__device__ __forceinline__ void join_sums(const char* lds, int t, int r, int ranks, float scale,
                                          nu4 (&out)[2]) {
  float h[8];
  if (r < ranks) {
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float* part = reinterpret_cast<const float*>(lds + w * STRIDE) + t * D::kPartRow + r;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] += part[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] *= scale;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = 0.0f;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) out[e / 4][e % 4] = __builtin_bit_cast(uint32_t, h[e]);
}

// Rows c .. c + COLS - 1 of B, which follow each other in memory, 16 bytes per
// lane and load; in LDS a row has an odd number of chunks, so that eight lanes that
// read one chunk of eight rows meet no bank twice.
template <int RS, int COLS, int THREADS>
struct BRows {
  static constexpr int kLoads = (COLS * 4 * RS + THREADS - 1) / THREADS;   // at the largest rank
  static constexpr int kBytes = COLS * (4 * RS + 1) * 16;
  nu4 v[kLoads];
  __device__ __forceinline__ void load(const LoraArgs& g, const uint16_t* b, int c, int thread) {
    const int chunks = min(COLS, g.d_out - c) * (g.rank / 8);
    const nu4* src = reinterpret_cast<const nu4*>(b + static_cast<int64_t>(c) * g.rank);
#pragma unroll
    for (int n = 0; n < kLoads; ++n)
      if (n * THREADS < chunks) v[n] = src[min(n * THREADS + thread, chunks - 1)];   // uniform
  }
  __device__ __forceinline__ void put(const LoraArgs& g, int c, char* lds, int thread) const {
    const int per = g.rank / 8, chunks = min(COLS, g.d_out - c) * per;
    const uint32_t over = (65535u + per) / per;   // i / per = i * over >> 16 for i * per < 2^16
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      const int i = n * THREADS + thread;
      if (i < chunks) {
        const int row = i * over >> 16;
        *reinterpret_cast<nu4*>(lds + 16 * (row * (per | 1) + (i - row * per))) = v[n];
      }
    }
  }
  // Lane's chunk of row `row`: ranks 32 s + 8 quad .., zeros past the adapter's.
  static __device__ __forceinline__ nu4 get(const LoraArgs& g, const char* lds, int row, int s) {
    const int per = g.rank / 8, chunk = 4 * s + ((threadIdx.x & 63) >> 4);
    const nu4 b = *reinterpret_cast<const nu4*>(lds + 16 * (row * (per | 1) + min(chunk, per - 1)));
    return chunk < per ? b : nu4{0, 0, 0, 0};
  }
};

// A wavefront's 16 rows of COLS columns of base and y as they lie: a lane holds kN
// columns of each of kLoads rows.  Eight fp32 columns are two stores that leave gaps,
// and 7% of what they write goes out twice: 8,192 rows of eight prompts, rank 64, with
// eight and four 53.2 and 50.8 us.  Few rows are better off with eight (one row 6.69
// against 6.75 us, 512 rows, rank 64, 14.0 against 14.2).
template <typename YT, int COLS, int kN>
struct YRows {
  static constexpr int kPerRow = COLS / kN, kRows = 64 / kPerRow, kLoads = 16 / kRows;
  RowPart<YT, kN> v[kLoads];
  // Rows and columns past the end re-read the last ones: no load depends on a
  // comparison, so that waiting for one need not be waiting for all.  ALL: the list
  // has 16 rows, whatever their number.
  template <bool ALL = false, bool LISTED>
  __device__ __forceinline__ void load(const LoraArgs& g, const Rows<LISTED>& rows, int c) {
    const int lane = threadIdx.x & 63, col = min(c + kN * (lane % kPerRow), g.d_out - kN);
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      const int i = n * kRows + lane / kPerRow;
      const int t = max(rows.row0 + (ALL ? rows.after(i) : rows.held(i)), 0);
      v[n].load(static_cast<const YT*>(g.base) + static_cast<int64_t>(t) * g.d_out + col);
    }
  }
  // v = base + the results in LDS, [row][COLS + 4]
  __device__ __forceinline__ void add(const float* lds) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      const nf4* d = reinterpret_cast<const nf4*>(lds + (n * kRows + lane / kPerRow) * (COLS + 4) +
                                                  kN * (lane % kPerRow));
      nf4 r[kN / 4];
#pragma unroll
      for (int e = 0; e < kN / 4; ++e) r[e] = d[e];
      float f[kN];
#pragma unroll
      for (int e = 0; e < kN; ++e) f[e] = v[n].get(e) + r[e / 4][e % 4];
      v[n].set(f);
    }
  }
  template <bool LISTED>
  __device__ __forceinline__ void store(const LoraArgs& g, const Rows<LISTED>& rows, int c) const {
    const int lane = threadIdx.x & 63, col = c + kN * (lane % kPerRow);
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      const int t = n * kRows + lane / kPerRow;
      if (t < rows.n && col < g.d_out)
        v[n].template store<true>(static_cast<YT*>(g.y) + static_cast<int64_t>(rows.row0 + rows.after(t)) * g.d_out +
                                  col);
    }
  }
};

// B h of 16 columns per row tile of B and 16 tokens, to LDS [token][COLS + 4].
template <int RS, int COLS>
__device__ __forceinline__ void up_product(const nu4 (&bv)[RS], const nu4 (&hv)[kHParts][RS], float* lds, int tile) {
  const int lane = threadIdx.x & 63;
  nf4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int s = 0; s < RS; ++s)
#pragma unroll
    for (int p = 0; p < kHParts; ++p) acc = mfma(bv[s], hv[p][s], acc);
  *reinterpret_cast<nf4*>(lds + (lane & 15) * (COLS + 4) + 16 * tile + 4 * (lane >> 4)) = acc;
}

__device__ __forceinline__ int adapter_of(const LoraArgs& g, int request) {
  return __builtin_amdgcn_readfirstlane(g.adapter[request]);
}

// The rows and adapter (-1: none) of a tile, of one request.
template <int ROWS, bool LISTED>
__device__ __forceinline__ bool tile_rows(const LoraArgs& g, int tile, Rows<LISTED>& rows, int& m) {
  int row1, request;
  if (!find_tile(g, tile, ROWS, rows.row0, row1, request)) return false;
  rows.n = row1 - rows.row0;
  m = adapter_of(g, request);
  if (m >= g.n_adapters) m = -1;
  return true;
}

// The same of gathered rows.
template <int ROWS>
__device__ __forceinline__ bool tile_rows(const LoraArgs& g, int tile, TogetherShared<ROWS>& sh, Rows<true>& rows,
                                          int& m) {
  rows.list = sh.list;
  if (!find_together<ROWS>(g, tile, sh, m, rows.n)) return false;
  m = __builtin_amdgcn_readfirstlane(m);
  return true;
}

// Few rows, one launch.  MT: 16-rank tiles (rank <= 16 MT).
template <typename XT, typename YT, int MT>
__global__ __launch_bounds__(kThreads) void lora_kernel(LoraArgs g) {
  using D = Down<XT, MT, 1>;
  constexpr int RS = (MT + 1) / 2;   // 32-rank steps of the second product
  constexpr int kCols = 32;          // columns that a wavefront takes at a time
  using B = BRows<RS, kCols, 64>;
  constexpr int kUp = B::kBytes + 16 * (kCols + 4) * 4;
  constexpr int kWaveBytes = D::kBytes > kUp ? D::kBytes : kUp;
  static_assert(kWaveBytes % 16 == 0, "");
  __shared__ __align__(16) char s_wave[kWaves * kWaveBytes];
  __shared__ nu4 s_h[kHParts][RS][64];
  __shared__ TogetherShared<16> s_rows;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  Rows<true> rows{0, 0, s_rows.list};
  int m = -1;
  if (g.together) {
    if (!tile_rows(g, blockIdx.x, s_rows, rows, m)) return;
  } else {
    if (!tile_rows<16>(g, blockIdx.x, rows, m)) return;
    if (tid < 16) s_rows.list[tid] = tid;
    __syncthreads();
  }
  const int n0 = blockIdx.y * g.slice, n1 = min(g.d_out, n0 + g.slice);
  if (m < 0) {
    copy_base<YT>(g, rows, n0, n1, kThreads);
    return;
  }
  const float scale = g.scale ? g.scale[m] : 1.0f;
  char* mine = s_wave + wave * kWaveBytes;
  const uint16_t* b = g.b + static_cast<int64_t>(m) * g.d_out * g.rank;
  const int blocks = (n1 - n0 + kCols - 1) / kCols, per = (blocks + kWaves - 1) / kWaves;
  const int k0 = min(blocks, wave * per), k1 = min(blocks, k0 + per);
  // the first block's rows of B and base are on their way meanwhile
  B bl;
  YRows<YT, kCols, 8> yr;
  if (k0 < k1) {
    bl.load(g, b, n0 + k0 * kCols, lane);
    yr.load(g, rows, n0 + k0 * kCols);
  }
  for (int pass = 0; pass < MT / D::kRanks; ++pass) {
    down_product<XT, MT, 1>(g, m, rows, pass, mine);
    __syncthreads();
    constexpr int kSteps = (D::kRanks + 1) / 2;
    if (tid < 64 * kSteps) {
      const int r = 32 * wave + 8 * (lane >> 4);
      nu4 v[2], h[kHParts];
      join_sums<D, kWaveBytes>(s_wave, lane & 15, r, min(g.rank - 64 * pass, 16 * D::kRanks), scale, v);
      Parts<float>::split(v, h);
#pragma unroll
      for (int p = 0; p < kHParts; ++p) s_h[p][2 * pass + wave][lane] = h[p];
    }
    __syncthreads();
  }
  nu4 hv[kHParts][RS];
#pragma unroll
  for (int p = 0; p < kHParts; ++p)
#pragma unroll
    for (int s = 0; s < RS; ++s) hv[p][s] = s_h[p][s][lane];
  float* res = reinterpret_cast<float*>(mine + B::kBytes);
  for (int k = k0; k < k1; ++k) {
    const int c = n0 + k * kCols;
    wave_order();
    bl.put(g, c, mine, lane);
    wave_order();
    if (k + 1 < k1) bl.load(g, b, c + kCols, lane);
#pragma unroll
    for (int tile = 0; tile < kCols / 16; ++tile) {
      nu4 bv[RS];
#pragma unroll
      for (int s = 0; s < RS; ++s) bv[s] = B::get(g, mine, 16 * tile + (lane & 15), s);
      up_product<RS, kCols>(bv, hv, res, tile);
    }
    wave_order();
    yr.add(res);
    yr.store(g, rows, c);
    if (k + 1 < k1) yr.load(g, rows, c + kCols);
  }
}

// Many rows, two launches.  The workspace holds a table of the first one's tiles
// (first row, number of rows, adapter or -1) and, where they are gathered, their rows,
// which spares the second one the search, and h by 16 rows in the order of the second
// product's operand, in fp32, which is less to read than its parts: [tile][16 rows]
// [half][step][lane][4].
constexpr int kTileRows = 32;
constexpr int kTiles16 = kTileRows / 16;
constexpr int kUpWaves = 2;    // tiles of a workgroup
constexpr int kUpGridRows = 32768;

// Workgroups go to the eight XCDs in turn: four tiles that follow each other, which
// mostly share an adapter, go to one, whose L2 cache then reads it once (8,192 rows,
// rank 64, two launches, with 1, 4, 8 and all n / 8 tiles: eight prompts 28.2, 27.4,
// 28.3 and 29.7 us; single rows, 48 adapters, 48.2, 44.2, 43.1 and 47.7, 4 adapters
// 33.8, 33.9, 34.3 and 34.2).
__device__ __forceinline__ int tile_of(int block, int n) {
  constexpr int kRun = 4, kTurn = 8 * kRun;
  const int i = block % kTurn, first = block - i;
  return first + kTurn <= n ? first + i % 8 * kRun + i / 8 : block;
}

template <typename XT, int MT, bool LISTED>
__global__ __launch_bounds__(kThreads) void lora_down_kernel(LoraArgs g) {
  using D = Down<XT, MT, kTiles16>;
  constexpr int RS = (MT + 1) / 2;
  __shared__ __align__(16) char s_wave[kWaves * D::kBytes];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tile = tile_of(blockIdx.x, gridDim.x);
  Rows<LISTED> rows{0, 0, nullptr};
  int m = -1;
  if constexpr (LISTED) {
    __shared__ TogetherShared<kTileRows> s_rows;
    const bool found = tile_rows(g, tile, s_rows, rows, m);
    if (tid < kTileRows)   // rows past the end re-read the last one
      g.lists[tile * kTileRows + tid] = found ? rows.held(tid) : 0;
  } else {
    tile_rows<kTileRows>(g, tile, rows, m);
  }
  if (tid == 0) g.tiles[tile] = make_int4(rows.row0, rows.n, m, 0);
  if (m < 0) return;
  const float scale = g.scale ? g.scale[m] : 1.0f;
  for (int pass = 0; pass < MT / D::kRanks; ++pass) {
    if (pass) __syncthreads();   // the sums have been read
    down_product<XT, MT, kTiles16>(g, m, rows, pass, s_wave + wave * D::kBytes);
    __syncthreads();
    constexpr int kSteps = (D::kRanks + 1) / 2;
    if (wave < kSteps * kTiles16) {
      const int part16 = wave / kSteps, step = wave - part16 * kSteps;
      nu4 h[2];
      join_sums<D, D::kBytes>(s_wave, 16 * part16 + (lane & 15), 32 * step + 8 * (lane >> 4),
                                  min(g.rank - 64 * pass, 16 * D::kRanks), scale, h);
      nu4* out = g.h + (static_cast<int64_t>(tile) * kTiles16 + part16) * (2 * RS * 64) + lane;
#pragma unroll
      for (int p = 0; p < 2; ++p) out[(p * RS + 2 * pass + step) * 64] = h[p];
    }
  }
}

// A workgroup takes 64 columns of two tiles, one per wavefront (8,192 rows, rank 64,
// with one, two, three, four and eight tiles: 28.0, 27.6, 27.1, 27.3 and 34.3 us for
// both launches; single rows of 48 adapters 44.7, 44.0, 43.5, 44.3 and 50.2).  B goes through LDS for all of them, adapter by adapter where the
// tiles' requests have different ones.
template <typename YT, int RS, bool LISTED>
__global__ __launch_bounds__(64 * kUpWaves) void lora_up_kernel(LoraArgs g) {
  using B = BRows<RS, kGroup, 64 * kUpWaves>;
  __shared__ __align__(16) char s_b[B::kBytes];
  __shared__ __align__(16) float s_res[kUpWaves][16 * (kGroup + 4)];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // neighbouring workgroups take neighbouring columns of the same rows
  const int c = blockIdx.x * kGroup, tile0 = (blockIdx.z * kUpGridRows + blockIdx.y) * kUpWaves;
  const int tile = tile0 + wave;
  const int4 mine = tile < g.n_tiles ? g.tiles[tile] : make_int4(0, 0, -1, 0);
  const Rows<LISTED> rows{mine.x, mine.y, LISTED ? g.lists + min(tile, g.n_tiles - 1) * kTileRows : nullptr};
  const int m = mine.z;
  int all[kUpWaves];   // the tiles' adapters
#pragma unroll
  for (int w = 0; w < kUpWaves; ++w) {
    const int t = tile0 + w;
    all[w] = t < g.n_tiles ? g.tiles[t].z : -1;
  }
  int who = -1;
#pragma unroll
  for (int w = kUpWaves - 1; w >= 0; --w) who = all[w] >= 0 ? all[w] : who;
  if (who < 0) {   // no adapter in any of the tiles (uniform)
    copy_base<YT>(g, rows, c, min(g.d_out, c + kGroup), 64);
    return;
  }
  // Loads arrive in the order in which they are asked for: B, which all wait for
  // first, from the L2 cache, then h (whatever is there, for a tile without an
  // adapter), then base, which the results are added to.
  const auto rows_of_b = [&](int adapter) { return g.b + static_cast<int64_t>(adapter) * g.d_out * g.rank; };
  B bl;
  bl.load(g, rows_of_b(who), c, tid);
  nu4 hv[kTiles16][RS][2];
  const nu4* h = g.h + static_cast<int64_t>(min(tile, g.n_tiles - 1)) * kTiles16 * (2 * RS * 64) + lane;
#pragma unroll
  for (int j = 0; j < kTiles16; ++j)
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int s = 0; s < RS; ++s) hv[j][s][p] = h[((j * 2 + p) * RS + s) * 64];
  YRows<YT, kGroup, 16 / sizeof(YT)> yr[kTiles16];
#pragma unroll
  for (int j = 0; j < kTiles16; ++j) yr[j].template load<LISTED>(g, rows.from(16 * j), c);
  bool first = true;
  for (int w = 0; w < kUpWaves; ++w) {
    who = all[w];
    bool again = who < 0;
    for (int v = 0; v < w; ++v) again |= all[v] == who;
    if (again) continue;   // uniform
    if (!first) {
      bl.load(g, rows_of_b(who), c, tid);
      __syncthreads();   // the last adapter's rows have been read
    }
    first = false;
    bl.put(g, c, s_b, tid);
    __syncthreads();
    if (m != who) continue;
#pragma unroll
    for (int j = 0; j < kTiles16; ++j) {
      nu4 hp[kHParts][RS];
#pragma unroll
      for (int s = 0; s < RS; ++s) {
        nu4 v[kHParts];
        Parts<float>::split(hv[j][s], v);
#pragma unroll
        for (int p = 0; p < kHParts; ++p) hp[p][s] = v[p];
      }
#pragma unroll
      for (int t = 0; t < kGroup / 16; ++t) {
        nu4 bv[RS];
#pragma unroll
        for (int s = 0; s < RS; ++s) bv[s] = B::get(g, s_b, 16 * t + (lane & 15), s);
        up_product<RS, kGroup>(bv, hp, s_res[wave], t);
      }
      wave_order();
      yr[j].add(s_res[wave]);
      wave_order();
    }
  }
  if (m >= 0 || g.y != g.base) {   // without an adapter: base as it is
#pragma unroll
    for (int j = 0; j < kTiles16; ++j) yr[j].store(g, rows.from(16 * j), c);
  }
}

// ceil(n / rows) summed over the requests is at most this.
int most_tiles(int64_t T, int n_seq, int rows) {
  return static_cast<int>((T + (rows - 1) * std::min(static_cast<int64_t>(n_seq), T)) / rows);
}

template <typename XT, typename YT, int MT>
hipError_t launch_rank(LoraArgs g, hipStream_t s) {
  const int groups = (g.d_out + kGroup - 1) / kGroup;
  if (g.h) {
    const int rows = (g.n_tiles + kUpWaves - 1) / kUpWaves;
    const dim3 grid(groups, min(rows, kUpGridRows), (rows + kUpGridRows - 1) / kUpGridRows);
    if (g.together) {
      lora_down_kernel<XT, MT, true><<<g.n_tiles, kThreads, 0, s>>>(g);
      lora_up_kernel<YT, (MT + 1) / 2, true><<<grid, 64 * kUpWaves, 0, s>>>(g);
    } else {
      lora_down_kernel<XT, MT, false><<<g.n_tiles, kThreads, 0, s>>>(g);
      lora_up_kernel<YT, (MT + 1) / 2, false><<<grid, 64 * kUpWaves, 0, s>>>(g);
    }
    return hipGetLastError();
  }
  // about a workgroup per CU: slices of the columns while there are few tiles (one
  // row, 1,536 columns in 3 slices 7.6 us, in 24 6.7; 64 rows in 3 6.2, in 24 14.8)
  const int64_t tiles = g.together ? most_tiles(g.T, g.n_adapters + 1, 16)
                                   : g.seq ? most_tiles(g.T, g.n_seq, 16) : g.T;
  const int slices = static_cast<int>(std::max(int64_t{1}, std::min(int64_t{groups}, 256 / tiles)));
  g.slice = (groups + slices - 1) / slices * kGroup;
  const dim3 grid(static_cast<unsigned>(tiles), (g.d_out + g.slice - 1) / g.slice);
  lora_kernel<XT, YT, MT><<<grid, kThreads, 0, s>>>(g);
  return hipGetLastError();
}

template <typename XT, typename YT>
hipError_t launch_as(const LoraArgs& g, hipStream_t s) {
  if (g.rank <= 16) return launch_rank<XT, YT, 1>(g, s);
  if (g.rank <= 32) return launch_rank<XT, YT, 2>(g, s);
  if (g.rank <= 64) return launch_rank<XT, YT, 4>(g, s);
  return launch_rank<XT, YT, 8>(g, s);
}

// Rows from which two launches are made (eight requests, bfloat16, one launch against
// two: 2,048 columns, 2,048 rows at rank 16 14.1 against 12.0 us, at rank 64 19.4
// against 16.7; 1,024 rows 9.5 against 10.6 and 13.1 against 15.3, but with 4,096
// columns 14.7 against 13.7 and 21.7 against 20.4: the border lies between, the lower
// the longer the rows).
constexpr int64_t kManyRows = 1024;

// The same for gathered rows (one launch against two, bfloat16, rank 64, 48 adapters:
// a row for every request, 1,024 rows 19.1 against 19.3 us, with 4 adapters 14.4
// against 17.4; 2,048 rows 24.7 against 22.5; 8,192 rows 63 against 44; 1,000 requests
// of two rows 25.5 against 22.3; 512 single rows beside a prompt of 8,192 44 against 40).
constexpr int64_t kManyGathered = 1536;

// Requests beyond the number of adapters from which rows of one adapter share a
// workgroup: that many tiles at least are spared, for some 2 us of gathering (a row
// for every request, apart against together, bfloat16, rank 64, 4 and 48 adapters:
// 64 rows 10.5 against 10.3 and 11.3 against 15.4 us, 128 rows 13.0 against 9.4 and
// 14.4 against 15.4, 512 rows 23.1 against 13.0 and 31.0 against 16.2, 8,192 rows
// 274 against 34 and 438 against 44; where rows fill their tiles anyhow, 8,000 rows
// of 256 requests, 45 against 39, in fp32 59 against 60).
constexpr int kTogether = 64;

// Their offsets into x have 32 bits.
bool gathers(int64_t T, int n_seq, int n_adapters, int64_t row_bytes) {
  return n_seq >= n_adapters + kTogether && T * row_bytes < (int64_t{1} << 32) - (1 << 17);
}

}  // namespace

// n_seq = 0: a row for every request; then there are two launches only with gathered
// rows, of at most MOE_MAX_EXPERTS adapters and those without one.
size_t lora_workspace_bytes(int64_t T, int rank, int n_seq) {
  if (T < kManyRows || (n_seq == 0 && T > 65536)) return 0;
  const int64_t tiles = most_tiles(T, n_seq ? n_seq : MOE_MAX_EXPERTS + 1, kTileRows);
  const int64_t steps = rank <= 32 ? 1 : rank <= 64 ? 2 : 4;
  return static_cast<size_t>(align256(tiles * 16) + tiles * kTileRows * 4 + tiles * kTiles16 * 2 * steps * 1024);
}

hipError_t launch_lora(const void* base, const void* x, int x_dtype, int64_t T, int d_in, int d_out,
                       const uint16_t* a, const uint16_t* b, int n_adapters, int rank,
                       const int32_t* seq, int n_seq, const int32_t* adapter, const float* scale,
                       void* y, int y_dtype, void* ws, hipStream_t s) {
  LoraArgs g{base, x, a, b, seq, adapter, scale, y, static_cast<int>(T),
             d_in, d_out, n_adapters, rank, n_seq, 0, 0, nullptr, nullptr, nullptr, 0};
  g.together = gathers(T, n_seq, n_adapters, int64_t{d_in} * (x_dtype == MOE_DTYPE_F32 ? 4 : 2));
  if (g.together ? T >= kManyGathered : seq && T >= kManyRows) {
    g.n_tiles = most_tiles(T, g.together ? n_adapters + 1 : n_seq, kTileRows);
    char* at = static_cast<char*>(ws);
    g.tiles = reinterpret_cast<int4*>(at);
    at += align256(int64_t{g.n_tiles} * 16);
    g.lists = reinterpret_cast<int*>(at);
    g.h = reinterpret_cast<nu4*>(at + int64_t{g.n_tiles} * kTileRows * 4);
  }
  const bool xf = x_dtype == MOE_DTYPE_F32, yf = y_dtype == MOE_DTYPE_F32;
  const auto f = xf ? (yf ? launch_as<float, float> : launch_as<float, uint16_t>)
                    : (yf ? launch_as<uint16_t, float> : launch_as<uint16_t, uint16_t>);
  return f(g, s);
}

}  // namespace bitffn
