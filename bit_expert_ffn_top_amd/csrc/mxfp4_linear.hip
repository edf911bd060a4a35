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
  // the same in every thread: kept in scalar registers
  return RowTile{__builtin_amdgcn_readfirstlane(s_g), __builtin_amdgcn_readfirstlane(s_rows),
                 __builtin_amdgcn_readfirstlane(s_r0)};
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

// Four consecutive output columns of a row, stored at p.  GATED: the columns
// are (gate, up, gate, up) and two values are stored.
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
    const int64_t s = source_row(a, t.r0 + min(local, t.rows - 1), ok[m]);   // widened: offsets may pass 2^32
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
    if (local < t.rows) {
      const int col = n0 + 4 * q;
      const int64_t at = (t.r0 + local) * (GATED ? a.N / 2 : a.N) + (GATED ? col / 2 : col);
      store_out<GATED, BF16>(static_cast<uint8_t*>(a.y) + at * (BF16 ? 2 : 4),
                             ok[m] ? acc[m] : mf4{0, 0, 0, 0});
    }
  }
}

// Many rows per group.  A workgroup takes MG_ROWS weight rows and up to 16 CAP
// tokens of one group; each of its four wavefronts owns 32 of the weight rows
// (two MFMA tiles) for all the tokens, so every weight is read from memory
// straight into the registers of the one wavefront that uses it, three steps
// ahead.  The tokens' codes are shared: a step's 256 columns (128 bytes of each
// row) go to LDS by the loads that write it directly, two steps ahead, 16-byte
// piece p of row r at position p ^ swz(r), which spreads the 16 rows that a read
// of one piece touches over all banks.  Their scales, 8 bytes of a row per
// step, pass through registers.  Token tiles past a short group's rows are
// skipped.
constexpr int MG_ROWS = 128;
constexpr int MG_STEP = 256;             // columns per step
constexpr uint32_t MG_OUT = 0x80000000u; // an offset outside every buffer: reads zeros, no traffic

typedef __amdgpu_buffer_rsrc_t MgRsrc;
typedef __attribute__((address_space(3))) uint8_t LdsByte;

__host__ __device__ constexpr int mg_swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

__device__ __forceinline__ MgRsrc mg_rsrc(const uint8_t* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0,
                                           static_cast<int>(static_cast<uint32_t>(bytes)), 0x00020000);
}

// A wavefront's weights of one step: [tile][half of the lane's 64 columns].
// EVEN (rows are a whole number of steps): both halves' scale bytes in s[t][0].
struct MgWeights {
  mi4 c[2][2];
  uint16_t s[2][2];
};

// Eight scale bytes of a token's row, EVEN: in v[0] and v[1].
struct MgScales {
  uint32_t v[8];
};

// Buffers (a read past one gives zeros) and this lane's byte offsets in them.
struct MgLane {
  MgRsrc ac, as, wc, ws;
  uint32_t av[8];        // A codes: the row pieces this lane moves to LDS
  uint32_t asv;          // A scales: the row this thread carries
  uint32_t wv, wsv;      // weights and scales: this lane's row of the first tile
  int wtile, wstile;     // from the first tile to the second
  int nb, q, steps;
};

// Memory instructions of a step's loads.
template <bool EVEN>
constexpr int mg_w_loads() { return EVEN ? 6 : 8; }
template <bool EVEN>
constexpr int mg_s_loads() { return EVEN ? 1 : 8; }

template <bool EVEN>
__device__ __forceinline__ void mg_load_w(MgWeights& w, const MgLane& l, int c) {
  const uint32_t wv = c < l.steps ? l.wv : MG_OUT, wsv = c < l.steps ? l.wsv : MG_OUT;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int so = c * 128 + t * l.wtile, ss = c * 8 + t * l.wstile;
    w.c[t][0] = __builtin_bit_cast(mi4, __builtin_amdgcn_raw_buffer_load_b128(l.wc, wv, so, 0));
    w.c[t][1] = __builtin_bit_cast(mi4, __builtin_amdgcn_raw_buffer_load_b128(l.wc, wv + 16, so, 0));
    if constexpr (EVEN) {
      w.s[t][0] = __builtin_amdgcn_raw_buffer_load_b16(l.ws, wsv, ss, 0);
    } else {
      w.s[t][0] = __builtin_amdgcn_raw_buffer_load_b8(l.ws, wsv, ss, 0);
      w.s[t][1] = __builtin_amdgcn_raw_buffer_load_b8(l.ws, wsv + 1, ss, 0);
    }
  }
}

// The weights of step c as the MFMAs take them: a block past the row is zeros
// with scale 1 (what was loaded there belongs to the next row).
template <bool EVEN>
__device__ __forceinline__ void mg_ready(MgWeights& w, const MgLane& l, int c) {
  if constexpr (!EVEN) {
    const bool in0 = 8 * c + 2 * l.q < l.nb, in1 = 8 * c + 2 * l.q + 1 < l.nb;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w.c[t][0][i] = in0 ? w.c[t][0][i] : 0;
        w.c[t][1][i] = in1 ? w.c[t][1][i] : 0;
      }
      w.s[t][0] = static_cast<uint16_t>((in0 ? w.s[t][0] : kOne) | ((in1 ? w.s[t][1] : kOne) << 8));
    }
  }
}

template <bool EVEN>
__device__ __forceinline__ void mg_load_s(MgScales& s, const MgLane& l, int c) {
  const uint32_t v = c < l.steps ? l.asv : MG_OUT;
  if constexpr (EVEN) {
    const auto q = __builtin_amdgcn_raw_buffer_load_b64(l.as, v, 8 * c, 0);
    s.v[0] = q[0];
    s.v[1] = q[1];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) s.v[i] = __builtin_amdgcn_raw_buffer_load_b8(l.as, v + i, 8 * c, 0);
  }
}

template <bool EVEN>
__device__ __forceinline__ void mg_put_s(const MgScales& s, const MgLane& l, LdsByte* sb, int c) {
  mu2 v;
  if constexpr (EVEN) {
    v = mu2{s.v[0], s.v[1]};
  } else {
    v = mu2{0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i >> 2] |= (8 * c + i < l.nb ? s.v[i] : kOne) << (8 * (i & 3));
  }
  *(__attribute__((address_space(3))) mu2*)(sb + 8 * threadIdx.x) = v;
}

// The codes of step c: 8 rows per instruction, the four wavefronts in turn
// (always CAP / 2 instructions, so that waits can count them; rows past the
// tile have offsets outside the buffer).
template <int CAP>
__device__ __forceinline__ void mg_load_a(const MgLane& l, LdsByte* buf, int wave, int c) {
#pragma unroll
  for (int j = 0; j < CAP / 2; ++j)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        l.ac, (__attribute__((address_space(3))) void*)(buf + (4 * j + wave) * 1024), 16,
        c < l.steps ? l.av[j] : MG_OUT, c * 128, 0, 0);
}

// at: this lane's byte offsets of its two pieces of a tile's row, and of its
// scale bytes
struct MgRead {
  int k0, k1, s;
};

// The operands of two token tiles.
struct MgTokens {
  mi4 x[2][2];
  int s[2];
};

__device__ __forceinline__ MgTokens mg_read(const LdsByte* buf, const LdsByte* sbuf, const MgRead& at, int g) {
  MgTokens x;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = 2 * g + u;
    x.x[u][0] = *(__attribute__((address_space(3))) const mi4*)(buf + at.k0 + 2048 * i);
    x.x[u][1] = *(__attribute__((address_space(3))) const mi4*)(buf + at.k1 + 2048 * i);
    x.s[u] = *(__attribute__((address_space(3))) const uint16_t*)(sbuf + at.s + 128 * i);
  }
  return x;
}

template <int HALF>
__device__ __forceinline__ mf4 mg_mfma(mi4 w, mi4 x, mf4 c, uint32_t sw, int sx) {
  const mi8 a = {w.x, w.y, w.z, w.w, 0, 0, 0, 0};
  const mi8 b = {x.x, x.y, x.z, x.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, HALF, static_cast<int>(sw), HALF, sx);
}

// One step, two token tiles at a time, the next two on their way from LDS
// (past the last pair a read of whatever LDS holds there, not used).
template <int CAP>
__device__ __forceinline__ void mg_multiply(mf4 (&acc)[CAP][2], const MgWeights& w, const LdsByte* buf,
                                            const LdsByte* sbuf, const MgRead& at, int nt) {
  MgTokens x = mg_read(buf, sbuf, at, 0);
#pragma unroll
  for (int g = 0; g < CAP / 2; ++g) {
    if (2 * g < nt) {
      MgTokens next = x;
      if (g + 1 < CAP / 2) next = mg_read(buf, sbuf, at, g + 1);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          acc[2 * g + u][t] = mg_mfma<0>(w.c[t][0], x.x[u][0], acc[2 * g + u][t], w.s[t][0], x.s[u]);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          acc[2 * g + u][t] = mg_mfma<1>(w.c[t][1], x.x[u][1], acc[2 * g + u][t], w.s[t][0], x.s[u]);
      x = next;
    }
  }
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

// Step c, whose tokens are in buf and sb and whose weights are in w.  Into the
// buffers that step c - 1 has left go the tokens of step c + 2, into w the
// weights of step c + 3; the scales of step c + 1 move on to LDS.
template <int CAP, bool EVEN>
__device__ __forceinline__ void mg_step(mf4 (&acc)[CAP][2], const MgLane& l, const MgRead& at, int nt,
                                        int c, MgWeights& w, const LdsByte* buf, const LdsByte* sb,
                                        LdsByte* buf2, MgScales& s2, const MgScales& s1, LdsByte* sb1) {
  mg_load_a<CAP>(l, buf2, threadIdx.x >> 6, c + 2);
  mg_load_s<EVEN>(s2, l, c + 2);
  mg_ready<EVEN>(w, l, c);
  mg_multiply<CAP>(acc, w, buf, sb, at, nt);
  mg_load_w<EVEN>(w, l, c + 3);
  mg_put_s<EVEN>(s1, l, sb1, c + 1);
  // newer than the tokens of step c + 1: the weights of steps c + 2 and c + 3,
  // the tokens and scales of step c + 2
  mg_barrier<2 * mg_w_loads<EVEN>() + CAP / 2 + mg_s_loads<EVEN>()>();
}

template <int CAP, bool EVEN, bool GATED, bool BF16>
__device__ __forceinline__ void mg_tile(const LinearArgs& a, const RowTile& t, MgLane& l, int n0,
                                        LdsByte* buf0, LdsByte* buf1, LdsByte* buf2, LdsByte* sb0,
                                        LdsByte* sb1, LdsByte* sb2, int* s_src) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, q = lane >> 4;
  // opaque, so that no step's first products count as unconditional: the
  // compiler would move them past the barriers, to where their sums are used
  int nt = (t.rows + 15) / 16;
  asm volatile("" : "+s"(nt));
  MgWeights w0, w1, w2;
  MgScales s0, s1, s2;
  mg_load_w<EVEN>(w0, l, 0);
  mg_load_w<EVEN>(w1, l, 1);
  mg_load_w<EVEN>(w2, l, 2);
  // thread tid looks up tile row tid's source; the others take it from LDS
  int src = -1;
  if (tid < t.rows) {
    bool ok;
    src = source_row(a, t.r0 + tid, ok);
    if (tid < 16 * CAP) s_src[tid] = ok ? src : ~src;
  }
  l.asv = tid < t.rows ? static_cast<uint32_t>(src) * l.nb : MG_OUT;
  __syncthreads();
  // the row pieces this lane moves: tile row 8 (4 j + wave) + lane / 8
#pragma unroll
  for (int j = 0; j < CAP / 2; ++j) {
    const int row = 8 * (4 * j + wave) + (lane >> 3);
    const int v = s_src[row];
    l.av[j] = row < t.rows ? static_cast<uint32_t>(v < 0 ? ~v : v) * (a.K / 2) + 16 * ((lane & 7) ^ mg_swz(row & 15))
                           : MG_OUT;
  }
  const MgRead at = {r * 128 + 16 * ((2 * q) ^ mg_swz(r)), r * 128 + 16 * ((2 * q + 1) ^ mg_swz(r)),
                     r * 8 + 2 * q};
  mf4 acc[CAP][2] = {};
  mg_load_a<CAP>(l, buf0, wave, 0);
  mg_load_s<EVEN>(s0, l, 0);
  mg_load_a<CAP>(l, buf1, wave, 1);
  mg_load_s<EVEN>(s1, l, 1);
  mg_put_s<EVEN>(s0, l, sb0, 0);
  mg_barrier<CAP / 2 + mg_s_loads<EVEN>()>();
  int c = 0;
  for (; c + 3 <= l.steps; c += 3) {
    mg_step<CAP, EVEN>(acc, l, at, nt, c, w0, buf0, sb0, buf2, s2, s1, sb1);
    mg_step<CAP, EVEN>(acc, l, at, nt, c + 1, w1, buf1, sb1, buf0, s0, s2, sb2);
    mg_step<CAP, EVEN>(acc, l, at, nt, c + 2, w2, buf2, sb2, buf1, s1, s0, sb0);
  }
  // one or two steps left: nothing more to request.  (Their waits may not
  // count loads: the ones whose values nobody would use are not there.)
  if (c < l.steps) {
    mg_put_s<EVEN>(s1, l, sb1, c + 1);
    mg_barrier<0>();
    mg_ready<EVEN>(w0, l, c);
    mg_multiply<CAP>(acc, w0, buf0, sb0, at, nt);
    if (c + 1 < l.steps) {
      mg_ready<EVEN>(w1, l, c + 1);
      mg_multiply<CAP>(acc, w1, buf1, sb1, at, nt);
    }
  } else {
    mg_barrier<0>();   // a load still on its way to LDS may not outlive the workgroup
  }
  // 32-bit offsets from the tile's first row; a row without a source is zeros
  const int n = n0 + 32 * wave + 4 * q;
  const int width = GATED ? a.N / 2 : a.N;
  constexpr int kSize = BF16 ? 2 : 4;
  uint8_t* __restrict__ y = static_cast<uint8_t*>(a.y) + t.r0 * width * kSize;
#pragma unroll
  for (int i = 0; i < CAP; ++i) {
    const int local = 16 * i + r;
    if (local < t.rows) {
      const bool has = s_src[local] >= 0;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int col = n + 16 * w;
        if (col < a.N)
          store_out<GATED, BF16>(y + static_cast<uint32_t>(local * width + (GATED ? col / 2 : col)) * kSize,
                                 has ? acc[i][w] : mf4{0, 0, 0, 0});
      }
    }
  }
}

template <int CAP, bool EVEN, bool GATED, bool BF16>
__global__ __launch_bounds__(ML_THREADS, 2) void mx_linear_groups_kernel(LinearArgs a) {
  __shared__ __align__(16) uint8_t buf0[CAP * 2048], buf1[CAP * 2048], buf2[CAP * 2048];
  // every thread carries a row's scales
  __shared__ __align__(16) uint8_t sb0[ML_THREADS * 8], sb1[ML_THREADS * 8], sb2[ML_THREADS * 8];
  __shared__ int s_src[CAP * 16];   // each row's source, complemented where it has none
  // XCD x (workgroups go to the 8 XCDs in turn) takes row tiles x, x + 8, ...
  // with all their column slices, so a tile's token rows meet in one L2
  const int n_wg = (a.N + MG_ROWS - 1) / MG_ROWS;
  const int i = static_cast<int>(blockIdx.x) >> 3;
  const RowTile t = find_row_tile(a, 8 * (i / n_wg) + (static_cast<int>(blockIdx.x) & 7), 16 * CAP);
  if (t.rows <= 0) return;
  const int n0 = i % n_wg * MG_ROWS;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int nb = a.K / 32, crow = a.K / 2;
  MgLane l;
  l.nb = nb;
  l.q = lane >> 4;
  l.steps = (a.K + MG_STEP - 1) / MG_STEP;
  l.ac = mg_rsrc(a.ac, a.a_rows * crow);
  l.as = mg_rsrc(a.as, a.a_rows * nb);
  const int64_t wrow = static_cast<int64_t>(t.g) * a.N;
  l.wc = mg_rsrc(a.wc + wrow * crow, static_cast<int64_t>(a.N) * crow);
  l.ws = mg_rsrc(a.ws + wrow * nb, static_cast<int64_t>(a.N) * nb);
  const int row = n0 + 32 * wave + (lane & 15);
  l.wv = static_cast<uint32_t>(row * crow + 32 * l.q);
  l.wsv = static_cast<uint32_t>(row * nb + 2 * l.q);
  l.wtile = 16 * crow;
  l.wstile = 16 * nb;
  mg_tile<CAP, EVEN, GATED, BF16>(a, t, l, n0, (LdsByte*)buf0, (LdsByte*)buf1, (LdsByte*)buf2,
                                  (LdsByte*)sb0, (LdsByte*)sb1, (LdsByte*)sb2, s_src);
}

template <int CAP, bool GATED, bool BF16>
void launch_groups(const LinearArgs& a, hipStream_t s) {
  const int64_t m = 16 * CAP;
  const int64_t tiles = a.offsets ? a.R / m + min(static_cast<int64_t>(a.G), a.R) : (a.R + m - 1) / m;
  const int64_t n_wg = (a.N + MG_ROWS - 1) / MG_ROWS;
  const unsigned grid = static_cast<unsigned>((tiles + 7) / 8 * 8 * n_wg);
  if (a.K % MG_STEP == 0)
    mx_linear_groups_kernel<CAP, true, GATED, BF16><<<grid, ML_THREADS, 0, s>>>(a);
  else
    mx_linear_groups_kernel<CAP, false, GATED, BF16><<<grid, ML_THREADS, 0, s>>>(a);
}

template <bool GATED, bool BF16>
void launch_rows(const LinearArgs& a, hipStream_t s) {
  constexpr int MT = 4, SPLIT = 4;
  const int64_t full = (a.R + 16 * MT - 1) / (16 * MT);
  const int64_t tiles = a.offsets ? (a.R / (16 * MT)) + min(static_cast<int64_t>(a.G), a.R) : full;
  const unsigned grid = static_cast<unsigned>(tiles * ((a.N + 15) / 16));
  mx_linear_rows_kernel<MT, SPLIT, GATED, BF16><<<grid, ML_THREADS, 0, s>>>(a);
}

template <bool GATED, bool BF16>
void launch_product(const LinearArgs& a, hipStream_t s) {
  const int64_t avg = a.R / a.G;
  if (avg < 16 || a.a_rows * (a.K / 2) >= int64_t{MG_OUT})   // the other kernel has 32-bit offsets into A
    launch_rows<GATED, BF16>(a, s);
  else if (avg > 32)
    launch_groups<8, GATED, BF16>(a, s);
  else
    launch_groups<4, GATED, BF16>(a, s);
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
