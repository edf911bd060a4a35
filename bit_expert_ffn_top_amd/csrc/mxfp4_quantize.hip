// Microscaled 4-bit floats: quantization of fp32 or bf16 rows and the values
// back (codes and scales as bitffn_moe.h lays them out).
//
// A row is a whole number of 32-value blocks, so both directions run over the
// matrix as one flat array of 8-value pieces, four lanes to a block: one
// 16-byte load of bf16 (two of fp32) per lane, contiguous over the wavefront.
// The block's largest magnitude is the largest of the |x| bit patterns as
// unsigned numbers (finite < inf < NaN), joined over the four lanes by two
// quad permutes; its exponent field less 2 is the scale byte, and
// v_cvt_scalef32_pk_fp4_f32 divides by the power of two, rounds to nearest
// even and saturates, two values per instruction.  Blocks below 2^-61 are
// lifted by 2^64 first (exact), so that no input of the conversion is
// subnormal.  Bound: HBM (4 or 2 bytes read, 17/32 written per value); a launch of
// 1 row of 2048 takes 1.4 us, one of 8192 x 2048 bf16 values 9.2 us (4.6 TB/s),
// their values back 8.4 us (5.1 TB/s); in fp32 15.2 and 15.8 us (5.0 and 4.8).
#include "moe_internal.h"
#include "mx_device.h"

namespace bitffn {
namespace {

constexpr int MQ_THREADS = 256;
constexpr int MQ_PIECES = 4;   // pieces per thread, all loads before any arithmetic

typedef uint32_t mu4 __attribute__((ext_vector_type(4)));

template <typename X>
struct Piece;   // 8 values as loaded

template <>
struct Piece<float> {
  mu4 a, b;
  __device__ __forceinline__ void load(const float* x, int64_t i) {
    const mu4* p = reinterpret_cast<const mu4*>(x + 8 * i);
    a = __builtin_nontemporal_load(p);
    b = __builtin_nontemporal_load(p + 1);
  }
  __device__ __forceinline__ void values(uint32_t (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = a[j];
      v[4 + j] = b[j];
    }
  }
};

template <>
struct Piece<uint16_t> {
  mu4 a;
  __device__ __forceinline__ void load(const uint16_t* x, int64_t i) {
    a = __builtin_nontemporal_load(reinterpret_cast<const mu4*>(x + 8 * i));
  }
  __device__ __forceinline__ void values(uint32_t (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = a[j] << 16;
      v[2 * j + 1] = a[j] & 0xFFFF0000u;
    }
  }
};

template <int CTRL>
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
                    0, static_cast<int>(v), CTRL, 0xF, 0xF, false)));
}

// pieces is a multiple of 4, so a block's four lanes are inside or outside
// the array together.
template <typename X>
__global__ __launch_bounds__(MQ_THREADS) void mx_quantize_kernel(const X* __restrict__ x,
                                                                 int64_t pieces,
                                                                 uint8_t* __restrict__ codes,
                                                                 uint8_t* __restrict__ scales) {
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (MQ_THREADS * MQ_PIECES) + threadIdx.x;
  Piece<X> in[MQ_PIECES];
#pragma unroll
  for (int q = 0; q < MQ_PIECES; ++q) {
    const int64_t i = i0 + q * MQ_THREADS;
    if (i < pieces) in[q].load(x, i);
  }
#pragma unroll
  for (int q = 0; q < MQ_PIECES; ++q) {
    const int64_t i = i0 + q * MQ_THREADS;
    if (i >= pieces) return;
    uint32_t v[8];
    in[q].values(v);
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, v[j] & 0x7FFFFFFFu);
    top = quad_max<0xB1>(top);   // quad_perm [1,0,3,2]
    top = quad_max<0x4E>(top);   // quad_perm [2,3,0,1]
    const uint32_t e = top >> 23;
    uint32_t s = e > 2 ? e - 2 : 0;
    uint32_t out = 0;
    if (e == 255) {
      s = 255;
    } else {
      // x 2^64 and s + 64 for small blocks: the same quotient, no subnormals
      const bool small = s < 64;
      const float lift = small ? 18446744073709551616.0f : 1.0f;
      const float scale = __builtin_bit_cast(float, (small ? s + 64 : s) << 23);
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = __builtin_bit_cast(float, v[j]) * lift;
      out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, f[0], f[1], scale, 0);
      out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, f[2], f[3], scale, 1);
      out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, f[4], f[5], scale, 2);
      out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, f[6], f[7], scale, 3);
    }
    reinterpret_cast<uint32_t*>(codes)[i] = out;
    if ((i & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(s);
  }
}

// A lane turns 4 bytes of codes into 8 values.  The scale is a float with the
// byte as its exponent field (0: the subnormal 2^-127), 255 NaN.
template <typename Y>
__global__ __launch_bounds__(MQ_THREADS) void mx_dequantize_kernel(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t pieces,
    Y* __restrict__ y) {
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (MQ_THREADS * MQ_PIECES) + threadIdx.x;
  uint32_t c[MQ_PIECES], s[MQ_PIECES];
#pragma unroll
  for (int q = 0; q < MQ_PIECES; ++q) {
    const int64_t i = i0 + q * MQ_THREADS;
    if (i < pieces) {
      c[q] = reinterpret_cast<const uint32_t*>(codes)[i];
      s[q] = scales[i >> 2];
    }
  }
#pragma unroll
  for (int q = 0; q < MQ_PIECES; ++q) {
    const int64_t i = i0 + q * MQ_THREADS;
    if (i >= pieces) return;
    float f[8];
    mx_values8(c[q], s[q], f);
    if constexpr (sizeof(Y) == 4) {
      float4* p = reinterpret_cast<float4*>(y + 8 * i);
      p[0] = make_float4(f[0], f[1], f[2], f[3]);
      p[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
      // exact in bf16: the high halves of the fp32 patterns
      mu4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = (__builtin_bit_cast(uint32_t, f[2 * j]) >> 16) |
               (__builtin_bit_cast(uint32_t, f[2 * j + 1]) & 0xFFFF0000u);
      *reinterpret_cast<mu4*>(y + 8 * i) = o;
    }
  }
}

unsigned grid_of(int64_t pieces) {
  return static_cast<unsigned>((pieces + MQ_THREADS * MQ_PIECES - 1) / (MQ_THREADS * MQ_PIECES));
}

}  // namespace

hipError_t launch_mx_quantize(const void* x, int x_dtype, int64_t rows, int cols, uint8_t* codes,
                              uint8_t* scales, hipStream_t s) {
  const int64_t pieces = rows * (cols / 8);
  if (x_dtype == MOE_DTYPE_F32)
    mx_quantize_kernel<float><<<grid_of(pieces), MQ_THREADS, 0, s>>>(
        static_cast<const float*>(x), pieces, codes, scales);
  else
    mx_quantize_kernel<uint16_t><<<grid_of(pieces), MQ_THREADS, 0, s>>>(
        static_cast<const uint16_t*>(x), pieces, codes, scales);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                int cols, void* y, int y_dtype, hipStream_t s) {
  const int64_t pieces = rows * (cols / 8);
  if (y_dtype == MOE_DTYPE_F32)
    mx_dequantize_kernel<float><<<grid_of(pieces), MQ_THREADS, 0, s>>>(
        codes, scales, pieces, static_cast<float*>(y));
  else
    mx_dequantize_kernel<uint16_t><<<grid_of(pieces), MQ_THREADS, 0, s>>>(
        codes, scales, pieces, static_cast<uint16_t*>(y));
  return hipGetLastError();
}

}  // namespace bitffn
