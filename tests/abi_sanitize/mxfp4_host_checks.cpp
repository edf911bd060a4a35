// Host-side argument checks of the 4-bit float and router-loss entry points,
// built and run as abi_host_checks.cpp is (tests/test_abi_mxfp4_sanitized.py).
// Every call fails its checks before any HIP call; the pointers are fake, the
// moe_mxfp4 structs real.
#include <climits>
#include <cstdint>
#include <cstdio>

#include "bitffn_moe.h"

namespace {

int g_checks = 0, g_failed = 0;

void expect(long long got, long long want, const char* what, int line) {
  ++g_checks;
  if (got != want) {
    ++g_failed;
    std::printf("FAILED line %d: %s returned %lld, expected %lld\n", line, what, got, want);
  }
}
#define EXPECT(call, want) expect(static_cast<long long>(call), static_cast<long long>(want), #call, __LINE__)

template <typename T = void>
T* fp(uintptr_t off = 0) {
  return reinterpret_cast<T*>(0x7F0000000000ull + off);
}
const hipStream_t s0 = nullptr;

moe_mxfp4 mx(int n, int rows, int cols, uintptr_t at = 0) {
  return moe_mxfp4{n, rows, cols, 0, fp(at), fp(at + (1 << 20))};
}

void group_pairs() {
  const auto call = [](int T, int k, int E, size_t bytes) {
    return moe_group_pairs(fp<int32_t>(), T, k, E, fp<int32_t>(1 << 12), fp<int32_t>(1 << 13),
                           fp<int32_t>(1 << 14), fp(1 << 16), bytes, s0);
  };
  const size_t need = moe_group_workspace_bytes(8192, 512);
  EXPECT(need > 0, 1);
  EXPECT(call(8192, 10, 512, need - 1), MOE_ENOSPC);
  for (int T : {0, -1, 65537, INT_MAX, INT_MIN}) EXPECT(call(T, 10, 512, need), MOE_EINVAL);
  for (int k : {0, -1, MOE_MAX_TOPK + 1, INT_MAX}) EXPECT(call(8192, k, 512, need), MOE_EINVAL);
  for (int E : {0, -1, MOE_MAX_EXPERTS + 1, INT_MAX}) EXPECT(call(8192, 10, E, need), MOE_EINVAL);
  EXPECT(moe_group_workspace_bytes(INT_MAX, INT_MAX), 0);
  EXPECT(moe_group_workspace_bytes(INT_MIN, 1), 0);
}

void quantize() {
  uint8_t *c = fp<uint8_t>(1 << 20), *s = fp<uint8_t>(1 << 21);
  for (int64_t rows : {int64_t{-1}, int64_t{1} << 24, INT64_MAX, INT64_MIN}) {
    EXPECT(moe_mxfp4_quantize(fp(), MOE_DTYPE_F32, rows, 64, c, s, s0), MOE_EINVAL);
    EXPECT(moe_mxfp4_dequantize(c, s, rows, 64, fp(), MOE_DTYPE_BF16, s0), MOE_EINVAL);
  }
  for (int cols : {0, -32, 16, 33, MOE_MAX_MX_COLS + 32, INT_MAX, INT_MIN}) {
    EXPECT(moe_mxfp4_quantize(fp(), MOE_DTYPE_F32, 4, cols, c, s, s0), MOE_EINVAL);
    EXPECT(moe_mxfp4_dequantize(c, s, 4, cols, fp(), MOE_DTYPE_BF16, s0), MOE_EINVAL);
  }
  EXPECT(moe_mxfp4_quantize(fp(), 7, 4, 64, c, s, s0), MOE_EINVAL);
  EXPECT(moe_mxfp4_quantize(nullptr, MOE_DTYPE_F32, 4, 64, c, s, s0), MOE_EINVAL);
  EXPECT(moe_mxfp4_quantize(fp(2), MOE_DTYPE_F32, 4, 64, c, s, s0), MOE_EALIGN);
  EXPECT(moe_mxfp4_dequantize(c, s + 8, 4, 64, fp(), MOE_DTYPE_F32, s0), MOE_EALIGN);
  EXPECT(moe_mxfp4_quantize(nullptr, MOE_DTYPE_F32, 0, 64, nullptr, nullptr, s0), MOE_OK);
}

void products() {
  const auto call = [](moe_mxfp4 A, moe_mxfp4 W, int div, int64_t R, bool offsets = true, bool src = true,
                       bool gated = false) {
    const auto f = gated ? moe_mxfp4_gate_up : moe_mxfp4_linear;
    return f(&A, &W, offsets ? fp<int32_t>(1 << 24) : nullptr, src ? fp<int32_t>(1 << 25) : nullptr, div, R,
             fp(8), MOE_DTYPE_F32, s0);
  };
  const moe_mxfp4 A = mx(1, 100, 256, 1 << 8), W = mx(8, 128, 256, 1 << 27);
  EXPECT(call(A, W, 2, 50), MOE_EALIGN);   // everything else is in order: y is misaligned
  EXPECT(moe_mxfp4_linear(nullptr, &W, nullptr, nullptr, 1, 1, fp(), MOE_DTYPE_F32, s0), MOE_EINVAL);
  EXPECT(moe_mxfp4_linear(&A, nullptr, nullptr, nullptr, 1, 1, fp(), MOE_DTYPE_F32, s0), MOE_EINVAL);
  for (int div : {0, -1, INT_MIN}) EXPECT(call(A, W, div, 50), MOE_EINVAL);
  for (int64_t R : {int64_t{-1}, int64_t{1} << 24, INT64_MAX, INT64_MIN}) EXPECT(call(A, W, 2, R), MOE_EINVAL);
  EXPECT(call(A, W, 2, 50, false), MOE_EINVAL);         // eight matrices need bounds
  EXPECT(call(A, W, 1, 101, true, false), MOE_EINVAL);  // more rows than A has
  EXPECT(call(mx(2, 100, 256), W, 2, 50), MOE_EINVAL);
  EXPECT(call(A, mx(8, 120, 256), 2, 50), MOE_EINVAL);
  EXPECT(call(A, mx(8, 96, 256), 2, 50, true, true, true), MOE_EINVAL);
  EXPECT(call(A, mx(8, 128, 288), 2, 50), MOE_EINVAL);
  EXPECT(call(A, mx(8, 65552, 256), 2, 50), MOE_EINVAL);
  EXPECT(call(A, mx(MOE_MAX_EXPERTS + 1, 128, 256), 2, 50), MOE_EINVAL);
  EXPECT(call(A, mx(INT_MIN, INT_MIN, INT_MIN), 2, 50), MOE_EINVAL);
  EXPECT(call(mx(1, INT_MAX, 256), W, 2, 50), MOE_EINVAL);
  EXPECT(call(A, W, INT_MAX, 0), MOE_OK);
}

void decode() {
  const size_t need = moe_mxfp4_ffn_decode_workspace_bytes(4, 10, 768);
  EXPECT(need > 0, 1);
  const auto call = [](moe_mxfp4 GU, moe_mxfp4 D, int shared, int T, int k, size_t bytes) {
    return moe_mxfp4_ffn_decode(&GU, &D, shared, fp<float>(), T, k, fp<int32_t>(1 << 16), fp<float>(1 << 17),
                                fp<float>(1 << 18), fp(1 << 19), bytes, s0);
  };
  const moe_mxfp4 GU = mx(64, 1536, 2048), D = mx(64, 2048, 768);
  EXPECT(call(GU, D, 63, 4, 10, need - 1), MOE_ENOSPC);
  for (int s : {-2, 64, INT_MAX, INT_MIN}) EXPECT(call(GU, D, s, 4, 10, need), MOE_EINVAL);
  for (int T : {0, -1, 5, INT_MAX, INT_MIN}) EXPECT(call(GU, D, -1, T, 10, need), MOE_EINVAL);
  for (int k : {-1, 17, MOE_MAX_TOPK + 1, INT_MAX, INT_MIN}) EXPECT(call(GU, D, -1, 4, k, need), MOE_EINVAL);
  EXPECT(call(mx(63, 1536, 2048), D, -1, 4, 10, need), MOE_EINVAL);
  EXPECT(call(mx(64, 1536, 4128), mx(64, 4128, 768), -1, 1, 1, need), MOE_EINVAL);
  EXPECT(call(mx(64, 1 << 24, 2048), mx(64, 2048, 1 << 23), -1, 1, 1, need), MOE_EINVAL);
  for (int f : {0, 31, 4128, INT_MAX, INT_MIN}) EXPECT(moe_mxfp4_ffn_decode_workspace_bytes(4, 10, f), 0);
  EXPECT(moe_mxfp4_ffn_decode_workspace_bytes(4, INT_MAX, 768), 0);
  EXPECT(moe_mxfp4_ffn_decode_workspace_bytes(INT_MAX, 10, 768), 0);
}

void balance() {
  const int T = 65536, E = 512, S = 16;
  const size_t need = moe_route_balance_workspace_bytes(T, E, S);
  EXPECT(need > 0, 1);
  EXPECT(moe_route_balance_workspace_bytes((1 << 24) - 1, MOE_MAX_EXPERTS, 65536) > 0, 1);
  for (int t : {-1, 1 << 24, INT_MAX, INT_MIN}) EXPECT(moe_route_balance_workspace_bytes(t, E, S), 0);
  for (int s : {0, -1, 65537, INT_MAX}) EXPECT(moe_route_balance_workspace_bytes(T, E, s), 0);
  const auto forward = [](int t, int e, int k, int s, size_t bytes) {
    return moe_route_balance(fp<float>(), fp<int32_t>(1 << 16), t, e, k, fp<int32_t>(1 << 17), s, nullptr,
                             fp<float>(1 << 18), fp<float>(1 << 19), fp<int32_t>(1 << 20), fp<float>(1 << 21),
                             fp<int32_t>(1 << 22), fp(1 << 23), bytes, s0);
  };
  const auto backward = [](int t, int e, int k, int s, float* out) {
    return moe_route_backward(fp<float>(), fp<int32_t>(1 << 16), t, e, k, fp<int32_t>(1 << 17), s, nullptr,
                              fp<int32_t>(1 << 20), fp<int32_t>(1 << 22), fp<float>(1 << 18), fp<float>(1 << 19),
                              nullptr, nullptr, out, s0);
  };
  EXPECT(forward(T, E, 10, S, need - 1), MOE_ENOSPC);
  EXPECT(backward(T, E, 10, S, fp<float>()), MOE_EINVAL);   // onto the logits
  EXPECT(backward(T, E, 10, S, fp<float>(4)), MOE_EALIGN);
  for (int v : {-1, 1 << 24, INT_MAX, INT_MIN}) {
    EXPECT(forward(v, E, 10, S, need), MOE_EINVAL);
    EXPECT(backward(v, E, 10, S, fp<float>(1 << 24)), MOE_EINVAL);
    EXPECT(forward(T, v, 10, S, need), MOE_EINVAL);
    EXPECT(forward(T, E, v, S, need), MOE_EINVAL);
    EXPECT(forward(T, E, 10, v, need), MOE_EINVAL);
    EXPECT(backward(T, E, 10, v, fp<float>(1 << 24)), MOE_EINVAL);
  }
}

}  // namespace

int main() {
  group_pairs();
  quantize();
  products();
  decode();
  balance();
  std::printf("abi host checks: %d passed, %d failed\n", g_checks - g_failed, g_failed);
  return g_failed == 0 ? 0 : 1;
}
