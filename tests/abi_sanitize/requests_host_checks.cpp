// Host-side argument checks of the dispatch to the experts and back, the adapters
// and the verification of drafted tokens, built and run as abi_host_checks.cpp is
// (tests/test_abi_requests_sanitized.py).  Every call fails its checks before any
// HIP call; the pointers are fake.
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
T* fp(uintptr_t n, uintptr_t off = 0) {
  return reinterpret_cast<T*>(0x7F0000000000ull + (n << 32) + off);
}
const hipStream_t s0 = nullptr;
const int kInts[] = {INT_MIN, INT_MIN + 1, -65536, -1, 0, 1, 3, 65535, 65537, 1 << 24, INT_MAX - 1, INT_MAX};

void dispatch() {
  const auto call = [](int T, int d, int k, int E, size_t bytes, uintptr_t off = 8) {
    return moe_dispatch(fp(0), MOE_DTYPE_F32, T, d, fp<int32_t>(1), k, E, fp(2, off), fp<int32_t>(3),
                        fp<int32_t>(4), fp(5), bytes, s0);
  };
  EXPECT(call(64, 2048, 10, 512, 0), MOE_EALIGN);   // everything else is in order
  for (int T : kInts)
    if (T < 0 || T > 65536) {
      EXPECT(call(T, 64, 2, 8, SIZE_MAX), MOE_EINVAL);
      EXPECT(moe_dispatch_workspace_bytes(T, 2, 8), 0);
    }
  for (int v : kInts) {
    if (v < 1 || v > MOE_MAX_TOPK) {
      EXPECT(call(64, 64, v, 8, SIZE_MAX), MOE_EINVAL);
      EXPECT(moe_dispatch_workspace_bytes(64, v, 8), 0);
    }
    if (v < 1 || v > MOE_MAX_EXPERTS) {
      EXPECT(call(64, 64, 2, v, SIZE_MAX), MOE_EINVAL);
      EXPECT(moe_dispatch_workspace_bytes(64, 2, v), 0);
    }
    if (v < 4 || v > MOE_MAX_MX_COLS || v % 4) EXPECT(call(64, v, 2, 8, SIZE_MAX), MOE_EINVAL);
  }
  const size_t need = moe_dispatch_workspace_bytes(65536, MOE_MAX_TOPK, MOE_MAX_EXPERTS);
  EXPECT(need > 0, 1);
  EXPECT(call(65536, MOE_MAX_MX_COLS, MOE_MAX_TOPK, MOE_MAX_EXPERTS, need - 1, 0), MOE_ENOSPC);
}

void combine() {
  const auto rows = [](int64_t R, int T, int d, int k, uintptr_t off = 8) {
    return moe_combine_rows(fp(0), MOE_DTYPE_BF16, R, T, d, k, fp<int32_t>(1), fp<float>(2), fp(3),
                            MOE_DTYPE_F32, fp(4, off), MOE_DTYPE_BF16, s0);
  };
  const auto back = [](int64_t R, int T, int d, int k, uintptr_t off = 8) {
    return moe_combine_backward(fp(0), MOE_DTYPE_F32, fp(1), MOE_DTYPE_BF16, R, T, d, k, fp<int32_t>(2),
                                fp<float>(3), fp(4, off), fp<float>(5), s0);
  };
  EXPECT(rows(INT_MAX, (1 << 24) - 1, MOE_MAX_MX_COLS, MOE_MAX_TOPK), MOE_EALIGN);
  EXPECT(back(INT_MAX, (1 << 24) - 1, MOE_MAX_MX_COLS, MOE_MAX_TOPK), MOE_EALIGN);
  for (int64_t R : {int64_t{-1}, INT64_MIN, INT64_MAX, int64_t{1} << 31}) {
    EXPECT(rows(R, 4, 64, 2), MOE_EINVAL);
    EXPECT(back(R, 4, 64, 2), MOE_EINVAL);
  }
  for (int v : kInts) {
    if (v < 0 || v >= 1 << 24) {
      EXPECT(rows(8, v, 64, 2), MOE_EINVAL);
      EXPECT(back(8, v, 64, 2), MOE_EINVAL);
    }
    if (v < 4 || v > MOE_MAX_MX_COLS || v % 4) {
      EXPECT(rows(8, 4, v, 2), MOE_EINVAL);
      EXPECT(back(8, 4, v, 2), MOE_EINVAL);
    }
    if (v < 1 || v > MOE_MAX_TOPK) {
      EXPECT(rows(8, 4, 64, v), MOE_EINVAL);
      EXPECT(back(8, 4, 64, v), MOE_EINVAL);
    }
  }
}

void lora() {
  const auto call = [](int64_t T, int d_in, int d_out, int n, int rank, int S, bool seq, size_t bytes,
                       uintptr_t off = 8) {
    return moe_lora(fp(0), fp(1), MOE_DTYPE_BF16, T, d_in, d_out, fp<uint16_t>(2), fp<uint16_t>(3), n, rank,
                    seq ? fp<int32_t>(4) : nullptr, S, fp<int32_t>(5), fp<float>(6), fp(7, off), MOE_DTYPE_F32,
                    fp(8), bytes, s0);
  };
  EXPECT(call(100, 64, 48, 4, 16, 7, true, SIZE_MAX), MOE_EALIGN);
  EXPECT(call(100, 64, 48, 4, 16, 7, false, SIZE_MAX), MOE_EINVAL);
  for (int64_t T : {int64_t{-1}, INT64_MIN, INT64_MAX, int64_t{1} << 24}) {
    EXPECT(call(T, 64, 48, 4, 16, 7, true, SIZE_MAX), MOE_EINVAL);
    EXPECT(moe_lora_workspace_bytes(T, 16, 7), 0);
  }
  for (int v : kInts) {
    if (v < 32 || v % 32 || v > MOE_MAX_MX_COLS) EXPECT(call(100, v, 48, 4, 16, 7, true, SIZE_MAX), MOE_EINVAL);
    if (v < 16 || v % 16 || v > MOE_MAX_MX_COLS) EXPECT(call(100, 64, v, 4, 16, 7, true, SIZE_MAX), MOE_EINVAL);
    if (v < 1 || v > MOE_MAX_EXPERTS) EXPECT(call(100, 64, 48, v, 16, 7, true, SIZE_MAX), MOE_EINVAL);
    if (v < 8 || v % 8 || v > MOE_MAX_RANK) {
      EXPECT(call(100, 64, 48, 4, v, 7, true, SIZE_MAX), MOE_EINVAL);
      EXPECT(moe_lora_workspace_bytes(5000, v, 7), 0);
    }
    if (v < 1 || v > 65536) EXPECT(call(100, 64, 48, 4, 16, v, true, SIZE_MAX), MOE_EINVAL);
    if (v < 0 || v > 65536) EXPECT(moe_lora_workspace_bytes(5000, 16, v), 0);
    if (v != 100) EXPECT(call(100, 64, 48, 4, 16, v, false, SIZE_MAX), MOE_EINVAL);
  }
  EXPECT(call(65537, 64, 48, 4, 16, 65537, false, SIZE_MAX), MOE_EINVAL);
  const size_t need = moe_lora_workspace_bytes((1 << 24) - 1, MOE_MAX_RANK, 65536);
  EXPECT(need > (size_t{1} << 32), 1);
  EXPECT(call((1 << 24) - 1, 64, 48, 4, MOE_MAX_RANK, 65536, true, need - 1, 0), MOE_ENOSPC);
}

void verify() {
  const auto call = [](int B, int n, int V, size_t bytes, uintptr_t off = 8) {
    return moe_verify_drafts(fp(0), fp(1), MOE_DTYPE_F32, B, n, V, fp<int32_t>(2), fp<int32_t>(3), fp<float>(4),
                             fp<float>(5), fp<int32_t>(6, off), fp<int32_t>(7), fp(8), bytes, s0);
  };
  EXPECT(call(3, 4, 1000, 0), MOE_EALIGN);
  for (int v : kInts) {
    if (v < 0 || v > 65536) {
      EXPECT(call(v, 4, 1000, SIZE_MAX), MOE_EINVAL);
      EXPECT(moe_verify_drafts_workspace_bytes(v, 1000), 0);
    }
    if (v < 0 || v > MOE_MAX_DRAFTS) EXPECT(call(3, v, 1000, SIZE_MAX), MOE_EINVAL);
    if (v < 1 || v >= 1 << 24) {
      EXPECT(call(3, 4, v, SIZE_MAX), MOE_EINVAL);
      EXPECT(moe_verify_drafts_workspace_bytes(3, v), 0);
    }
  }
  const size_t need = moe_verify_drafts_workspace_bytes(65536, (1 << 24) - 1);
  EXPECT(need >= size_t{1} << 34, 1);
  EXPECT(call(65536, MOE_MAX_DRAFTS, (1 << 24) - 1, need - 1, 0), MOE_ENOSPC);
}

}  // namespace

int main() {
  dispatch();
  combine();
  lora();
  verify();
  std::printf("abi host checks: %d passed, %d failed\n", g_checks - g_failed, g_failed);
  return g_failed ? 1 : 0;
}
