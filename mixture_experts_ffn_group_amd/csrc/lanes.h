// Lane reductions and compile-time sort networks of the routers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {
namespace {

// Wave-wide reductions on DPP lane moves (GFX9 controls): the two quad
// permutations and row rotations by 4 and 8 reduce each 16-lane row, and the
// row broadcasts of lanes 15 and 31 carry the rows into lane 63, which is
// then read as a scalar. A few cycles per step, where a cross-lane shuffle
// through the LDS crossbar waits on its result every step.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, ROW_MASK, 0xf, false);
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max(v, dpp_u32<0xb1, 0xf>(v));   // quad_perm [1,0,3,2]
  v = max(v, dpp_u32<0x4e, 0xf>(v));   // quad_perm [2,3,0,1]
  v = max(v, dpp_u32<0x124, 0xf>(v));  // row_ror:4
  v = max(v, dpp_u32<0x128, 0xf>(v));  // row_ror:8
  v = max(v, dpp_u32<0x142, 0xa>(v));  // row_bcast:15 into rows 1, 3
  v = max(v, dpp_u32<0x143, 0xc>(v));  // row_bcast:31 into rows 2, 3
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ float wave_sum(float v) {
  auto add = [](float a, uint32_t b) { return a + __uint_as_float(b); };
  v = add(v, dpp_u32<0xb1, 0xf>(__float_as_uint(v)));
  v = add(v, dpp_u32<0x4e, 0xf>(__float_as_uint(v)));
  v = add(v, dpp_u32<0x124, 0xf>(__float_as_uint(v)));
  v = add(v, dpp_u32<0x128, 0xf>(__float_as_uint(v)));
  // rows 1 and 3 add the previous row's total; row 3 then adds rows 0 + 1 (carried by lane 31)
  const uint32_t b15 = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x142, 0xa, 0xf, false);
  v = v + __uint_as_float(b15);
  const uint32_t b31 = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x143, 0xc, 0xf, false);
  v = v + __uint_as_float(b31);
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// 16-lane (row) reductions with symmetric exchanges: quad swaps, then the
// half-row and row mirrors. Every lane combines its value with a partner's
// in the same association, so all 16 lanes end with the identical result.
__device__ __forceinline__ float row_sum(float v) {
  v = v + __uint_as_float(dpp_u32<0xb1, 0xf>(__float_as_uint(v)));
  v = v + __uint_as_float(dpp_u32<0x4e, 0xf>(__float_as_uint(v)));
  v = v + __uint_as_float(dpp_u32<0x141, 0xf>(__float_as_uint(v)));
  v = v + __uint_as_float(dpp_u32<0x140, 0xf>(__float_as_uint(v)));
  return v;
}

// Row maximum with each lane move feeding the max directly (every lane of a
// row has a source under these four patterns, so no lane keeps an old value).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max_step(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ uint32_t row_max_fused(uint32_t v) {
  v = dpp_max_step<0xb1>(v);   // quad_perm [1,0,3,2]
  v = dpp_max_step<0x4e>(v);   // quad_perm [2,3,0,1]
  v = dpp_max_step<0x141>(v);  // row_half_mirror
  v = dpp_max_step<0x140>(v);  // row_mirror
  return v;
}

// Batcher's odd-even merge sort network on N = 2^m elements (Knuth, TAOCP
// vol. 3, 5.3.4), as a compile-time list of compare-exchange pairs.
struct CxPair {
  int a, b;
};
template <int N>
struct OddEvenMergeNet {
  CxPair p[N * N] = {};
  int n = 0;
  constexpr OddEvenMergeNet() {
    for (int pp = 1; pp < N; pp <<= 1)
      for (int kk = pp; kk >= 1; kk >>= 1)
        for (int j = kk % pp; j + kk < N; j += 2 * kk)
          for (int i = 0; i < kk && i + j + kk < N; ++i)
            if ((i + j) / (2 * pp) == (i + j + kk) / (2 * pp)) p[n++] = CxPair{i + j, i + j + kk};
  }
};
template <int N>
__device__ __forceinline__ void sort_desc(uint64_t (&c)[N]) {
  constexpr OddEvenMergeNet<N> net{};
#pragma unroll
  for (int q = 0; q < net.n; ++q) {
    uint64_t& a = c[net.p[q].a];
    uint64_t& b = c[net.p[q].b];
    const bool sw = b > a;
    const uint64_t hi = sw ? b : a, lo = sw ? a : b;
    a = hi;
    b = lo;
  }
}
// 32-bit keys: a compare-exchange is a max and a min.
template <int N>
__device__ __forceinline__ void sort_desc(uint32_t (&c)[N]) {
  constexpr OddEvenMergeNet<N> net{};
#pragma unroll
  for (int q = 0; q < net.n; ++q) {
    const uint32_t a = c[net.p[q].a], b = c[net.p[q].b];
    c[net.p[q].a] = max(a, b);
    c[net.p[q].b] = min(a, b);
  }
}

}  // namespace
}  // namespace moe
