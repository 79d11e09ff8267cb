// The whole MoE FFN layer for a few tokens (a decode step): router, experts and
// combine without the permute and the 256-row tiles of the grouped GEMMs.
//
// With T <= 64 tokens the layer is a stream over the weights of the experts that
// have a token: 6 * emb * mlp bytes each in bf16, for 2 to 2 * T multiply-adds an
// element. So the kernels are built around the weight loads: a wave loads 16 bytes
// a lane straight into registers in the operand order of the matrix cores, nothing
// of a weight goes through LDS, and each weight byte is read once for all (up to 16)
// rows of its expert.
//
// Kernels: few_logits (64-bit sums on the fp64 matrix cores, cut along emb),
// few_topk (one wave a token), few_experts (a workgroup per expert, 16 of its rows,
// and a slice of mlp columns: gate/up, SwiGLU, and the slice's share of the down
// product) and few_sum (a token's shares, weighted).
#include "common.h"
#include "kernels.h"
#include "lanes.h"

namespace moe {
namespace {

typedef double f64x4_t __attribute__((ext_vector_type(4)));

constexpr int kRows = 16;   // rows of a tile: the matrix instruction's side
constexpr int kFewMaxSlice = 256;  // most mlp columns of a workgroup
constexpr int kCols = 64;   // mlp columns of a sub-slice: 64 gate and 64 up columns are the 128 columns of a load step

// ---------------------------------------------------------------- router

// logits[split][t][e] = sum over the split's rows of x[t, i] wr[i, e]. The products (8 + 24 bits) are exact in
// fp64 and the sums are off by 2^-53 a step, so picks are those of exact arithmetic but for ties to 2^-40.
// A wave takes 16 experts and a run of emb; v_mfma_f64_16x16x4 has A[i = lane%16][k = lane/16],
// B[k = lane/16][j = lane%16] and D[i = 4r + lane/16][j = lane%16].
constexpr int kLogitWaves = 8;

template <int NT>
__global__ __launch_bounds__(kLogitWaves * 64) void few_logits_kernel(int T, int emb, int E, int run,
                                                                     const uint16_t* __restrict__ x,
                                                                     const float* __restrict__ wr,
                                                                     double* __restrict__ out) {
  __shared__ double red[kLogitWaves][NT * 16][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x * 16 + (lane & 15);
  const int ec = e < E ? e : E - 1;  // columns past E are computed on the last one and not stored
  const int k0 = (blockIdx.y * kLogitWaves + wave) * run;
  const int k1 = min(k0 + run, emb);
  const int kl = lane >> 4;
  f64x4_t acc[NT];
  const uint16_t* xr[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    acc[n] = f64x4_t{0, 0, 0, 0};
    const int t = n * 16 + (lane & 15);
    xr[n] = x + (int64_t)(t < T ? t : T - 1) * emb + kl;
  }
  const float* wp = wr + (int64_t)kl * E + ec;
#pragma unroll 4
  for (int k = k0; k < k1; k += 4) {  // emb and run are multiples of 4
    const double b = (double)wp[(int64_t)k * E];
#pragma unroll
    for (int n = 0; n < NT; ++n)
      acc[n] = __builtin_amdgcn_mfma_f64_16x16x4f64((double)bf16_to_f32(xr[n][k]), b, acc[n], 0, 0, 0);
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][n * 16 + 4 * r + kl][lane & 15] = acc[n][r];
  __syncthreads();
  for (int i = threadIdx.x; i < NT * 256; i += kLogitWaves * 64) {
    const int t = i >> 4, ee = blockIdx.x * 16 + (i & 15);
    if (t >= T || ee >= E) continue;
    double s = 0;
#pragma unroll
    for (int w = 0; w < kLogitWaves; ++w) s += red[w][t][i & 15];
    out[((int64_t)blockIdx.y * T + t) * E + ee] = s;
  }
}

// Order-preserving 64-bit key: larger logit, larger key; -0 like +0; NaN 1, below every number; 0 is "taken".
__device__ __forceinline__ uint64_t key64(double v) {
  if (v != v) return 1;
  if (v == 0) v = 0;
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double key64_value(uint64_t k) {
  if (k == 1) return -__builtin_inf();
  return __longlong_as_double((long long)((k >> 63) ? (k & 0x7fffffffffffffffull) : ~k));
}

// One wave picks token t's experts: lane j ends with pick j's expert and weight (lanes past k: unspecified).
__device__ __forceinline__ void few_pick(int T, int E, int k, int splits, int t, const double* __restrict__ logits,
                                         const float* __restrict__ bias, int lane, int& pick, float& weight) {
  uint64_t key[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane + 64 * i;
    key[i] = 0;
    if (e < E) {
      double s = 0;
      for (int c = 0; c < splits; ++c) s += logits[((int64_t)c * T + t) * E + e];
      if (bias) s += (double)bias[e];
      key[i] = key64(s);
    }
  }
  pick = 0;
  double l = -__builtin_inf();
  for (int j = 0; j < k; ++j) {
    uint64_t best = key[0];
    int bi = 0;
#pragma unroll
    for (int i = 1; i < 4; ++i)
      if (key[i] > best) best = key[i], bi = i;
    const uint32_t hi = (uint32_t)(best >> 32), lo = (uint32_t)best;
    const uint32_t mh = wave_max_u32(hi);
    const uint32_t ml = wave_max_u32(hi == mh ? lo : 0u);
    const bool top = hi == mh && lo == ml;
    // equal values: the lowest id
    const int e = 0xffff - (int)wave_max_u32(top ? 0xffffu - (uint32_t)(lane + 64 * bi) : 0u);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 64 * i == e) key[i] = 0;
    if (lane == j) pick = e, l = key64_value((uint64_t)mh << 32 | ml);
  }
  const double l0 = __shfl(l, 0);
  double w = lane < k && l != -__builtin_inf() ? exp(l - l0) : 0.0;  // a disabled expert's weight is 0
  double s = w;
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) s += __shfl_xor(s, m);
  weight = s == 0 ? 0.0f : (float)(w / s);
}

__global__ __launch_bounds__(64) void few_topk_kernel(int T, int E, int k, int splits, const double* __restrict__ logits,
                                                      const float* __restrict__ bias, int32_t* __restrict__ topk_idx,
                                                      float* __restrict__ topk_w) {
  const int lane = threadIdx.x, t = blockIdx.x;
  int pick;
  float weight;
  few_pick(T, E, k, splits, t, logits, bias, lane, pick, weight);
  if (lane < k) {
    topk_idx[t * k + lane] = pick;
    topk_w[t * k + lane] = weight;
  }
}

// ---------------------------------------------------------------- experts

// Both weight forms are read in steps of 8 KB a wave (8 loads of 16 bytes a lane) over 128 columns, and both give the
// matrix instruction (v_mfma_f32_16x16x32_bf16: A[row lane%16][k 8*(lane/16) + i], B[k][column lane%16], D[row
// 4*(lane/16) + r][column lane%16]) its B operand straight from the registers they were loaded into.
//
// bf16, row-major [K, N], a step is 32 rows: lane (g = lane/16, c = lane%16) loads columns 8c..8c+7 of rows 8g..8g+7.
// Product j takes column 8c + j of every lane c; its 8 values along K lie in the lane's 8 rows, and one byte permute
// puts two of them into a register.
struct StepBf16 {
  static constexpr int kK = 32;
  u32x4_t v[8];
  __device__ __forceinline__ void load(const uint16_t* p, int64_t ld) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = ld16(p + i * ld);
  }
  __device__ __forceinline__ bf16x8_t frag(int j) const {
    const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
    u32x4_t r;
#pragma unroll
    for (int p = 0; p < 4; ++p) r[p] = __builtin_amdgcn_perm(v[2 * p + 1][j >> 1], v[2 * p][j >> 1], sel);
    return __builtin_bit_cast(bf16x8_t, r);
  }
};

// MXFP8, K-contiguous rows [N, K], a step is 64 values of K: of column 16j + c lane (g, c) loads codes 16g..16g+15 and
// the dword with the scales of the step's two 32-blocks. They convert to bf16 exactly (3 bits of mantissa; a scale
// code below 3, which only blocks of subnormal weights have, or above 246 leaves bf16's range), 8 values an operand.
struct StepMx {
  static constexpr int kK = 64;
  u32x4_t v[8];
  uint32_t sc[8];
  __device__ __forceinline__ void load(int j, const uint8_t* code, const uint8_t* scale) {
    v[j] = ld16(code);
    sc[j] = *reinterpret_cast<const uint32_t*>(scale);
  }
  __device__ __forceinline__ bf16x8_t frag(int j, int h, int g) const {
    // the conversion's scale operand is a float of which it takes the exponent
    const float s = __uint_as_float(((g & 2) ? (sc[j] >> 8) & 0xffu : sc[j] & 0xffu) << 23);
    u32x4_t r;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      r[2 * p] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[j][2 * h + p], s, false));
      r[2 * p + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[j][2 * h + p], s, true));
    }
    return __builtin_bit_cast(bf16x8_t, r);
  }
};

__device__ __forceinline__ f32x4_t mfma(bf16x8_t a, bf16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Workgroup (tile, slice): up to 16 rows (slots t*k + j) of one expert, and `slice` of its mlp columns. The waves share
// the contraction of the first product (emb) and add up through LDS; of the second (the slice's columns) each takes
// output columns. part[slot][slice][emb] receives the slice's share of the slot's output row.
template <bool MX, int NW>
__global__ __launch_bounds__(NW * 64, 2) void few_experts_kernel(int S, int k, int emb, int mlp, int E, int slice, int ns,
                                                                 const uint16_t* __restrict__ x,
                                                                 const int32_t* __restrict__ topk_idx, FewWeights wt,
                                                                 float* __restrict__ part) {
  constexpr int kLdA = kFewMaxSlice + 8;
  __shared__ __align__(16) float red[NW][kRows][128];
  __shared__ __align__(16) uint16_t a_hi[kRows][kLdA], a_lo[kRows][kLdA];
  __shared__ int cnt[kMaxExperts];
  __shared__ int found[2];
  __shared__ int rows[kRows];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = lane & 15, g = lane >> 4;
  const int tile = blockIdx.x / ns, sl = blockIdx.x - tile * ns;

  // which expert (tiles go by expert, then by row), and which of its rows
  for (int i = tid; i < kMaxExperts; i += NW * 64) cnt[i] = 0;
  if (tid < kRows) rows[tid] = -1;
  if (tid == 0) found[0] = -1;
  __syncthreads();
  for (int i = tid; i < S; i += NW * 64) {
    const int e = topk_idx[i];
    if ((unsigned)e < (unsigned)E) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  if (wave == 0) {
    int base = 0;
    for (int q = 0; q < E; q += 64) {
      const int n = (cnt[q + lane] + kRows - 1) / kRows;
      int inc = n;
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) {
        const int up = __shfl_up(inc, m);
        if (lane >= m) inc += up;
      }
      const int first = base + inc - n;
      if (tile >= first && tile < first + n) found[0] = q + lane, found[1] = tile - first;
      base += __shfl(inc, 63);
    }
  }
  __syncthreads();
  const int e = found[0];
  if (e < 0) return;
  const int r0 = found[1] * kRows;
  if (wave == 0) {
    int base = 0;
    for (int q = 0; q < S; q += 64) {
      const bool mine = q + lane < S && topk_idx[q + lane] == e;
      const uint64_t m = __ballot(mine);
      const int r = base + popc64(m & ((1ull << lane) - 1)) - r0;
      if (mine && r >= 0 && r < kRows) rows[r] = q + lane;
      base += popc64(m);
    }
  }
  __syncthreads();
  const int nrows = min(kRows, cnt[e] - r0);
  // lanes past the last row compute on the first one; their rows of the results are not used
  const uint16_t* xr = x + (int64_t)((c < nrows ? rows[c] : rows[0]) / k) * emb;

  const int m0 = sl * slice;
  const int width = min(slice, mlp - m0);
  for (int s0 = 0; s0 < width; s0 += kCols) {
    // first product: 64 gate and the 64 up columns from m0 + s0
    f32x4_t acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = f32x4_t{0, 0, 0, 0};
    if constexpr (!MX) {
      const int64_t ld = 2 * (int64_t)mlp;
      const uint16_t* p = wt.wi + ((int64_t)e * emb + 8 * g) * ld + m0 + s0 + (c < 8 ? 8 * c : mlp + 8 * (c - 8));
#pragma unroll 2
      for (int kk = wave * StepBf16::kK; kk < emb; kk += NW * StepBf16::kK) {
        StepBf16 st;
        st.load(p + kk * ld, ld);
        const bf16x8_t a = __builtin_bit_cast(bf16x8_t, ld16(xr + kk + 8 * g));
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = mfma(a, st.frag(j), acc[j]);
      }
    } else {
      const int64_t row = (int64_t)e * 2 * mlp + m0 + s0 + c;
      const uint8_t* p = wt.wic + row * emb + 16 * g;
      const uint8_t* q = wt.wis + ((int64_t)e * (emb / 64) * 2 * mlp + m0 + s0 + c) * 4;
#pragma unroll 2
      for (int kk = wave * StepMx::kK; kk < emb; kk += NW * StepMx::kK) {
        StepMx st;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int n = j < 4 ? 16 * j : mlp + 16 * (j - 4);
          st.load(j, p + (int64_t)n * emb + kk, q + ((int64_t)(kk / 64) * 2 * mlp + n) * 4);
        }
        bf16x8_t a[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) a[h] = __builtin_bit_cast(bf16x8_t, ld16(xr + kk + 16 * g + 8 * h));
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] = mfma(a[h], st.frag(j, h, g), acc[j]);
      }
    }
    if (s0) __syncthreads();  // the previous sub-slice's sums have been read
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (4 * g + r >= nrows) continue;
      float* d = red[wave][4 * g + r];
      if constexpr (!MX) {
        *reinterpret_cast<f32x4_t*>(d + 8 * c) = f32x4_t{acc[0][r], acc[1][r], acc[2][r], acc[3][r]};
        *reinterpret_cast<f32x4_t*>(d + 8 * c + 4) = f32x4_t{acc[4][r], acc[5][r], acc[6][r], acc[7][r]};
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[16 * j + c] = acc[j][r];
      }
    }
    __syncthreads();
    for (int i = tid; i < kRows * kCols; i += NW * 64) {
      const int r = i / kCols, q = i % kCols;
      float gate = 0, up = 0;
      if (r < nrows) {
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          gate += red[w][r][q];
          up += red[w][r][kCols + q];
        }
      }
      // The product enters the second one as the sum of two bf16 numbers, 16 bits of it: the matrix cores are idle most
      // of the time, so the layer's bf16 rounding of a is not needed here.
      const float a = silu_f(gate) * up;
      const uint16_t hi = (uint16_t)pack_bf16x2(a, 0.0f);
      a_hi[r][s0 + q] = hi;
      a_lo[r][s0 + q] = (uint16_t)pack_bf16x2(a - bf16_to_f32(hi), 0.0f);
    }
  }
  __syncthreads();

  float* po[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) po[r] = part + ((int64_t)max(rows[4 * g + r], 0) * ns + sl) * emb;
  for (int n0 = wave * 128; n0 < emb; n0 += NW * 128) {
    f32x4_t acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = f32x4_t{0, 0, 0, 0};
    // emb is a multiple of 64: the last block may have 64 columns, the other half then computes on the first ones
    if constexpr (!MX) {
      const int n = n0 + 8 * c;
      const uint16_t* p = wt.wo + ((int64_t)e * mlp + m0 + 8 * g) * emb + (n < emb ? n : n0);
#pragma unroll 2
      for (int kk = 0; kk < width; kk += StepBf16::kK) {
        StepBf16 st;
        st.load(p + (int64_t)kk * emb, emb);
        const bf16x8_t ah = __builtin_bit_cast(bf16x8_t, ld16(&a_hi[c][kk + 8 * g]));
        const bf16x8_t al = __builtin_bit_cast(bf16x8_t, ld16(&a_lo[c][kk + 8 * g]));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bf16x8_t b = st.frag(j);
          acc[j] = mfma(al, b, mfma(ah, b, acc[j]));
        }
      }
      if (n >= emb) continue;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (4 * g + r >= nrows) continue;
        *reinterpret_cast<f32x4_t*>(po[r] + n) = f32x4_t{acc[0][r], acc[1][r], acc[2][r], acc[3][r]};
        *reinterpret_cast<f32x4_t*>(po[r] + n + 4) = f32x4_t{acc[4][r], acc[5][r], acc[6][r], acc[7][r]};
      }
    } else {
      const uint8_t* p = wt.woc + ((int64_t)e * emb + n0 + c) * mlp + m0 + 16 * g;
      const uint8_t* q = wt.wos + ((int64_t)e * (mlp / 64) * emb + n0 + c) * 4;
#pragma unroll 2
      for (int kk = 0; kk < width; kk += StepMx::kK) {
        StepMx st;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int n = n0 + 16 * j < emb ? 16 * j : 16 * (j - 4);
          st.load(j, p + (int64_t)n * mlp + kk, q + ((int64_t)((m0 + kk) / 64) * emb + n) * 4);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bf16x8_t ah = __builtin_bit_cast(bf16x8_t, ld16(&a_hi[c][kk + 16 * g + 8 * h]));
          const bf16x8_t al = __builtin_bit_cast(bf16x8_t, ld16(&a_lo[c][kk + 16 * g + 8 * h]));
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const bf16x8_t b = st.frag(j, h, g);
            acc[j] = mfma(al, b, mfma(ah, b, acc[j]));
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (4 * g + r >= nrows) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (n0 + 16 * j < emb) po[r][n0 + 16 * j + c] = acc[j][r];
      }
    }
  }
}

// ---------------------------------------------------------------- sum

// y[t] = sum over the picks of w times the sum of their slices' shares; 16 waves share a token's rows of 256 columns.
constexpr int kSumWaves = 16;

__global__ __launch_bounds__(kSumWaves * 64) void few_sum_kernel(int k, int emb, int E, int ns,
                                                                 const float* __restrict__ part,
                                                                 const int32_t* __restrict__ topk_idx,
                                                                 const float* __restrict__ topk_w,
                                                                 uint16_t* __restrict__ y) {
  __shared__ f32x4_t red[kSumWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = blockIdx.y;
  const int n = blockIdx.x * 256 + 4 * lane;
  const int nc = n < emb ? n : 0;
  f32x4_t acc = {0, 0, 0, 0};
  const float* p = part + (int64_t)t * k * ns * emb + nc;
#pragma unroll 8
  for (int r = wave; r < k * ns; r += kSumWaves) {
    const int j = t * k + r / ns;
    // an expert id out of range has no share
    const float w = (unsigned)topk_idx[j] < (unsigned)E ? topk_w[j] : 0.0f;
    const f32x4_t v = *reinterpret_cast<const f32x4_t*>(p + (int64_t)r * emb);
    if ((unsigned)topk_idx[j] < (unsigned)E) {
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(w, v[i], acc[i]);
    }
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (wave) return;
#pragma unroll
  for (int w = 1; w < kSumWaves; ++w) acc += red[w][lane];
  if (n < emb) st8(y + (int64_t)t * emb + n, u32x2_t{pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3])});
}

// Slices of mlp and cuts of emb in the router, from the shape alone (the workspace's size follows).
struct FewPlan {
  int slice, ns;       // mlp columns of a workgroup, workgroups of a tile
  int run, splits;     // rows of emb of a router wave, router workgroups along emb
  int tiles;           // most tiles of 16 rows that the routing can give
};

FewPlan few_plan(int64_t T, int emb, int mlp, int E, int k) {
  FewPlan p;
  const int S = (int)T * k, experts = S < E ? S : E;
  p.slice = kCols;
  while (2 * p.slice <= kFewMaxSlice && (int64_t)experts * ((mlp + 2 * p.slice - 1) / (2 * p.slice)) >= 512) p.slice *= 2;
  p.ns = (mlp + p.slice - 1) / p.slice;
  const int most = experts + S / kRows;
  p.tiles = most < S ? most : S;
  // 64 rows a wave, in at most 8 workgroups along emb
  const int ways = (emb + kLogitWaves * 64 - 1) / (kLogitWaves * 64);
  const int splits = ways < 8 ? ways : 8;
  p.run = ((emb + kLogitWaves * splits - 1) / (kLogitWaves * splits) + 3) / 4 * 4;
  p.splits = (emb + kLogitWaves * p.run - 1) / (kLogitWaves * p.run);
  return p;
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

size_t few_workspace(int64_t T, int emb, int mlp, int E, int k) {
  const FewPlan p = few_plan(T, emb, mlp, E, k);
  return up256((size_t)p.splits * T * E * 8) + up256((size_t)T * k * p.ns * emb * 4);
}

hipError_t launch_few(int64_t T, int emb, int mlp, int E, int k, const uint16_t* x, const float* wr, const float* bias,
                      int32_t* topk_idx, float* topk_w, const FewWeights& wt, uint16_t* y, void* ws, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const FewPlan p = few_plan(T, emb, mlp, E, k);
  double* logits = static_cast<double*>(ws);
  float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + up256((size_t)p.splits * T * E * 8));
  if (wr) {
    const dim3 grid((E + 15) / 16, p.splits), block(kLogitWaves * 64);
    const int nt = ((int)T + 15) / 16;
    if (nt == 1) few_logits_kernel<1><<<grid, block, 0, stream>>>((int)T, emb, E, p.run, x, wr, logits);
    else if (nt == 2) few_logits_kernel<2><<<grid, block, 0, stream>>>((int)T, emb, E, p.run, x, wr, logits);
    else few_logits_kernel<4><<<grid, block, 0, stream>>>((int)T, emb, E, p.run, x, wr, logits);
    few_topk_kernel<<<dim3((unsigned)T), dim3(64), 0, stream>>>((int)T, E, k, p.splits, logits, bias, topk_idx, topk_w);
  }
  const dim3 grid(p.tiles * p.ns);
  if (wt.wi)
    few_experts_kernel<false, 4><<<grid, dim3(256), 0, stream>>>((int)T * k, k, emb, mlp, E, p.slice, p.ns, x, topk_idx, wt,
                                                                 part);
  else
    few_experts_kernel<true, 4><<<grid, dim3(256), 0, stream>>>((int)T * k, k, emb, mlp, E, p.slice, p.ns, x, topk_idx, wt,
                                                                part);
  few_sum_kernel<<<dim3((emb + 255) / 256, (unsigned)T), dim3(kSumWaves * 64), 0, stream>>>(k, emb, E, p.ns, part, topk_idx,
                                                                                          topk_w, y);
  return hipGetLastError();
}

}  // namespace moe
