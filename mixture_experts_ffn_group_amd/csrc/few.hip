// The whole MoE FFN layer for a few tokens (a decode step): router, experts and
// combine without the permute and the 256-row tiles of the grouped GEMMs.
//
// With T <= 64 tokens the layer is a stream over the weights of the experts that
// have a token: 6 * emb * mlp bytes each in bf16, 3.2 in MXFP8, for 2 to 2 * T
// multiply-adds an element. So the kernels are built around the weight loads: 16
// bytes a lane and whole 128-byte lines, read once for all (up to 16 or 32) rows of
// the expert, two steps of 8 KB a wave in flight at all times. bf16 goes from its
// registers straight into the matrix cores, MXFP8 through the wave's own LDS; there
// is no barrier but around the two sums between the products.
//
// Kernels: few_logits (64-bit sums on the fp64 matrix cores, cut along emb);
// few_topk (one wave a token; for up to 8 tokens the experts' kernel picks itself);
// few_experts (a workgroup per tile of an expert's rows and slice of mlp columns:
// gate/up, SwiGLU, and the slice's share of the down product; with few workgroups
// the two products in kernels of their own, cut further); few_sum (a token's shares,
// weighted). A slice's share is [rows, emb] fp32: adding it up in memory would need
// atomics, whose order changes results.
//
// Measured, us, kernels alone (weight bytes per second): one token, top-8 of 128, emb
// 2048, mlp 768: 3.5 + 13.8 + 8.4 + 4.2, launch and latency of four kernels; 4 tokens
// with 8 picks each, emb 7168, mlp 2048: experts 412 (6.5 TB/s), sum 5; 64 tokens,
// top-8 of 128, emb 2048, mlp 768: 7 + 5 + 203 (5.9 TB/s) + 6; 19 tokens with 8 picks
// each on MXFP8, emb 7168, mlp 2048: 6 + 5 + 477 (5.8 TB/s) + 13. What holds the long
// ones below a read's 7.2 TB/s: the shares (S * mlp / 128 * emb * 4 bytes, written and
// read again: 64 experts of emb 7168, mlp 2048 take 929 us with one row each, 1074 with
// eight), and workgroups that do not come out even over the compute units (6.2 TB/s
// with 512 of them, 5.8 with 640).
#include <math.h>

#include <type_traits>

#include "common.h"
#include "kernels.h"
#include "lanes.h"

namespace moe {
namespace {

typedef double f64x4_t __attribute__((ext_vector_type(4)));

constexpr int kSide = 16;          // rows of the matrix instruction; a tile has 16 or 32
constexpr int kMaxRows = 32;
constexpr int kWaves = 4;          // waves of a workgroup of the experts' kernels
constexpr int kFewMaxSlice = 128;  // most mlp columns of a workgroup
constexpr int kParts = 3;          // bf16 numbers that the SwiGLU output is the sum of

// ---------------------------------------------------------------- router

// logits[split][t][e] = sum over the split's rows of x[t, i] wr[i, e]. The products (8 + 24 bits) are exact in
// fp64 and the sums are off by 2^-53 a step, so picks are those of exact arithmetic but where logits lie within that.
// A wave takes 16 experts and 64 rows of emb at a time, all of whose loads are in flight at once (the kernel is one
// memory latency long). v_mfma_f64_16x16x4 has A[i = lane%16][k = lane/16], B[k = lane/16][j = lane%16] and
// D[i = 4r + lane/16][j = lane%16]; step i of the 16 takes row 16 (lane/16) + i of the 64.
constexpr int kLogitWaves = 4;

template <int NT>
__global__ __launch_bounds__(kLogitWaves * 64) void few_logits_kernel(int T, int emb, int E, int run,
                                                                     const uint16_t* __restrict__ x,
                                                                     const float* __restrict__ wr,
                                                                     double* __restrict__ out) {
  __shared__ double red[kLogitWaves][16][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  const int e = blockIdx.x * 16 + c;
  const int ec = e < E ? e : E - 1;  // columns past E are computed on the last one and not stored
  const int k0 = (blockIdx.y * kLogitWaves + wave) * run;
  const int k1 = min(k0 + run, emb);
  f64x4_t acc[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n] = f64x4_t{0, 0, 0, 0};
  for (int k = k0 + 16 * g; k < k1; k += 64) {  // emb and run are multiples of 64
    float b[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) b[i] = wr[(int64_t)(k + i) * E + ec];
    u32x4_t v[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int t = n * 16 + c;
      const uint16_t* xr = x + (int64_t)(t < T ? t : T - 1) * emb + k;
      v[n][0] = ld16(xr);
      v[n][1] = ld16(xr + 8);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const double w = (double)b[i];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint32_t d = v[n][i >> 3][(i >> 1) & 3];
        acc[n] = __builtin_amdgcn_mfma_f64_16x16x4f64((double)((i & 1) ? bf16_hi(d) : bf16_lo(d)), w, acc[n], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (n) __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][4 * r + g][c] = acc[n][r];
    __syncthreads();
    const int i = threadIdx.x;  // 256 of them
    const int t = n * 16 + (i >> 4), ee = blockIdx.x * 16 + (i & 15);
    if (t >= T || ee >= E) continue;
    double s = 0;
#pragma unroll
    for (int w = 0; w < kLogitWaves; ++w) s += red[w][i >> 4][i & 15];
    out[((int64_t)blockIdx.y * T + t) * E + ee] = s;
  }
}

// Order-preserving key of a logit, all 64 bits of it: larger logit, larger key, -0 like +0, NaN below -inf. 0 is no key.
constexpr uint64_t kNanKey = 1;
__device__ __forceinline__ uint64_t pick_key(double v) {
  if (v != v) return kNanKey;
  if (v == 0) v = 0;
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double pick_value(uint64_t k) {
  if (k <= kNanKey) return __builtin_nan("");
  return __longlong_as_double((long long)((k >> 63) ? (k & 0x7fffffffffffffffull) : ~k));
}
// The lane's four keys in descending order; equal ones stay in theirs, by id (neighbours change places only).
__device__ __forceinline__ void sort_picks(uint64_t (&key)[4], int (&id)[4]) {
#pragma unroll
  for (int last = 3; last > 0; --last) {
#pragma unroll
    for (int a = 0; a < last; ++a) {
      const bool sw = key[a + 1] > key[a];
      const uint64_t hi = sw ? key[a + 1] : key[a], lo = sw ? key[a] : key[a + 1];
      const int first = sw ? id[a + 1] : id[a], second = sw ? id[a] : id[a + 1];
      key[a] = hi, key[a + 1] = lo;
      id[a] = first, id[a + 1] = second;
    }
  }
}
// Largest value of the wave, in every lane: the rows' maxima meet in scalar registers.
__device__ __forceinline__ uint32_t wave_max_fused(uint32_t v) {
  v = row_max_fused(v);
  const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)v, 0), b = (uint32_t)__builtin_amdgcn_readlane((int)v, 16);
  const uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)v, 32), d = (uint32_t)__builtin_amdgcn_readlane((int)v, 48);
  return max(max(a, b), max(c, d));
}

// One wave picks token t's experts: lane j gets pick j and its logit (lanes past k: 0 and -inf).
__device__ __forceinline__ void few_pick(int T, int E, int k, int splits, int t, const double* __restrict__ logits,
                                         const float* __restrict__ bias, int lane, int& pick, double& logit) {
  // all of the cuts' sums in flight at once, in batches of 8 (cuts and experts that are not there load others')
  double sum[4] = {0, 0, 0, 0};
  const double* p = logits + (int64_t)t * E;
  const int64_t cut = (int64_t)T * E;
  for (int c0 = 0; c0 < splits; c0 += 8) {
    double v[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (64 * i >= E) continue;
#pragma unroll
      for (int c = 0; c < 8; ++c) v[i][c] = p[min(c0 + c, splits - 1) * cut + min(lane + 64 * i, E - 1)];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (64 * i >= E) continue;
#pragma unroll
      for (int c = 0; c < 8; ++c) sum[i] += c0 + c < splits ? v[i][c] : 0;
    }
  }
  uint64_t key[4];
  int id[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    id[i] = lane + 64 * i;
    key[i] = id[i] < E ? pick_key(bias ? sum[i] + (double)bias[id[i]] : sum[i]) : 0;
  }
  if (E > 64) sort_picks(key, id);
  uint64_t mine = 0;
  pick = 0;
  for (int j = 0; j < k; ++j) {
    const uint32_t hi = (uint32_t)(key[0] >> 32), lo = (uint32_t)key[0];
    const uint32_t mh = wave_max_fused(hi);
    uint64_t m = __ballot(hi == mh);
    if (m & (m - 1)) {  // several lanes, seldom
      const uint32_t ml = wave_max_fused(hi == mh ? lo : 0u);
      const bool top = hi == mh && lo == ml;
      m = __ballot(top);
      if (m & (m - 1)) {  // equal logits: the lowest id
        const uint32_t low = wave_max_fused(top ? 256u - (uint32_t)id[0] : 0u);
        m = __ballot(top && 256u - (uint32_t)id[0] == low);
      }
    }
    const int l = __builtin_ctzll(m);
    const uint32_t ml = (uint32_t)__builtin_amdgcn_readlane((int)lo, l);
    const int e = __builtin_amdgcn_readlane(id[0], l);
    if (lane == l) {
      key[0] = key[1], key[1] = key[2], key[2] = key[3], key[3] = 0;
      id[0] = id[1], id[1] = id[2], id[2] = id[3];
    }
    if (lane == j) mine = (uint64_t)mh << 32 | ml, pick = e;
  }
  logit = lane < k ? pick_value(mine) : -__builtin_inf();
}

// Weight of pick `lane`: the softmax over the k picks; 0 of a disabled expert (-inf or NaN), NaN where all logits are.
__device__ __forceinline__ float few_weight(int k, double logit, int lane) {
  const double l0 = __shfl(logit, 0);
  const double w = lane < k && logit > -__builtin_inf() ? exp(logit - l0) : 0.0;
  double s = w;
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) s += __shfl_xor(s, m);
  return l0 != l0 ? __builtin_nanf("") : s == 0 ? 0.0f : (float)(w / s);
}

__global__ __launch_bounds__(64) void few_topk_kernel(int T, int E, int k, int splits, const double* __restrict__ logits,
                                                      const float* __restrict__ bias, int32_t* __restrict__ topk_idx,
                                                      float* __restrict__ topk_w) {
  const int lane = threadIdx.x, t = blockIdx.x;
  int pick;
  double logit;
  few_pick(T, E, k, splits, t, logits, bias, lane, pick, logit);
  const float w = few_weight(k, logit, lane);
  if (lane < k) {
    topk_idx[t * k + lane] = pick;
    topk_w[t * k + lane] = w;
  }
}

// ---------------------------------------------------------------- experts

// Weights are read once and not again: non-temporal loads (a plain read of 4 GiB ran at 6.2 TB/s, a non-temporal one
// at 7.2).
__device__ __forceinline__ u32x4_t ldw16(const void* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p));
}

__device__ __forceinline__ f32x4_t mfma(bf16x8_t a, bf16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ bf16x8_t as_bf16(u32x4_t v) { return __builtin_bit_cast(bf16x8_t, v); }

// A wave reads weights in steps of 8 KB whose every load covers whole 128-byte lines (8 to a load: half-line requests
// cost half the rate, 3.7 against 6.7 TB/s). The matrix instruction is v_mfma_f32_16x16x32_bf16: A[row lane%16]
// [k 8*(lane/16) + i], B[k][column lane%16], D[row 4*(lane/16) + r][column lane%16]; g = lane/16, c = lane%16. The rows'
// part (x, the A operand) is loaded with the weights, so that waiting for it does not wait for the loads issued after it.
//
// bf16, row-major [K, N], 128 columns by 32 rows: the lane loads columns 8c..8c+7 of rows 8g..8g+7 (of the first
// product, c < 8 gate and c >= 8 up columns). Product j takes column 8c + j of every lane; its 8 values along K lie in
// the lane's 8 rows, and one byte permute puts two of them into a register: the B operand comes straight from the
// registers that were loaded.
struct StepBf16 {
  u32x4_t v[8];
  __device__ __forceinline__ void load(const char* p, int64_t ld, uint32_t lane) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = ldw16(p + i * ld + lane);
  }
  __device__ __forceinline__ bf16x8_t col(int j) const {
    const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
    u32x4_t r;
#pragma unroll
    for (int p = 0; p < 4; ++p) r[p] = __builtin_amdgcn_perm(v[2 * p + 1][j >> 1], v[2 * p][j >> 1], sel);
    return as_bf16(r);
  }
};

// MXFP8, K-contiguous [N, K], 64 columns by 128 values of K. Product t takes column 4c + t of every lane, so that a lane
// ends up with four neighbouring results. Load j covers columns (j & 3) + 32 (j >> 2) + 4 r8, r8 = lane / 8, 16 codes a
// lane: the lanes of a column hold its K side by side, where the matrix instruction wants columns side by side. The step
// goes through the wave's own 8 KB of LDS, row 16t + c for column 4c + t, from where lane (g, c) reads codes 16(4p + g)...
// Within a row the 16-byte units are stored at u ^ (row & 7), so that both the writes and the reads spread over the banks;
// the swizzle is in the address the lane loads from. `scale` holds the dwords of the 64 columns for the step's two
// 64-blocks. Codes convert to bf16 exactly (3 bits of mantissa), but to multiples of 2^-133 below scale code 3, which only
// blocks of weights below 2^-116 have; a scale code above 246 leaves bf16's range.
// Slices of 64 mlp columns give the second product rows of 64 bytes: 128 columns by 64 values of K then, in the
// operand's own order (v[j]: column 64 (j >> 2) + 4c + (j & 3), codes 16g..), through plain loads.
struct StepMx {
  u32x4_t v[8];
  uint32_t scale[2];
};

__device__ __forceinline__ bf16x8_t mx_values(u32x4_t codes, int h, uint32_t code) {
  // the conversion's scale operand is a float of which it takes the exponent
  const float s = __uint_as_float((code & 0xffu) << 23);
  u32x4_t r;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    r[2 * p] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[2 * h + p], s, false));
    r[2 * p + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[2 * h + p], s, true));
  }
  return as_bf16(r);
}

// Finds tile `tile`: up to ROWS slots (t*k + j) of one expert, in slot order. Lane r < ROWS gets row r's slot.
//
// Up to 64 slots, slot l's expert in lane l: every wave by itself, in registers. A slot whose rank among its expert's
// is a multiple of ROWS starts a tile.
template <int ROWS>
__device__ __forceinline__ void find_tile64(int S, int E, int tile, int e, int lane, int& te, int& tn,
                                            int& slot) {
  const bool valid = lane < S && (unsigned)e < (unsigned)E;
  for (int j = 0; j < S; ++j) {
    const int ej = __builtin_amdgcn_readlane(e, j);
    if ((unsigned)ej >= (unsigned)E) continue;
    const uint64_t m = __ballot(valid && e == ej);
    const int rank = popc64(m & ((1ull << j) - 1));
    if (rank % ROWS || tile--) continue;
    const int r = popc64(m & ((1ull << lane) - 1)) - rank;
    const bool in = valid && e == ej && r >= 0 && r < ROWS;
    // lanes outside send to lane 63, which is no row's
    slot = __builtin_amdgcn_ds_permute((in ? r : 63) * 4, lane);
    te = ej;
    tn = min(ROWS, popc64(m) - rank);
    break;
  }
}

// Any number of slots, through LDS; tiles go by expert. Called by the whole workgroup.
template <int ROWS>
__device__ __forceinline__ void find_tile(int S, int E, int tile, const int32_t* __restrict__ idx, int* cnt, int* found,
                                          int* rows, int& te, int& tn, int& slot) {
  const int tid = threadIdx.x, lane = tid & 63;
  for (int i = tid; i < kMaxExperts; i += kWaves * 64) cnt[i] = 0;
  if (tid == 0) found[0] = -1;
  __syncthreads();
  for (int i = tid; i < S; i += kWaves * 64) {
    const int e = idx[i];
    if ((unsigned)e < (unsigned)E) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  if (tid < 64) {
    int base = 0;
    for (int q = 0; q < E; q += 64) {
      const int n = (cnt[q + lane] + ROWS - 1) / ROWS;
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
  const int r0 = found[1] * ROWS;
  if (tid < 64) {
    int base = 0;
    for (int q = 0; q < S; q += 64) {
      const bool mine = q + lane < S && idx[q + lane] == e;
      const uint64_t m = __ballot(mine);
      const int r = base + popc64(m & ((1ull << lane) - 1)) - r0;
      if (mine && r >= 0 && r < ROWS) rows[r] = q + lane;
      base += popc64(m);
    }
  }
  __syncthreads();
  te = e;
  tn = min(ROWS, cnt[e] - r0);
  slot = rows[lane < tn ? lane : 0];
}

struct FewArgs {
  int T, k, emb, mlp, E, slice, ns, blocks, splits;
  const uint16_t* x;
  const double* logits;  // PICK: the picks are made here
  const float* bias;
  int32_t* topk_idx;
  float* topk_w;
  FewWeights wt;
  float* part;
  // the products in kernels of their own: cuts of emb (rows of each) and of the output columns; hpart: the first one's
  // sums [slot][slice][cut][64 gate, 64 up]
  int cuts, run, cuts2;
  float* hpart;
};

// Workgroup (tile, slice): the tile's rows, and `slice` (64 or 128) of its expert's mlp columns, 64 at a time in the
// first product. The waves share the contraction of the first product (emb) and add up through LDS; of the second (over
// the slice's columns) each takes output columns. part[slot][slice][emb] receives the slice's share of the slot's
// output row.
//
// A wave's weight steps, those of the first product and then those of the second, form one sequence of which two are
// always in flight, over the barriers between the products too: the second product's first weights arrive while the
// first one's sums go through LDS.
// PART: kFused, both products; or, where that gives less than a workgroup a compute unit, kFirst and kSecond in kernels
// of their own, the first one's contraction (emb) and the second one's columns cut over blockIdx.y.
// PICK (T <= 8, T*k <= 64): every workgroup first picks the experts from the logits, a wave a token, instead of
// waiting for another kernel to do it; workgroup 0 writes the routing.
enum { kFused = 0, kFirst = 1, kSecond = 2 };
constexpr int kMaxCuts = 8;

// Each part holds what it uses, so that three workgroups of a cut product fit a compute unit on tiles of 32 rows too.
template <int PART, int ROWS, bool MX>
struct FewLds {
  static constexpr int kRows = ROWS;
  union {
    // first product: each wave's sums; MXFP8: before and after, the wave's step
    float red[PART == kSecond && !MX ? 1 : kWaves][kSide][128];
    struct {                    // before both: the search for the tile
      int cnt[kMaxExperts], found[2], picks[64];
    };
  };
  uint16_t a[PART == kFirst ? 1 : kParts][ROWS][PART == kFirst ? 8 : kFewMaxSlice + 8];
  int rows[kMaxRows];
  int64_t share[kMaxRows];  // where each row's share starts in part
};

// Which rows, of which expert. False: the routing has no such tile.
template <bool PICK, class Lds>
__device__ __forceinline__ bool few_tile(const FewArgs& q, int tile, Lds& lds, int lane, int wave, int& e, int& nrows, int& slot) {
  constexpr int ROWS = Lds::kRows;
  e = -1;
  nrows = slot = 0;
  const int S = q.T * q.k;
  if constexpr (PICK) {
    for (int t = wave; t < q.T; t += kWaves) {
      int pick;
      double logit;
      few_pick(q.T, q.E, q.k, q.splits, t, q.logits, q.bias, lane, pick, logit);
      if (lane < q.k) lds.picks[t * q.k + lane] = pick;
      if (blockIdx.x == 0 && blockIdx.y == 0) {
        const float w = few_weight(q.k, logit, lane);
        if (lane < q.k) {
          q.topk_idx[t * q.k + lane] = pick;
          q.topk_w[t * q.k + lane] = w;
        }
      }
    }
    __syncthreads();
    find_tile64<ROWS>(S, q.E, tile, lane < S ? lds.picks[lane] : -1, lane, e, nrows, slot);
  } else if (S <= 64) {
    find_tile64<ROWS>(S, q.E, tile, lane < S ? q.topk_idx[lane] : -1, lane, e, nrows, slot);
  } else {
    find_tile<ROWS>(S, q.E, tile, q.topk_idx, lds.cnt, lds.found, lds.rows, e, nrows, slot);
  }
  __syncthreads();  // the search is over, its LDS free
  e = __builtin_amdgcn_readfirstlane(e);
  nrows = __builtin_amdgcn_readfirstlane(nrows);
  return e >= 0;
}

// silu(g) = g * sigmoid(g) to a few steps of fp32, with no exponential past fp32's range.
__device__ __forceinline__ float few_silu(float g) {
  const float e = expf(-__builtin_fabsf(g));
  return (g < 0 ? g * e : g) / (1.0f + e);
}

// Row r, column n of the second product's left operand. It enters as the sum of three bf16 numbers, which is all of
// fp32's 24 bits: the matrix cores are idle most of the time, so nothing is rounded here. (Elements of y that are not the
// rounded 64-bit result, 64 tokens of emb 2048, mlp 768, top-8 of 128: 41 of 131072; fp32 operations one after another:
// 66; with two numbers, 16 bits: 340.)
template <class Lds>
__device__ __forceinline__ void few_set_a(Lds& lds, int r, int n, float gate, float up) {
  float a = few_silu(gate) * up;
#pragma unroll
  for (int p = 0; p < kParts; ++p) {
    const uint16_t v = (uint16_t)pack_bf16x2(a, 0.0f);
    lds.a[p][r][n] = v;
    // past bf16's range the others are 0: inf - inf would make the row NaN
    a = (v & 0x7f80) == 0x7f80 ? 0.0f : a - bf16_to_f32(v);
  }
}

// The waves' sums of 64 gate and 64 up columns of rows r0.. -> SwiGLU -> a's columns s0...
template <class Lds>
__device__ __forceinline__ void few_swiglu(Lds& lds, int nrows, int r0, int s0) {
  for (int i = threadIdx.x; i < kSide * 64; i += kWaves * 64) {
    const int r = i >> 6, n = i & 63;
    float gate = 0, up = 0;
    if (r0 + r < nrows) {
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        gate += lds.red[w][r][n];
        up += lds.red[w][r][64 + n];
      }
    }
    few_set_a(lds, r0 + r, s0 + n, gate, up);
  }
}

// kFirst: the waves' sums to hpart.
template <class Lds>
__device__ __forceinline__ void few_store_h(const FewArgs& q, const Lds& lds, int nrows, int r0, int sl) {
  for (int i = threadIdx.x; i < min(kSide, nrows - r0) * 128; i += kWaves * 64) {
    const int r = i >> 7, n = i & 127;
    float h = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) h += lds.red[w][r][n];
    q.hpart[(((int64_t)lds.rows[r0 + r] * q.ns + sl) * q.cuts + blockIdx.y) * 128 + n] = h;
  }
}

// kSecond: hpart -> SwiGLU -> a.
template <class Lds>
__device__ __forceinline__ void few_load_h(const FewArgs& q, Lds& lds, int nrows, int sl) {
  const int n = threadIdx.x & 63;
#pragma unroll
  for (int it = 0; it < Lds::kRows / kWaves; ++it) {
    if (it * kWaves >= nrows) continue;  // rows past the last: their results are not used
    const int r = it * kWaves + (threadIdx.x >> 6);
    const float* h = q.hpart + ((int64_t)lds.rows[r < nrows ? r : 0] * q.ns + sl) * q.cuts * 128 + n;
    float g[kMaxCuts], u[kMaxCuts];
#pragma unroll
    for (int i = 0; i < kMaxCuts; ++i) {
      const int at = min(i, q.cuts - 1) * 128;
      g[i] = h[at];
      u[i] = h[at + 64];
    }
    float gate = 0, up = 0;
#pragma unroll
    for (int i = 0; i < kMaxCuts; ++i)
      if (i < q.cuts && r < nrows) gate += g[i], up += u[i];
    few_set_a(lds, r, n, gate, up);
  }
}

__device__ __forceinline__ const char* bytes(const void* p) { return static_cast<const char*>(p); }

// The second product alone runs three workgroups a compute unit on tiles of 32 rows too, though three registers of the 172
// it would take are then kept in memory: 64 tokens, top-1 of 4, emb 4096, mlp 2048: 74.5 us against 79.5 with two.
template <int PART, bool WIDE, bool PICK, int R>
__global__ __launch_bounds__(kWaves * 64, R == 1 || PART == kSecond ? 3 : 2) void few_experts_kernel(FewArgs q) {
  constexpr int kRows = R * kSide;
  __shared__ __align__(16) FewLds<PART, kRows, false> lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int emb = q.emb, mlp = q.mlp;
  const int tile = blockIdx.x / q.ns, sl = blockIdx.x - tile * q.ns;
  int e, nrows, slot;
  if (!few_tile<PICK>(q, tile, lds, lane, wave, e, nrows, slot)) return;
  const int m0 = sl * q.slice, width = min(q.slice, mlp - m0);
  // lanes past the last row compute on the first one; their rows of the results are not used
  uint32_t xlane[R];
#pragma unroll
  for (int m = 0; m < R; ++m)
    xlane[m] = 2 * ((uint32_t)__shfl(slot, m * kSide + c < nrows ? m * kSide + c : 0) / (uint32_t)q.k * (uint32_t)emb + 8 * g);
  // read after a barrier
  if (wave == 0 && lane < kRows) lds.share[lane] = ((int64_t)slot * q.ns + sl) * emb, lds.rows[lane] = slot;

  // The sequence of a wave's steps: n1 pairs of the first product (WIDE: a step for each 64 of the slice's 128 columns;
  // else two steps of its 64), then one step per 32 columns of the slice for each of its output blocks of 128 columns.
  // Steps past the wave's share, and past the end, load the same few words over and over: loads are never skipped, so
  // that the wait for a step counts on those behind.
  constexpr int kPair = WIDE ? 32 : 64;  // rows of emb in a pair
  const int kb = PART == kFirst ? blockIdx.y * q.run : 0, ke = PART == kFirst ? min(emb, kb + q.run) : emb;
  const int n1 = PART == kSecond ? 0 : (ke - kb + kWaves * kPair - 1) / (kWaves * kPair);
  const int nb = PART == kFirst ? emb : ((PART == kSecond ? blockIdx.y * kWaves : 0) + wave) * 128;  // the wave's blocks
  const int nstride = (PART == kSecond ? q.cuts2 : 1) * kWaves * 128;
  int lw = 0, ln = nb, lk = 0;
  const int64_t ld1 = 4 * (int64_t)mlp, ld2 = 2 * (int64_t)emb;  // bytes from row to row
  const uint32_t lane1 = 8 * g * (uint32_t)ld1 + 2 * (c < 8 ? 8 * c : mlp + 8 * (c - 8));
  const uint32_t lane2 = 8 * g * (uint32_t)ld2 + 16 * c;
  const auto load = [&](StepBf16& st, int u, auto x) {  // u: which of the pair; x: nullptr where it is not needed
    const bool first = PART == kFirst || (PART == kFused && lw < n1);
    const int k1 = kb + (lw * kWaves + wave) * kPair + (WIDE ? 0 : 32 * u);
    const bool real = first ? k1 < ke && (!WIDE || 64 * u < width) : ln < emb;
    // emb is a multiple of 64: the last block may have 64 columns, the other half then takes the first ones
    const uint32_t l2 = ln + 64 >= emb && c >= 8 ? lane2 - 128 : lane2;
    const char* p1 = bytes(q.wt.wi) + ((int64_t)e * emb + k1) * ld1 + 2 * (m0 + (WIDE ? 64 * u : 0));
    const char* p2 = bytes(q.wt.wo) + ((int64_t)e * mlp + m0 + lk) * ld2 + 2 * ln;
    st.load(real ? first ? p1 : p2 : bytes(q.x), real ? first ? ld1 : ld2 : 0, real ? first ? lane1 : l2 : 0);
    if constexpr (!std::is_same_v<decltype(x), std::nullptr_t>) {
      const char* xp = bytes(q.x) + (first && real ? 2 * k1 : 0);
#pragma unroll
      for (int m = 0; m < R; ++m) x[m] = ld16(xp + xlane[m]);
    }
    const bool wrap = lk + 32 >= width;
    lk = first ? lk : wrap ? 0 : lk + 32;
    ln = !first && wrap ? ln + nstride : ln;
    lw = u == 1 && first ? lw + 1 : lw;
  };

  // x of a pair's first step, which WIDE's second one shares, and of the second one
  StepBf16 st[2];
  u32x4_t xs[2][R];
  load(st[0], 0, &xs[0][0]);
  if constexpr (WIDE) load(st[1], 1, nullptr);
  else load(st[1], 1, &xs[1][0]);
  if constexpr (PART == kSecond) {
    __syncthreads();  // the slots
    few_load_h(q, lds, nrows, sl);
  }
  f32x4_t sum[WIDE ? 2 : 1][R][8];
#pragma unroll
  for (int u = 0; u < (WIDE ? 2 : 1); ++u)
#pragma unroll
    for (int m = 0; m < R; ++m)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[u][m][j] = f32x4_t{0, 0, 0, 0};
  for (int w = 0; w < n1; ++w) {
    const bool on = kb + (w * kWaves + wave) * kPair < ke;  // emb is a multiple of 64: both steps of a pair or none
    u32x4_t x[R];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int m = 0; m < R; ++m) x[m] = WIDE && u ? x[m] : xs[u][m];
      if (on) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bf16x8_t b = st[u].col(j);
#pragma unroll
          for (int m = 0; m < R; ++m) sum[WIDE ? u : 0][m][j] = mfma(as_bf16(x[m]), b, sum[WIDE ? u : 0][m][j]);
        }
      }
      if (WIDE && u) load(st[u], u, nullptr);
      else load(st[u], u, &xs[u][0]);
    }
  }
#pragma unroll
  for (int u = 0; u < (PART == kSecond ? 0 : WIDE ? 2 : 1); ++u) {
#pragma unroll
    for (int m = 0; m < R; ++m) {
      if (64 * u >= width) continue;
      if (u || m) __syncthreads();  // the sums before have been read
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (m * kSide + 4 * g + r >= nrows) continue;
        const f32x4_t* v = sum[u][m];
        float* d = &lds.red[wave][4 * g + r][8 * c];
        *reinterpret_cast<f32x4_t*>(d) = f32x4_t{v[0][r], v[1][r], v[2][r], v[3][r]};
        *reinterpret_cast<f32x4_t*>(d + 4) = f32x4_t{v[4][r], v[5][r], v[6][r], v[7][r]};
      }
      __syncthreads();
      if constexpr (PART == kFirst) few_store_h(q, lds, nrows, m * kSide, sl);
      else few_swiglu(lds, nrows, m * kSide, 64 * u);
    }
  }
  if constexpr (PART == kFirst) return;
  __syncthreads();

  f32x4_t acc[R][8];
  for (int n0 = nb; n0 < emb; n0 += nstride) {
#pragma unroll
    for (int m = 0; m < R; ++m)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[m][j] = f32x4_t{0, 0, 0, 0};
    for (int kk = 0; kk < width; kk += 64) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        bf16x8_t a[R][kParts];
#pragma unroll
        for (int m = 0; m < R; ++m)
#pragma unroll
          for (int p = 0; p < kParts; ++p) a[m][p] = as_bf16(ld16(&lds.a[p][m * kSide + c][kk + 32 * u + 8 * g]));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bf16x8_t b = st[u].col(j);
#pragma unroll
          for (int p = 0; p < kParts; ++p)
#pragma unroll
            for (int m = 0; m < R; ++m) acc[m][j] = mfma(a[m][p], b, acc[m][j]);
        }
        load(st[u], u, nullptr);
      }
    }
    wave_lds_fence();  // `share` is read again, not kept in registers
    const int n = n0 + 8 * c;
    if (n >= emb) continue;
#pragma unroll
    for (int m = 0; m < R; ++m) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = m * kSide + 4 * g + r;
        if (row >= nrows) continue;
        const f32x4_t* v = acc[m];
        float* d = q.part + lds.share[row] + n;
        *reinterpret_cast<f32x4_t*>(d) = f32x4_t{v[0][r], v[1][r], v[2][r], v[3][r]};
        *reinterpret_cast<f32x4_t*>(d + 4) = f32x4_t{v[4][r], v[5][r], v[6][r], v[7][r]};
      }
    }
  }
}

// The same on MXFP8 weights.
template <int PART, bool PICK, int R>
__global__ __launch_bounds__(kWaves * 64, 2) void few_experts_mx_kernel(FewArgs q) {
  constexpr int kRows = R * kSide;
  __shared__ __align__(16) FewLds<PART, kRows, true> lds;
  __shared__ uint32_t scale[kWaves][2][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int emb = q.emb, mlp = q.mlp;
  int b = blockIdx.x;
  if (q.slice == 64) {
    // two slices share each 128-byte line of wo: blocks b and b + 8 run on the same XCD
    b = (b & ~15) | ((b & 7) << 1) | ((b >> 3) & 1);
    if (b >= q.blocks) return;
  }
  const int tile = b / q.ns, sl = (b - tile * q.ns + (q.slice == 64 ? 0 : tile)) % q.ns;
  int e, nrows, slot;
  if (!few_tile<PICK>(q, tile, lds, lane, wave, e, nrows, slot)) return;
  const int m0 = sl * q.slice, width = min(q.slice, mlp - m0);
  const bool narrow = width == 64;  // of the second product's steps
  uint32_t xlane[R];
#pragma unroll
  for (int m = 0; m < R; ++m)
    xlane[m] = 2 * ((uint32_t)__shfl(slot, m * kSide + c < nrows ? m * kSide + c : 0) / (uint32_t)q.k * (uint32_t)emb + 16 * g);
  // read after a barrier
  if (wave == 0 && lane < kRows) lds.share[lane] = ((int64_t)slot * q.ns + sl) * emb, lds.rows[lane] = slot;

  // The sequence: for each 64 columns, n1 pairs of steps (gate, up) of 128 values of emb; then output blocks of 128
  // columns, one narrow or two wide steps each, an even number in all.
  const int kb = PART == kFirst ? blockIdx.y * q.run : 0, ke = PART == kFirst ? min(emb, kb + q.run) : emb;
  const int n1 = PART == kSecond ? 0 : (ke - kb + kWaves * 128 - 1) / (kWaves * 128);
  const int nb = PART == kFirst ? emb : ((PART == kSecond ? blockIdx.y * kWaves : 0) + wave) * 128;  // the wave's blocks
  const int nstride = (PART == kSecond ? q.cuts2 : 1) * kWaves * 128;
  const uint32_t r8 = lane >> 3, unit = (lane & 7) ^ r8;  // wide: the lane's column of a load, and its unit
  int ls = 0, lw = 0, ln = nb;
  const auto load = [&](StepMx& st, int u, auto x) {  // u: which of the pair; x: nullptr where it is not needed
    const bool first = PART == kFirst || (PART == kFused && ls < width);
    const int k1 = kb + (lw * kWaves + wave) * 128;
    const bool real = first ? ls < width && k1 < ke : ln < emb;
    const int64_t ld = first ? emb : mlp;
    // wide: the first column, and the values of K that are there (emb is a multiple of 64)
    const int n = first ? m0 + ls + (u ? mlp : 0) : ln + (narrow ? 0 : 64 * u);
    const bool there = first || n < emb;  // the last output block may have 64 columns
    const bool half = first && k1 + 64 >= emb;
    const int64_t row = (int64_t)e * (first ? 2 * mlp : emb) + (there ? n : ln);
    const char* p = (first ? bytes(q.wt.wic) : bytes(q.wt.woc)) + row * ld + (first ? k1 : m0);
    const int64_t planes = first ? 2 * mlp : emb;
    const char* s = (first ? bytes(q.wt.wis) : bytes(q.wt.wos)) +
                    (((int64_t)e * (ld / 64) + (first ? k1 : m0) / 64) * planes + (there ? n : ln)) * 4;
    const bool direct = !first && narrow;
    uint32_t lo = direct ? 4 * c * (uint32_t)mlp + 16 * g : 4 * r8 * (uint32_t)ld + 16 * (half ? unit & 3 : unit);
    int64_t step = ld;
    // columns 64..127 of a narrow step may not be there
    int64_t upper = !direct ? 32 * ld : ln + 64 >= emb ? 0 : 64 * ld;
    int64_t plane = direct ? (ln + 64 >= emb ? 0 : 256) : half ? 0 : 4 * planes;
    if (!real) p = bytes(q.wt.wic), s = bytes(q.wt.wis), step = upper = plane = 0, lo = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      st.v[j] = ldw16(p + j * step + lo);
      st.v[4 + j] = ldw16(p + upper + j * step + lo);
    }
    st.scale[0] = *reinterpret_cast<const uint32_t*>(s + 4 * lane);
    st.scale[1] = *reinterpret_cast<const uint32_t*>(s + plane + 4 * lane);
    if constexpr (!std::is_same_v<decltype(x), std::nullptr_t>) {
      const char* xp = bytes(q.x) + (first && real ? 2 * k1 : 0);
      const int xh = half || !real || !first ? 0 : 128;
#pragma unroll
      for (int m = 0; m < R; ++m) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          x[m][h] = ld16(xp + xlane[m] + 16 * h);
          x[m][2 + h] = ld16(xp + xh + xlane[m] + 16 * h);
        }
      }
    }
    const bool wrap = lw + 1 == n1;
    const bool pair = u == 1;
    ls = first && pair && wrap ? ls + 64 : ls;
    lw = !first || !pair ? lw : wrap ? 0 : lw + 1;
    ln = !first && (narrow || pair) ? ln + nstride : ln;
  };
  // wide step -> LDS; then 16 codes (unit 4p + g) of product t's column, and their scale code
  u32x4_t* my = reinterpret_cast<u32x4_t*>(lds.red[wave]);
  const auto stage = [&](const StepMx& st) {
    wave_lds_fence();
#pragma unroll
    for (int j = 0; j < 8; ++j) my[128 * (j & 3) + 64 * (j >> 2) + lane] = st.v[j];
    scale[wave][0][lane] = st.scale[0];
    scale[wave][1][lane] = st.scale[1];
    wave_lds_fence();
  };
  const auto codes = [&](int t, int p) { return my[(16 * t + c) * 8 + ((4 * p + g) ^ (c & 7))]; };
  const auto code_of = [&](uint32_t d) { return (g & 2) ? d >> 8 : d; };

  StepMx st[2];
  u32x4_t xs[R][4];  // both of a pair multiply the same x
  load(st[0], 0, &xs[0]);
  load(st[1], 1, nullptr);
  if constexpr (PART == kSecond) {
    __syncthreads();  // the slots
    few_load_h(q, lds, nrows, sl);
    __syncthreads();
  }
  f32x4_t acc[R][8];
  const auto clear = [&]() {
#pragma unroll
    for (int m = 0; m < R; ++m)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[m][j] = f32x4_t{0, 0, 0, 0};
  };
  for (int s0 = 0; s0 < (PART == kSecond ? 0 : width); s0 += 64) {
    clear();
    for (int w = 0; w < n1; ++w) {
      const int k1 = kb + (w * kWaves + wave) * 128;
      u32x4_t x[R][4];
#pragma unroll
      for (int m = 0; m < R; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[m][i] = xs[m][i];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (k1 < ke) {
          stage(st[u]);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            if (p && k1 + 64 >= emb) continue;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const u32x4_t v = codes(t, p);
              const uint32_t s = code_of(scale[wave][p][4 * c + t]);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const bf16x8_t b = mx_values(v, h, s);
#pragma unroll
                for (int m = 0; m < R; ++m) acc[m][4 * u + t] = mfma(as_bf16(x[m][2 * p + h]), b, acc[m][4 * u + t]);
              }
            }
          }
        }
        if (u) load(st[u], u, nullptr);
        else load(st[u], u, &xs[0]);
      }
    }
    // the wave's own LDS from here on holds its sums, until all have read them
    wave_lds_fence();
#pragma unroll
    for (int m = 0; m < R; ++m) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (m * kSide + 4 * g + r >= nrows) continue;
        const f32x4_t* v = acc[m];
        float* d = &lds.red[wave][4 * g + r][4 * c];
        *reinterpret_cast<f32x4_t*>(d) = f32x4_t{v[0][r], v[1][r], v[2][r], v[3][r]};
        *reinterpret_cast<f32x4_t*>(d + 64) = f32x4_t{v[4][r], v[5][r], v[6][r], v[7][r]};
      }
      __syncthreads();
      if constexpr (PART == kFirst) few_store_h(q, lds, nrows, m * kSide, sl);
      else few_swiglu(lds, nrows, m * kSide, s0);
      __syncthreads();
    }
  }
  if constexpr (PART == kFirst) return;

  // acc[.][j] += a times v
  const auto multiply = [&](const bf16x8_t (&a)[R][kParts], bf16x8_t v, int j) {
#pragma unroll
    for (int p = 0; p < kParts; ++p)
#pragma unroll
      for (int m = 0; m < R; ++m) acc[m][j] = mfma(a[m][p], v, acc[m][j]);
  };
  const auto a_of = [&](int k, bf16x8_t (&a)[R][kParts]) {
#pragma unroll
    for (int m = 0; m < R; ++m)
#pragma unroll
      for (int p = 0; p < kParts; ++p) a[m][p] = as_bf16(ld16(&lds.a[p][m * kSide + c][k]));
  };
  const auto store = [&](int n0) {
    wave_lds_fence();  // `share` is read again, not kept in registers
#pragma unroll
    for (int m = 0; m < R; ++m) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = m * kSide + 4 * g + r;
        if (row >= nrows) continue;
        const f32x4_t* v = acc[m];
        float* d = q.part + lds.share[row] + n0 + 4 * c;
        *reinterpret_cast<f32x4_t*>(d) = f32x4_t{v[0][r], v[1][r], v[2][r], v[3][r]};
        if (n0 + 64 < emb) *reinterpret_cast<f32x4_t*>(d + 64) = f32x4_t{v[4][r], v[5][r], v[6][r], v[7][r]};
      }
    }
  };
  if (!narrow) {
    for (int n0 = nb; n0 < emb; n0 += nstride) {
      clear();
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        stage(st[u]);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            bf16x8_t a[R][kParts];
            a_of(64 * p + 16 * g + 8 * h, a);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              multiply(a, mx_values(codes(t, p), h, code_of(scale[wave][p][4 * c + t])), 4 * u + t);
            }
          }
        }
        load(st[u], u, nullptr);
      }
      store(n0);
    }
  } else {
    for (int n0 = nb; n0 < emb; n0 += 2 * nstride) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (n0 + u * nstride < emb) {
          clear();
          wave_lds_fence();
          scale[wave][0][lane] = st[u].scale[0];
          scale[wave][1][lane] = st[u].scale[1];
          wave_lds_fence();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            bf16x8_t a[R][kParts];
            a_of(16 * g + 8 * h, a);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              multiply(a, mx_values(st[u].v[j], h, code_of(scale[wave][j >> 2][4 * c + (j & 3)])), j);
            }
          }
          store(n0 + u * nstride);
        }
        load(st[u], u, nullptr);
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
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), t = blockIdx.y;
  const int n = blockIdx.x * 256 + 4 * lane;
  const float* p = part + (int64_t)t * k * ns * emb + (n < emb ? n : 0);
  int id = -1;
  float w = 0;
  if (lane < k) id = topk_idx[t * k + lane], w = topk_w[t * k + lane];
  f32x4_t acc = {0, 0, 0, 0};
  const int rows = k * ns;
  constexpr int kBatch = 12;
  for (int r0 = wave; r0 < rows; r0 += kSumWaves * kBatch) {
    f32x4_t v[kBatch];
    const int jl = (r0 + lane * kSumWaves) / ns;  // lane i: the pick of the batch's row i
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = min(r0 + i * kSumWaves, rows - 1);
      v[i] = *reinterpret_cast<const f32x4_t*>(p + (int64_t)r * emb);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + i * kSumWaves;
      const int j = min(__builtin_amdgcn_readlane(jl, i), k - 1);
      const float wj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), j));
      // an expert id out of range has no share: its rows hold nothing; and a weight of 0 takes no part, whatever a
      // disabled expert's weights hold
      if (r < rows && (unsigned)__builtin_amdgcn_readlane(id, j) < (unsigned)E && wj != 0.0f) {
#pragma unroll
        for (int u = 0; u < 4; ++u) acc[u] = __builtin_fmaf(wj, v[i][u], acc[u]);
      }
    }
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (wave) return;
#pragma unroll
  for (int i = 1; i < kSumWaves; ++i) acc += red[i][lane];
  if (n < emb) st8(y + (int64_t)t * emb + n, u32x2_t{pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3])});
}

// Slices of mlp and cuts of emb in the router, from the shape alone (the workspace's size follows).
struct FewPlan {
  int slice, ns;       // mlp columns of a workgroup, workgroups of a tile
  int cuts, run1;      // of emb in the first product (rows of each); 1: both fused
  int cuts2;           // of the second one's columns
  int run, splits;     // rows of emb of a router wave, router workgroups along emb
  int rows, tiles;     // rows of a tile, most tiles that the routing can give
};

FewPlan few_plan(int64_t T, int emb, int mlp, int E, int k, bool mx) {
  FewPlan p;
  const int S = (int)T * k, experts = S < E ? S : E;
  // Rows of a tile: an expert with more reads its weights again for the next tile, but tiles of 32 leave half the
  // workgroups where 16 would have done. us, 16 against 32 rows, by the mean rows of an expert (emb 4096, mlp 14336, top-2
  // of 8): 8: 580 / 582, 12: 652 / 611, 16: 895 / 644; MXFP8 350 / 354, 397 / 379, 540 / 420; one expert (emb 2048, mlp
  // 8192), 32 tokens: 64 / 67 and MXFP8 53 / 67, 48 tokens: 97 / 74 and 80 / 63.
  p.rows = T > 2 * kSide && S >= 12 * E ? 2 * kSide : kSide;
  // Slices of 128 columns are read in longer runs and leave half the shares, slices of 64 give twice the workgroups, of
  // which three fit a compute unit, 768 in all. What counts are the workgroups with work: of the experts that T tokens of k
  // picks are expected to reach (they are not known here, and min(S, E) is more: 8 tokens of top-8 of 128 reach about 52).
  // us, slices of 64 against 128, by the workgroups that 128 gives these experts. emb 2048, mlp 768 or 1408: 174: 65 / 59,
  // 212: 73 / 70, 229: 72 / 71, 247: 84.6 / 86.0 (the picks scatter: past 256 some compute units get a second one), 273: 91
  // / 98, 279: 96 / 105, 309: 101 / 108, 314: 103 / 112, 351: 108 / 110, 365: 110 / 113, 384: 117 / 112 (64 gives more than
  // fit), 414: 125 / 116, 494: 145 / 133. emb 4096 and more, where a longer run counts for more: 240: 252 / 218, 279: 192 /
  // 203, 310: 203 / 207, 321: 265 / 260, 338: 357 / 352, 355: 282 / 274, 424: 424 / 384. On MXFP8 weights, whose rows of wo
  // are only 64 bytes long in slices of 64, by the most workgroups that 128 can give: 96: 37 / 48, 144: 50 / 50, 288: 81 /
  // 72, 576: 96 / 82.
  const int n128 = (mlp + 127) / 128;
  const int64_t wide = (int64_t)experts * n128;
  const double reached = E * (1 - pow(1 - (double)k / E, (double)T)) * n128;
  const bool one = reached <= (emb >= 4096 ? 256 : 244), past = reached >= (emb >= 4096 ? 320 : 376);
  p.slice = wide >= 144 && (mx || one || past) ? 128 : 64;
  p.ns = (mlp + p.slice - 1) / p.slice;
  // Few workgroups: the products in kernels of their own, cut along emb (in up to four, up to eight where that leaves few
  // workgroups still) and along the output columns. us fused and cut in four, by the workgroups fused: 8 (emb 7168, mlp
  // 128) 58 / 28, 18 (emb 4096, mlp 192) 44 / 25, 64 (emb 7168, mlp 2048) 93 / 44, 96 (emb 2048, mlp 768) 33 / 29, 128
  // (emb 2048, mlp 1024) 36 / 30, 144 (emb 2048, mlp 1152) 34.5 / 34.6, 160 (emb 7168, mlp 1280) 99 / 90, 192 (emb 2048,
  // mlp 768) 40 / 40 and (emb 4096, mlp 1536) 68 / 62; on MXFP8 weights the last four 28.7 / 32.1, 68 / 67, 31 / 37, 47 /
  // 48. In four and in eight: 16 (emb 4096, mlp 128) 24.1 / 22.1, 32 (emb 2048, mlp 256) 20.9 / 19.7, 64 (emb 7168, mlp
  // 512) 47 / 47, 96 (emb 4096, mlp 1536) 42.5 / 40.1, 128 (emb 2048, mlp 1024) 29.2 / 31.5. A cut leaves each of the
  // first product's waves a pair of steps at least: MXFP8 at emb 2048 loses by eight (96: 26.1 / 27.4).
  const int64_t filled = (S + p.rows - 1) / p.rows;
  const int64_t units = (experts > filled ? experts : filled) * p.ns;
  p.cuts = p.cuts2 = 1;
  p.run1 = emb;
  if (p.slice == 64 && units <= (!mx && emb >= 4096 ? 192 : 128) && emb >= 2 * 512) {
    const int most = units <= 96 ? kMaxCuts : 4, pairs = emb / (kWaves * (mx ? 128 : 64));
    const int cuts = pairs < most ? pairs : most;
    p.cuts2 = emb / (kWaves * 128) < 4 ? emb / (kWaves * 128) : 4;
    p.run1 = (emb + 128 * cuts - 1) / (128 * cuts) * 128;
    p.cuts = (emb + p.run1 - 1) / p.run1;
  }
  p.tiles = experts + S / p.rows < S ? experts + S / p.rows : S;
  // a router wave takes 64 rows of emb, more where that would cut emb into more than 16
  p.run = (emb + kLogitWaves * 16 * 64 - 1) / (kLogitWaves * 16 * 64) * 64;
  p.splits = (emb + kLogitWaves * p.run - 1) / (kLogitWaves * p.run);
  return p;
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

template <int PART, bool PICK, int R>
void launch_part(const FewArgs& q, hipStream_t st) {
  const dim3 block(kWaves * 64), grid(q.blocks, PART == kFirst ? q.cuts : PART == kSecond ? q.cuts2 : 1);
  if (!q.wt.wi)
    few_experts_mx_kernel<PART, PICK, R><<<dim3(q.slice == 64 ? (q.blocks + 15) / 16 * 16 : q.blocks, grid.y), block, 0, st>>>(q);
  else if (q.slice == 64)
    few_experts_kernel<PART, false, PICK, R><<<grid, block, 0, st>>>(q);
  else if constexpr (PART == kFused)
    few_experts_kernel<kFused, true, PICK, R><<<grid, block, 0, st>>>(q);
}

template <bool PICK, int R>
void launch_experts(const FewArgs& q, hipStream_t st) {
  if (q.cuts == 1) return launch_part<kFused, PICK, R>(q, st);
  launch_part<kFirst, PICK, R>(q, st);
  launch_part<kSecond, false, R>(q, st);
}

}  // namespace

size_t few_workspace(int64_t T, int emb, int mlp, int E, int k) {
  const FewPlan p = few_plan(T, emb, mlp, E, k, false), m = few_plan(T, emb, mlp, E, k, true);
  return up256((size_t)p.splits * T * E * 8) + up256((size_t)T * k * (p.ns > m.ns ? p.ns : m.ns) * emb * 4) +
         (p.cuts > 1 || m.cuts > 1 ? up256((size_t)T * k * (mlp / 64) * kMaxCuts * 128 * 4) : 0);
}

int64_t few_blocks(int64_t T, int emb, int mlp, int E, int k) {
  const FewPlan p = few_plan(T, emb, mlp, E, k, false), m = few_plan(T, emb, mlp, E, k, true);
  return (int64_t)p.tiles * (p.ns > m.ns ? p.ns : m.ns);
}

hipError_t launch_few(int64_t T, int emb, int mlp, int E, int k, const uint16_t* x, const float* wr, const float* bias,
                      int32_t* topk_idx, float* topk_w, const FewWeights& wt, uint16_t* y, void* ws, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const FewPlan p = few_plan(T, emb, mlp, E, k, !wt.wi);
  double* logits = static_cast<double*>(ws);
  float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + up256((size_t)p.splits * T * E * 8));
  float* hpart = part + up256((size_t)T * k * p.ns * emb * 4) / 4;
  const bool pick = wr && T <= 8 && T * k <= 64;
  if (wr) {
    const dim3 grid((E + 15) / 16, p.splits), block(kLogitWaves * 64);
    if (T <= 16) few_logits_kernel<1><<<grid, block, 0, stream>>>((int)T, emb, E, p.run, x, wr, logits);
    else if (T <= 32) few_logits_kernel<2><<<grid, block, 0, stream>>>((int)T, emb, E, p.run, x, wr, logits);
    else few_logits_kernel<4><<<grid, block, 0, stream>>>((int)T, emb, E, p.run, x, wr, logits);
    if (!pick)
      few_topk_kernel<<<dim3((unsigned)T), dim3(64), 0, stream>>>((int)T, E, k, p.splits, logits, bias, topk_idx, topk_w);
  }
  const FewArgs q{(int)T, k, emb, mlp, E, p.slice, p.ns, p.tiles * p.ns, p.splits, x, logits, bias, topk_idx, topk_w, wt, part,
                  p.cuts, p.run1, p.cuts2, hpart};
  if (pick) launch_experts<true, 1>(q, stream);
  else if (p.rows == kSide) launch_experts<false, 1>(q, stream);
  else launch_experts<false, 2>(q, stream);
  few_sum_kernel<<<dim3((emb + 255) / 256, (unsigned)T), dim3(kSumWaves * 64), 0, stream>>>(
      k, emb, E, p.ns, part, topk_idx, topk_w, y);
  return hipGetLastError();
}

}  // namespace moe
