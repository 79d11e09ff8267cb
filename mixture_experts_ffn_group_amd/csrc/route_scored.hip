// Routing by scores, and its gradient.
//
// With s = softmax(l) or sigmoid(l) of a token's logits and an optional balance
// bias b, the choice value of an expert is c = s + b. The E experts form
// n_group equal runs; a group's value is the sum of its group_top largest
// choice values, the topk_group best groups stay, and the k largest choice
// values in them are picked. The weights are the scores at the picks (the bias
// only steers the choice), renormalised to sum 1 if asked, times a scale.
//
// A disabled expert (logit -inf or NaN, bias -inf or NaN) has the choice value
// -inf and, picked for lack of others, the weight 0.
//
// Decisions are made on 64-bit choice values: neighbouring scores of 256
// experts are a few 1e-3 apart, so over 10^5 tokens some lie closer than the
// rounding of a 32-bit score, and the pick would hang on how the exponential
// was computed. Without a bias the order of the choice values is the order of
// the logits, which is exact.
#include "common.h"
#include "kernels.h"
#include "lanes.h"

namespace moe {
namespace {

constexpr int kMaxE = 256;

// Order-preserving key of a choice value: larger value -> larger key, -0 like
// +0. Every value's key is above 0, which marks an expert already taken.
__device__ __forceinline__ uint64_t order_key64(double v) {
  uint64_t u = (uint64_t)__double_as_longlong(v);
  if ((u << 1) == 0) u = 0;
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
constexpr uint64_t kKeyNegInf = 0x000fffffffffffffull;  // key of -inf

template <class V>
__device__ __forceinline__ float load_logit(const V* p);
template <>
__device__ __forceinline__ float load_logit<float>(const float* p) {
  return *p;
}
template <>
__device__ __forceinline__ float load_logit<uint16_t>(const uint16_t* p) {
  return bf16_to_f32(*p);
}

struct RouteP {
  int64_t T;
  int E, k;
  int score, n_group, topk_group, group_top, renorm;
  float scale;
  const float* bias;
  int32_t* idx;
  float* w;
};

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
  const uint32_t hi = wave_max_u32((uint32_t)(v >> 32));
  const uint32_t lo = wave_max_u32((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ int wave_min_i32(int v) { return (int)~wave_max_u32(~(uint32_t)v); }  // v >= 0
__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) v += __shfl_xor(v, s);
  return v;
}
__device__ __forceinline__ float wave_max_f32(float v) {
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) v = fmaxf(v, __shfl_xor(v, s));
  return v;
}

// One token on one wave, everything in 64 bits. The row's scores and keys stay
// in LDS (row_s, row_k [E], row_g [n_group], the wave's own) rather than in
// registers: the four-token kernel below runs this for few tokens, and the
// registers it would hold there cost that kernel half its waves.
template <class V>
__device__ void route_row_exact(const RouteP& p, int64_t t, const V* row, double* row_s, uint64_t* row_k,
                                uint64_t* row_g) {
  const int lane = threadIdx.x & 63;
  const int E = p.E;
  float mx = -INFINITY;
#pragma unroll 1
  for (int e = lane; e < E; e += 64) mx = fmaxf(mx, fmaxf(load_logit(row + e), -INFINITY));
  mx = wave_max_f32(mx);
  double sum = 0.0;
  wave_lds_fence();
#pragma unroll 1
  for (int e = lane; e < E; e += 64) {
    const float l = load_logit(row + e);
    double s = 0.0;
    if (l > -INFINITY) {  // false for NaN
      const double x = p.score == 0 ? (l == mx ? 0.0 : (double)l - (double)mx) : -(double)l;
      s = exp(x);
      if (p.score != 0) s = 1.0 / (1.0 + s);
    }
    row_s[e] = s;
    sum += s;
  }
  if (p.score == 0) sum = wave_sum_f64(sum);
  else sum = 1.0;
  const bool by_logit = p.group_top == 1 && !p.bias;  // group values that order as the logits
  wave_lds_fence();
#pragma unroll 1
  for (int e = lane; e < E; e += 64) {
    const float l = load_logit(row + e), b = p.bias ? p.bias[e] : 0.0f;
    const bool on = l > -INFINITY && b > -INFINITY;
    const double s = row_s[e] / sum;  // sum 0: no logit is on
    if (on) row_s[e] = s;
    row_k[e] = on ? order_key64(p.bias ? s + (double)b : (double)l) : kKeyNegInf;
  }
  wave_lds_fence();
  if (p.topk_group < p.n_group) {
    const int gs = E / p.n_group;
#pragma unroll 1
    for (int g = lane; g < p.n_group; g += 64) {
      uint64_t ka = 0, kb = 0;            // the two largest keys
      double a = 0.0, b = 0.0;            // and the two largest choice values of enabled experts
#pragma unroll 1
      for (int i = 0; i < gs; ++i) {
        const int e = g * gs + i;
        const uint64_t kk = row_k[e];
        if (kk <= kKeyNegInf) continue;
        const double v = row_s[e] + (p.bias ? (double)p.bias[e] : 0.0);
        if (kb == 0 && ka == 0) a = v;
        else if (kb == 0) b = v > a ? a : v, a = v > a ? v : a;
        else if (v > a) b = a, a = v;
        else if (v > b) b = v;
        kb = max(kb, min(ka, kk));
        ka = max(ka, kk);
      }
      const uint64_t top2 = kb != 0 ? order_key64(a + b) : (ka != 0 ? order_key64(a) : kKeyNegInf);
      row_g[g] = p.group_top == 2 ? top2 : (by_logit || ka == 0 ? (ka != 0 ? ka : kKeyNegInf) : order_key64(a));
    }
    wave_lds_fence();
    // a group stays if fewer than topk_group others come before it (4 groups a lane at most)
    uint32_t keep = 0;
#pragma unroll 1
    for (int i = 0, g = lane; g < p.n_group; ++i, g += 64) {
      const uint64_t mine = row_g[g];
      int before = 0;
#pragma unroll 1
      for (int h = 0; h < p.n_group; ++h) before += row_g[h] > mine || (row_g[h] == mine && h < g);
      if (before < p.topk_group) keep |= 1u << i;
    }
    wave_lds_fence();
#pragma unroll 1
    for (int i = 0, g = lane; g < p.n_group; ++i, g += 64) row_g[g] = (keep >> i) & 1;
    wave_lds_fence();
#pragma unroll 1
    for (int e = lane; e < E; e += 64)
      if (!row_g[e / gs]) row_k[e] = kKeyNegInf;
    wave_lds_fence();
  }
  int my_e = 0;
  double my_s = 0.0;
  uint64_t key[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) key[q] = lane + 64 * q < E ? row_k[lane + 64 * q] : 0ull;
#pragma unroll 1
  for (int j = 0; j < p.k; ++j) {
    uint64_t best = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) best = key[q] > best ? key[q] : best;
    best = wave_max_u64(best);
    int e = E - 1;
#pragma unroll
    for (int q = 3; q >= 0; --q)
      if (key[q] == best && lane + 64 * q < E) e = min(e, lane + 64 * q);
    e = wave_min_i32(e);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (e == lane + 64 * q) key[q] = 0ull;
    if (lane == j) {
      my_e = e;
      my_s = best > kKeyNegInf ? row_s[e] : 0.0;
    }
  }
  if (p.renorm) {
    const double tot = wave_sum_f64(my_s);
    my_s = tot > 0.0 ? my_s / tot : 0.0;
  }
  if (lane < p.k) {
    p.idx[t * p.k + lane] = my_e;
    p.w[t * p.k + lane] = (float)(my_s * (double)p.scale);
  }
  wave_lds_fence();
}

template <class V>
__global__ __launch_bounds__(256) void route_scored_kernel(RouteP p, const V* __restrict__ logits) {
  __shared__ double s_s[4][kMaxE];
  __shared__ uint64_t s_k[4][kMaxE], s_g[4][kMaxE];
  const int wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t < p.T) route_row_exact(p, t, logits + t * p.E, s_s[wave], s_k[wave], s_g[wave]);
}

// Four tokens a wave, token g of the group on lanes 16g .. 16g+15, for k <= 32.
//
// The choice runs on 28-bit integers: lane r holds experts 4 (r + 16 q) + i as
// keys value << 4 | (15 - (4 q + i)), so a sort is min and max only and a pick's
// key tells which of its lane's experts it is. Without a bias the value is
// (l - row maximum) in units of 2^-22, which never inverts the order of two
// logits; with one it is c in units of 2^-26 from 32-bit arithmetic, off by
// less than `thr` / 2 units. The picks stand if every pick and the first expert
// not picked differ from the next by more than thr. Otherwise (about one token
// in 1000 with a bias) the 16 best candidates are ranked by their exact values,
// one a lane; that needs 64-bit scores of 16 experts rather than all (softmax:
// and the 64-bit sum, 16 lanes a row). What is left goes to route_row_exact: a
// pick that is disabled, values out of the integers' range, more close values
// than candidates. Groups too close at the edge of
// those that stay are ranked the same way, by the exact scores of their two
// best. bf16 logits without a bias leave 16 bits for the expert itself: those
// keys are exact, ties included.
//
// Bound by the issue of vector instructions: per four tokens of 128 experts
// some 480 (of them 190 in the k = 8 rounds, 80 in the 64-bit weights) and no
// LDS without groups, against some 4000 of the 64-bit form a token. Measured:
// 32768 tokens x 128, softmax: 9.3 us (49 us with a token a wave in 64 bits);
// with a bias, where close values are frequent, 15.5 us; 8192 x 256, sigmoid,
// bias, 4 of 8 groups: 9.8 us (40 us), softmax, 13 to 17 us; 4 tokens x 256:
// 6.0 us (18 us), the latency of one wave. Their logits alone, at a copy's
// rate, take 4.0 and 1.9 us.
//
// "Out of the integers' range" is |c| >= 1.99 for any enabled expert of the row, picked or not: with a bias that
// puts one there, or a soft mask of -1e4 on one expert, every row goes to the 64-bit form: 8192 x 256 in groups 9.7 ->
// 62 to 81 us. (An expert disabled by a bias of -inf costs nothing.)
constexpr int kHalf28 = 1 << 27;

template <class V, int N>
__device__ __forceinline__ void load_row16(const V* row, int E, int r, float (&l)[N]) {
  const bool vec = (E & 3) == 0;
#pragma unroll
  for (int q = 0; q < N / 4; ++q) {
    const int e0 = 4 * (r + 16 * q);
    if (vec) {
      if (e0 < E) {
        if (sizeof(V) == 4) {
          const f32x4_t v = *reinterpret_cast<const f32x4_t*>(row + e0);
#pragma unroll
          for (int i = 0; i < 4; ++i) l[4 * q + i] = v[i];
        } else {
          const u32x2_t v = *reinterpret_cast<const u32x2_t*>(row + e0);
#pragma unroll
          for (int i = 0; i < 4; ++i) l[4 * q + i] = (i & 1) ? bf16_hi(v[i >> 1]) : bf16_lo(v[i >> 1]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) l[4 * q + i] = -INFINITY;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) l[4 * q + i] = e0 + i < E ? load_logit(row + e0 + i) : -INFINITY;
    }
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float row_max_f32(float v) {
  v = fmaxf(v, dpp_f32<0xb1>(v));
  v = fmaxf(v, dpp_f32<0x4e>(v));
  v = fmaxf(v, dpp_f32<0x141>(v));
  return fmaxf(v, dpp_f32<0x140>(v));
}
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 0xf, 0xf, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), CTRL, 0xf, 0xf, true);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ double row_sum_f64(double v) {
  v += dpp_f64<0xb1>(v);
  v += dpp_f64<0x4e>(v);
  v += dpp_f64<0x141>(v);
  return v + dpp_f64<0x140>(v);
}
__device__ __forceinline__ uint32_t row_min_u32(uint32_t v) { return ~row_max_fused(~v); }

// group values before this lane's own, over the 16 lanes of the row (rotations by 1 .. 15)
template <int S>
__device__ __forceinline__ int count_larger(uint32_t v) {
  const int c = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x120 + S, 0xf, 0xf, true) > v;
  if constexpr (S < 15) return c + count_larger<S + 1>(v);
  return c;
}

// the same by (value, lower id first), a total order: a rank
template <int S>
__device__ __forceinline__ int count_before(double v, int id) {
  const double ov = dpp_f64<0x120 + S>(v);
  const int oid = __builtin_amdgcn_mov_dpp(id, 0x120 + S, 0xf, 0xf, true);
  const int c = ov > v || (ov == v && oid < id);
  if constexpr (S < 15) return c + count_before<S + 1>(v, id);
  return c;
}

// CHOICE: the order is that of c (a bias, or group values that are sums of scores), else of the logits. NP picks a
// lane, pick 16 i + r on lane r; with two, close values go to the 64-bit form.
template <class V, int N, bool CHOICE, int NP>
__global__ __launch_bounds__(256) void route_scored16_kernel(RouteP p, const V* __restrict__ logits) {
  constexpr bool EXACT16 = sizeof(V) == 2 && !CHOICE;
  // a wave's row in the 64-bit form (scores, keys), or its four rows of 32-bit group values or keys
  __shared__ double s_x[4][2 * kMaxE];
  __shared__ uint64_t s_g[4][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, r = lane & 15;
  const int E = p.E, k = p.k;
  const bool groups = p.topk_group < p.n_group;
  // 2 x the error of c in 2^-26: sigmoid 20 units (exponential, 1 + e, reciprocal, + b, truncation);
  // softmax 100 (its sum, 20 additions); and none for logits
  const uint32_t thr = CHOICE ? (p.score == 0 ? 256u : 64u) : 0u;
  const int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * 4;
  if (t0 < p.T) {  // no loop over tokens: it would keep every 64-bit constant in registers
    const int64_t t = min(t0 + g, p.T - 1);
    const V* row = logits + t * E;
    float l[N];
    load_row16<V, N>(row, E, r, l);
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      l[i] = fmaxf(l[i], -INFINITY);  // NaN -> -inf
      mx = fmaxf(mx, l[i]);
    }
    mx = row_max_f32(mx);
    bool flag = !(fabsf(mx) < INFINITY);
    uint32_t key[N];
    if (CHOICE) {
      float c[N];
      if (p.score == 0) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          c[i] = __expf(l[i] - mx);
          sum += c[i];
        }
        sum = row_sum(sum);
        const float inv = __builtin_amdgcn_rcpf(sum);
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] *= inv;
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] = sigmoid_f(l[i]);
      }
      if (p.bias) {
        float b[N];
        load_row16<float, N>(p.bias, E, r, b);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          c[i] += b[i];
          if (!(b[i] > -INFINITY)) l[i] = -INFINITY;  // disabled by its bias
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const bool on = l[i] > -INFINITY;
        flag |= on && !(fabsf(c[i]) < 1.99f);
        const int v = (int)(__builtin_amdgcn_fmed3f(c[i], -1.995f, 1.995f) * 67108864.0f) + kHalf28;
        key[i] = on ? ((uint32_t)max(v, 1) << 4) | (uint32_t)(15 - i) : 0u;
      }
    } else if (EXACT16) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        uint32_t u = __float_as_uint(l[i]) >> 16;
        if ((u & 0x7fffu) == 0) u = 0;
        u = (u & 0x8000u) ? (~u & 0xffffu) : (u | 0x8000u);
        const int e = 4 * (r + 16 * (i >> 2)) + (i & 3);
        key[i] = l[i] > -INFINITY ? (u << 16) | (uint32_t)(0xffff - e) : 0u;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int v = (int)(fmaxf(l[i] - mx, -33.0f) * 4194304.0f) + kHalf28;  // negative from 32 below mx on
        key[i] = v > 0 && l[i] > -INFINITY ? ((uint32_t)v << 4) | (uint32_t)(15 - i) : 0u;
      }
    }
    // exact score and choice value of an expert; softmax's sum over the row, logits read again, in 64 bits
    auto exact_sum = [&]() -> double {
      double sum = 0.0;
#pragma unroll 1
      for (int e = r; e < E; e += 16) {
        const float x = load_logit(row + e);
        if (x > -INFINITY) sum += exp((double)x - (double)mx);
      }
      return row_sum_f64(sum);
    };
    auto exact_choice = [&](int e, double sum) -> double {
      const double x = (double)load_logit(row + e);
      const double s = p.score == 0 ? exp(x - (double)mx) / sum : 1.0 / (1.0 + exp(-x));
      return s + (p.bias ? (double)p.bias[e] : 0.0);
    };
    if (groups) {
      // the two largest values of each run of four experts, then of each group on its own lane
      const int gs = E / p.n_group, nq = gs >> 2;
      uint32_t* quad = reinterpret_cast<uint32_t*>(s_x[wave]) + g * 128;
      constexpr int SH = EXACT16 ? 16 : 4;
      wave_lds_fence();
#pragma unroll
      for (int q = 0; q < N / 4; ++q) {
        const uint32_t a = max(key[4 * q], key[4 * q + 1]), b = min(key[4 * q], key[4 * q + 1]);
        const uint32_t c = max(key[4 * q + 2], key[4 * q + 3]), d = min(key[4 * q + 2], key[4 * q + 3]);
        *reinterpret_cast<u32x2_t*>(quad + 2 * (r + 16 * q)) = u32x2_t{max(a, c), max(min(a, c), max(b, d))};
      }
      wave_lds_fence();
      uint32_t a = 0, b = 0;
      if (r < p.n_group)
        for (int i = 0; i < nq; ++i) {
          const u32x2_t v = *reinterpret_cast<const u32x2_t*>(quad + 2 * (r * nq + i));
          b = max(min(a, v[0]), max(b, v[1]));
          a = max(a, v[0]);
        }
      a >>= SH;
      b >>= SH;
      uint32_t gv = a;
      if (EXACT16) gv = r < p.n_group ? (a << 4) | (uint32_t)(15 - r) : 0u;  // ties to the lower group
      else if (p.group_top == 2 && a != 0) gv = a + (b != 0 ? b : (uint32_t)kHalf28);
      bool keep = r < p.n_group && count_larger<1>(gv) < p.topk_group;
      uint32_t mask = (uint32_t)(__ballot(keep) >> (16 * g)) & 0xffffu;
      const uint32_t lo = row_min_u32(keep ? gv : 0xffffffffu);
      const uint32_t hi = row_max_fused(r < p.n_group && !keep ? gv : 0u);
      const bool edge = __builtin_popcount(mask) != p.topk_group || lo <= hi + 2 * thr;
      if (!EXACT16 && __ballot(edge) != 0) {
        // Groups too close at the edge: ranked by their exact values, from the two best experts of each,
        // scored in 64 bits on the group's lane. That needs both certain (the third further off than thr).
        uint32_t* const all = reinterpret_cast<uint32_t*>(s_x[wave]) + g * 256;
        wave_lds_fence();
#pragma unroll
        for (int i = 0; i < N; ++i) all[4 * (r + 16 * (i >> 2)) + (i & 3)] = key[i];
        wave_lds_fence();
        uint32_t ka = 0, kb = 0, kc = 0;
        int ea = 0, eb = 0;
        if (r < p.n_group)
          for (int i = 0; i < gs; ++i) {
            const uint32_t kk = all[r * gs + i];
            const bool fa = kk > ka, fb = kk > kb;
            kc = max(kc, fb ? kb : kk);
            eb = fa ? ea : (fb ? r * gs + i : eb);
            kb = fa ? ka : (fb ? kk : kb);
            ea = fa ? r * gs + i : ea;
            ka = fa ? kk : ka;
          }
        flag |= edge && (kc >= 16u && ((kb >> 4) - (kc >> 4)) <= thr);
        const double sum = CHOICE && p.score == 0 ? exact_sum() : 1.0;
        double va = -(double)INFINITY, vb = -(double)INFINITY;
        if (ka >= 16u) va = CHOICE ? exact_choice(ea, sum) : (double)load_logit(row + ea);
        if (kb >= 16u) vb = CHOICE ? exact_choice(eb, sum) : (double)load_logit(row + eb);
        double v = fmax(va, vb);
        if (p.group_top == 2 && kb >= 16u) v = va > vb ? va + vb : vb + va;
        const int rank = count_before<1>(v, r < p.n_group ? r : 16 + r);
        if (edge) keep = r < p.n_group && rank < p.topk_group;
        mask = (uint32_t)(__ballot(keep) >> (16 * g)) & 0xffffu;
      }
      wave_lds_fence();
#pragma unroll
      for (int q = 0; q < N / 4; ++q) {
        const bool in = (mask >> min((4 * (r + 16 * q)) / gs, 31)) & 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) key[4 * q + i] = in ? key[4 * q + i] : 0u;
      }
    }
    sort_desc(key);
    uint32_t my[NP], prev = 0xffffffffu;
    int my_r[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) my[i] = 0, my_r[i] = 0;
    bool near = false;
    constexpr uint32_t kFirst = EXACT16 ? 0x10000u : 16u;  // smallest key of an enabled expert
    // round j: the row's largest key goes to lane j (of its holders the lowest lane's; equal keys are near)
    auto round = [&](int j) -> uint32_t {
      const uint32_t m = row_max_fused(key[0]);
      const uint64_t wins = __ballot(key[0] == m);
      const int first = __builtin_ctz((uint32_t)(wins >> (16 * g)) & 0xffffu);
#pragma unroll
      for (int i = 0; i < NP; ++i)
        if (16 * i + r == j) {
          my[i] = m;
          my_r[i] = first;
        }
      // the winner's keys move up by one: a bitwise select on an opaque mask, which the compiler cannot
      // turn into a choice of registers at run time
      uint32_t pop = 0u - (uint32_t)(r == first);
      asm volatile("" : "+v"(pop));
#pragma unroll
      for (int i = 0; i < N; ++i) key[i] = ((i + 1 < N ? key[i + 1] : 0u) & pop) | (key[i] & ~pop);
      return m;
    };
    for (int j = 0; j < k; ++j) {
      const uint32_t m = round(j);
      if (!EXACT16) near |= ((prev >> 4) - (m >> 4)) <= thr;
      flag |= m < kFirst;
      prev = m;
    }
    if (!EXACT16) {  // the first one not picked, if there is one
      const uint32_t m = row_max_fused(key[0]);
      const bool close = m >= kFirst && ((prev >> 4) - (m >> 4)) <= thr;
      near |= close;
      flag |= close && k == 16;
      if (NP > 1) {
        flag |= near;
        near = false;
      }
    }
    auto expert = [&](int pick) -> int {
      if (EXACT16) return (int)(0xffffu - (my[pick] & 0xffffu));
      const int i = 15 - (int)(my[pick] & 15u);
      return 4 * (my_r[pick] + 16 * (i >> 2)) + (i & 3);
    };
    int e[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) e[i] = expert(i);
    if (!EXACT16 && NP == 1 && __ballot(near) != 0) {
      // Close values: the 16 best candidates, one a lane, ranked by their exact choice values. The order
      // stands if none beyond them can reach the picks.
      for (int j = k; j < 16; ++j) {
        const uint32_t m = round(j);
        if (j == 15) flag |= near && m >= kFirst && ((prev >> 4) - (m >> 4)) <= thr;
      }
      e[0] = expert(0);
      const double sum = p.bias && p.score == 0 ? exact_sum() : 1.0;
      double o = -(double)INFINITY;
      int id = 0x10000 + r;  // no candidate: after all others
      if (my[0] >= kFirst) {
        id = e[0];
        o = p.bias ? exact_choice(id, sum) : (double)load_logit(row + id);
      }
      const int rank = count_before<1>(o, id);
      e[0] = __builtin_amdgcn_ds_permute((16 * g + rank) << 2, e[0]);
    }
    const uint64_t flags = __ballot(flag);
    const bool slow = ((flags >> (16 * g)) & 0xffffull) != 0;
    // weights in 64 bits (the softmax's sum over all experts: 32-bit exponentials added in 64)
    double s[NP], tot = 0.0;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      s[i] = 0.0;
      if (16 * i + r < k && !slow) {
        const double x = (double)load_logit(row + e[i]);
        s[i] = p.score == 0 ? exp(x - (double)mx) : 1.0 / (1.0 + exp(-x));
      }
      tot += s[i];
    }
    if (p.renorm) {
      tot = row_sum_f64(tot);
#pragma unroll
      for (int i = 0; i < NP; ++i) s[i] = tot > 0.0 ? s[i] / tot : 0.0;
    } else if (p.score == 0) {
      double sum = 0.0;
      // (a bias may have disabled experts that count in the sum: their logits are read again)
      if (CHOICE) load_row16<V, N>(row, E, r, l);
#pragma unroll
      for (int i = 0; i < N; ++i) sum += (double)expf(fmaxf(l[i], -INFINITY) - mx);
      sum = row_sum_f64(sum);
#pragma unroll
      for (int i = 0; i < NP; ++i) s[i] /= sum;
    }
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (16 * i + r < k && !slow && t0 + g < p.T) {
        p.idx[t * k + 16 * i + r] = e[i];
        p.w[t * k + 16 * i + r] = (float)(s[i] * (double)p.scale);
      }
    if (flags != 0) {
      for (int h = 0; h < 4; ++h) {
        if (((flags >> (16 * h)) & 0xffffull) == 0 || t0 + h >= p.T) continue;
        route_row_exact(p, t0 + h, logits + (t0 + h) * E, s_x[wave],
                        reinterpret_cast<uint64_t*>(s_x[wave] + kMaxE), s_g[wave]);
      }
    }
  }
}

// Gradient, picks fixed: one token a wave. With g = dtopk_w and w the forward's
// weights (0 at a disabled pick, which then takes no part):
//   renorm:    D = sum_j g_j w_j / scale;  softmax dl_j = w_j (g_j - D), sigmoid times (1 - s_j)
//   no renorm: sigmoid dl_j = w_j (1 - s_j) g_j;  softmax dl_e = [e picked] w_e g_e - s_e sum_j w_j g_j
struct RouteBwdP {
  int64_t T;
  int E, k, score, renorm;
  float scale;
  const int32_t* idx;
  const float* w;
  const float* g;
};

__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) { *p = (uint16_t)pack_bf16x2(v, v); }

template <class V>
__global__ __launch_bounds__(256) void route_scored_bwd_kernel(RouteBwdP p, const V* __restrict__ logits,
                                                               V* __restrict__ dlogits) {
  __shared__ float s_row[4][kMaxE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float* row = s_row[wave];
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t < p.T) {
    const V* lt = logits + t * p.E;
    int e = -1;
    float w = 0.0f, g = 0.0f;
    if (lane < p.k) {
      e = p.idx[t * p.k + lane];
      w = p.w[t * p.k + lane];
      g = w != 0.0f ? p.g[t * p.k + lane] : 0.0f;
      if ((unsigned)e >= (unsigned)p.E) e = -1;
    }
    float wg = e >= 0 ? w * g : 0.0f, tot = wg;
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) tot += __shfl_xor(tot, s);
    if (p.renorm) wg = w * (g - tot / p.scale);
    if (p.score == 1 && e >= 0) wg *= 1.0f / (1.0f + expf(load_logit(lt + e)));
    const bool dense = p.score == 0 && !p.renorm;
    float base[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (dense) {
      float l[4], mx = -INFINITY;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        l[q] = lane + 64 * q < p.E ? load_logit(lt + lane + 64 * q) : -INFINITY;
        if (l[q] == l[q]) mx = fmaxf(mx, l[q]);
      }
      mx = wave_max_f32(mx);
      float sum = 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        base[q] = (l[q] == l[q] && l[q] != -INFINITY) ? (l[q] == mx ? 1.0f : expf(l[q] - mx)) : 0.0f;
        sum += base[q];
      }
#pragma unroll
      for (int s = 32; s >= 1; s >>= 1) sum += __shfl_xor(sum, s);
#pragma unroll
      for (int q = 0; q < 4; ++q) base[q] = base[q] != 0.0f ? -base[q] / sum * tot : 0.0f;
    }
    wave_lds_fence();
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (lane + 64 * q < p.E) row[lane + 64 * q] = base[q];
    wave_lds_fence();
    if (e >= 0 && w != 0.0f) row[e] += wg;
    wave_lds_fence();
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (lane + 64 * q < p.E) store_logit(dlogits + t * p.E + lane + 64 * q, row[lane + 64 * q]);
    wave_lds_fence();
  }
}

// The same, four tokens a wave on 16 lanes each (k <= 32), the row assembled in
// LDS and stored 4 elements a lane where E is a multiple of 4. Latency bounds
// it (2 us of memory at a copy's rate): 32749 x 60 bf16, every logit with a
// gradient, 5.0 us (12.8 us with a wave a token, most lanes idle); 8192 x 256
// fp32, picks only, 4.4 us (5.0 us).
template <class V, int N, int NP>
__global__ __launch_bounds__(256) void route_scored_bwd16_kernel(RouteBwdP p, const V* __restrict__ logits,
                                                                 V* __restrict__ dlogits) {
  __shared__ __attribute__((aligned(16))) float s_row[4][4][16 * N];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, r = lane & 15;
  const int E = p.E, k = p.k;
  const int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * 4;
  if (t0 >= p.T) return;  // wave-uniform
  const int64_t t = min(t0 + g, p.T - 1);
  const V* lt = logits + t * E;
  float* row = s_row[wave][g];
  int e[NP];
  float w[NP], gr[NP], wg[NP], tot = 0.0f;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    e[i] = -1;
    w[i] = gr[i] = 0.0f;
    if (16 * i + r < k) {
      e[i] = p.idx[t * k + 16 * i + r];
      w[i] = p.w[t * k + 16 * i + r];
      gr[i] = p.g[t * k + 16 * i + r];
      if ((unsigned)e[i] >= (unsigned)E || w[i] == 0.0f) e[i] = -1;
    }
    wg[i] = e[i] >= 0 ? w[i] * gr[i] : 0.0f;
    tot += wg[i];
  }
  float l[N];
  const bool dense = p.score == 0 && !p.renorm;
  if (dense) load_row16<V, N>(lt, E, r, l);
  tot = row_sum(tot);
#pragma unroll
  for (int i = 0; i < NP; ++i)
    if (e[i] >= 0) {
      if (p.renorm) wg[i] = w[i] * (gr[i] - tot / p.scale);
      if (p.score == 1) wg[i] *= 1.0f / (1.0f + expf(load_logit(lt + e[i])));
    }
  float base[N];
#pragma unroll
  for (int i = 0; i < N; ++i) base[i] = 0.0f;
  if (dense) {
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      l[i] = fmaxf(l[i], -INFINITY);  // NaN -> -inf
      mx = fmaxf(mx, l[i]);
    }
    mx = row_max_f32(mx);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      base[i] = l[i] > -INFINITY ? (l[i] == mx ? 1.0f : expf(l[i] - mx)) : 0.0f;
      sum += base[i];
    }
    sum = row_sum(sum);
    const float f = sum > 0.0f ? -tot / sum : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) base[i] *= f;
  }
#pragma unroll
  for (int q = 0; q < N / 4; ++q)
    *reinterpret_cast<f32x4_t*>(row + 4 * (r + 16 * q)) =
        f32x4_t{base[4 * q], base[4 * q + 1], base[4 * q + 2], base[4 * q + 3]};
  wave_lds_fence();
#pragma unroll
  for (int i = 0; i < NP; ++i)
    if (e[i] >= 0) row[e[i]] += wg[i];
  wave_lds_fence();
  if (t0 + g >= p.T) return;
  V* out = dlogits + t * E;
#pragma unroll
  for (int q = 0; q < N / 4; ++q) {
    const int e0 = 4 * (r + 16 * q);
    const f32x4_t v = *reinterpret_cast<const f32x4_t*>(row + e0);
    if ((E & 3) == 0) {
      if (e0 >= E) continue;
      if (sizeof(V) == 4) *reinterpret_cast<f32x4_t*>(out + e0) = v;
      else *reinterpret_cast<u32x2_t*>(out + e0) = u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e0 + i < E) store_logit(out + e0 + i, v[i]);
    }
  }
}

template <class V, int N, int NP>
void launch16(const RouteP& p, const V* logits, bool choice, hipStream_t stream) {
  const dim3 grid((unsigned)((p.T + 15) / 16));  // T * 64 < 2^31: the shape check of the call
  if (choice) route_scored16_kernel<V, N, true, NP><<<grid, dim3(256), 0, stream>>>(p, logits);
  else route_scored16_kernel<V, N, false, NP><<<grid, dim3(256), 0, stream>>>(p, logits);
}

template <class V, int NP>
void launch16_np(const RouteP& p, const V* l, bool choice, hipStream_t stream) {
  if (p.E <= 64) launch16<V, 4, NP>(p, l, choice, stream);
  else if (p.E <= 128) launch16<V, 8, NP>(p, l, choice, stream);
  else launch16<V, 16, NP>(p, l, choice, stream);
}

dim3 row_grid(int64_t T) { return dim3((unsigned)((T + 3) / 4)); }

template <class V, int NP>
void launch_bwd16(const RouteBwdP& p, const V* l, V* d, hipStream_t stream) {
  const dim3 grid((unsigned)((p.T + 15) / 16)), block(256);
  if (p.E <= 64) route_scored_bwd16_kernel<V, 4, NP><<<grid, block, 0, stream>>>(p, l, d);
  else if (p.E <= 128) route_scored_bwd16_kernel<V, 8, NP><<<grid, block, 0, stream>>>(p, l, d);
  else route_scored_bwd16_kernel<V, 16, NP><<<grid, block, 0, stream>>>(p, l, d);
}

template <class V>
void launch_bwd(const RouteBwdP& p, const V* l, V* d, hipStream_t stream) {
  if (p.k <= 16) launch_bwd16<V, 1>(p, l, d, stream);
  else if (p.k <= 32) launch_bwd16<V, 2>(p, l, d, stream);
  else route_scored_bwd_kernel<V><<<row_grid(p.T), dim3(256), 0, stream>>>(p, l, d);
}

}  // namespace

hipError_t launch_route_scored(int64_t T, int E, int k, int score, int n_group, int topk_group, int group_top,
                               int renorm, float scale, const void* logits, bool logits_bf16, const float* bias,
                               int32_t* topk_idx, float* topk_w, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const RouteP p{T, E, k, score, n_group, topk_group, group_top, renorm, scale, bias, topk_idx, topk_w};
  const bool groups = topk_group < n_group;
  const bool choice = bias != nullptr || (groups && group_top == 2);
  // k <= 32: one or two picks a lane; groups: one a lane, of whole runs of four experts. The rest takes the 64-bit
  // form, three to nine times as long (figures above; k = 24, 32768 x 128, softmax: 110 us against 17.5, and with a
  // bias, where close values are frequent, 107 against 54; k = 33: 140; 32768 x 60, k = 4: 6.2 us without groups, 57
  // and 46 with 4 and 10, of 15 and 6 experts; 8192 x 256 with 32 groups: 29).
  if (k <= 32 && (!groups || (n_group <= 16 && (E / n_group) % 4 == 0))) {
    if (logits_bf16) {
      const uint16_t* l = static_cast<const uint16_t*>(logits);
      if (k <= 16) launch16_np<uint16_t, 1>(p, l, choice, stream);
      else launch16_np<uint16_t, 2>(p, l, choice, stream);
    } else {
      const float* l = static_cast<const float*>(logits);
      if (k <= 16) launch16_np<float, 1>(p, l, choice, stream);
      else launch16_np<float, 2>(p, l, choice, stream);
    }
  } else if (logits_bf16) {
    route_scored_kernel<uint16_t><<<row_grid(T), dim3(256), 0, stream>>>(p, static_cast<const uint16_t*>(logits));
  } else {
    route_scored_kernel<float><<<row_grid(T), dim3(256), 0, stream>>>(p, static_cast<const float*>(logits));
  }
  return hipGetLastError();
}

hipError_t launch_route_scored_bwd(int64_t T, int E, int k, int score, int renorm, float scale, const void* logits,
                                   bool logits_bf16, const int32_t* topk_idx, const float* topk_w,
                                   const float* dtopk_w, void* dlogits, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const RouteBwdP p{T, E, k, score, renorm, scale, topk_idx, topk_w, dtopk_w};
  if (logits_bf16) launch_bwd(p, static_cast<const uint16_t*>(logits), static_cast<uint16_t*>(dlogits), stream);
  else launch_bwd(p, static_cast<const float*>(logits), static_cast<float*>(dlogits), stream);
  return hipGetLastError();
}

}  // namespace moe
