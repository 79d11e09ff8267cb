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
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) {
    const uint64_t o = (uint64_t)__shfl_xor((unsigned long long)v, s);
    v = o > v ? o : v;
  }
  return v;
}
__device__ __forceinline__ int wave_min_i32(int v) {
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) v = min(v, __shfl_xor(v, s));
  return v;
}
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

// One token on one wave, everything in 64 bits. l[q] is the logit of expert
// lane + 64 q (ignored at or past E); row_c and row_g are the wave's own LDS.
__device__ void route_row_exact(const RouteP& p, int64_t t, const float (&l)[4], double* row_c, uint64_t* row_g) {
  const int lane = threadIdx.x & 63;
  const int E = p.E;
  bool on[4];
  float mx = -INFINITY;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    on[q] = lane + 64 * q < E && l[q] == l[q] && l[q] != -INFINITY;
    if (on[q]) mx = fmaxf(mx, l[q]);
  }
  mx = wave_max_f32(mx);
  double s[4];
  double sum = 0.0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    s[q] = 0.0;
    if (!on[q]) continue;
    if (p.score == 0) s[q] = l[q] == mx ? 1.0 : exp((double)l[q] - (double)mx);
    else s[q] = 1.0 / (1.0 + exp(-(double)l[q]));
    sum += s[q];
  }
  if (p.score == 0) {
    sum = wave_sum_f64(sum);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (on[q]) s[q] /= sum;
  }
  uint64_t key[4];
  double choice[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int e = lane + 64 * q;
    double c = s[q];
    if (e < E && p.bias) {
      const float b = p.bias[e];
      on[q] = on[q] && b == b && b != -INFINITY;
      c += (double)b;
    }
    choice[q] = on[q] ? c : -(double)INFINITY;
    const double o = p.bias ? c : (double)l[q];
    key[q] = e < E ? (on[q] ? order_key64(o) : kKeyNegInf) : 0ull;
  }
  if (p.topk_group < p.n_group) {
    // group values by lane (several groups a lane past 64), from the row in LDS; a group's value
    // orders by the logits where it is one of them
    const int gs = E / p.n_group;
    wave_lds_fence();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int e = lane + 64 * q;
      if (e < E) row_c[e] = (!p.bias && p.group_top == 1 && on[q]) ? (double)l[q] : choice[q];
    }
    wave_lds_fence();
    for (int g = lane; g < p.n_group; g += 64) {
      double a = -(double)INFINITY, b = -(double)INFINITY;
      for (int i = 0; i < gs; ++i) {
        const double v = row_c[g * gs + i];
        b = fmax(b, fmin(a, v));
        a = fmax(a, v);
      }
      if (p.group_top == 2 && b != -(double)INFINITY) a += b;
      row_g[g] = order_key64(a);
    }
    wave_lds_fence();
    // a group stays if fewer than topk_group others come before it
    uint32_t keep = 0;
    for (int i = 0, g = lane; g < p.n_group; ++i, g += 64) {
      const uint64_t mine = row_g[g];
      int before = 0;
      for (int h = 0; h < p.n_group; ++h) before += row_g[h] > mine || (row_g[h] == mine && h < g);
      if (before < p.topk_group) keep |= 1u << i;
    }
    wave_lds_fence();
    for (int i = 0, g = lane; g < p.n_group; ++i, g += 64) row_g[g] = (keep >> i) & 1;
    wave_lds_fence();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int e = lane + 64 * q;
      if (e < E && !row_g[e / gs]) key[q] = kKeyNegInf;
    }
  }
  int my_e = 0;
  double my_s = 0.0;
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
    double sj = 0.0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (e == lane + 64 * q) {
        sj = key[q] > kKeyNegInf ? s[q] : 0.0;
        key[q] = 0ull;
      }
    sj = __shfl(sj, e & 63);
    if (lane == j) {
      my_e = e;
      my_s = sj;
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
}

template <class V>
__global__ __launch_bounds__(256) void route_scored_kernel(RouteP p, const V* __restrict__ logits) {
  __shared__ double s_c[4][kMaxE];
  __shared__ uint64_t s_g[4][kMaxE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < p.T; t += (int64_t)gridDim.x * 4) {
    float l[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) l[q] = lane + 64 * q < p.E ? load_logit(logits + t * p.E + lane + 64 * q) : -INFINITY;
    route_row_exact(p, t, l, s_c[wave], s_g[wave]);
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
  for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < p.T; t += (int64_t)gridDim.x * 4) {
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

dim3 row_grid(int64_t T) {
  const int64_t b = (T + 3) / 4;
  return dim3((unsigned)(b < (int64_t(1) << 20) ? b : (int64_t(1) << 20)));
}

}  // namespace

hipError_t launch_route_scored(int64_t T, int E, int k, int score, int n_group, int topk_group, int group_top,
                               int renorm, float scale, const void* logits, bool logits_bf16, const float* bias,
                               int32_t* topk_idx, float* topk_w, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const RouteP p{T, E, k, score, n_group, topk_group, group_top, renorm, scale, bias, topk_idx, topk_w};
  if (logits_bf16)
    route_scored_kernel<uint16_t><<<row_grid(T), dim3(256), 0, stream>>>(p, static_cast<const uint16_t*>(logits));
  else
    route_scored_kernel<float><<<row_grid(T), dim3(256), 0, stream>>>(p, static_cast<const float*>(logits));
  return hipGetLastError();
}

hipError_t launch_route_scored_bwd(int64_t T, int E, int k, int score, int renorm, float scale, const void* logits,
                                   bool logits_bf16, const int32_t* topk_idx, const float* topk_w,
                                   const float* dtopk_w, void* dlogits, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const RouteBwdP p{T, E, k, score, renorm, scale, topk_idx, topk_w, dtopk_w};
  if (logits_bf16)
    route_scored_bwd_kernel<uint16_t><<<row_grid(T), dim3(256), 0, stream>>>(
        p, static_cast<const uint16_t*>(logits), static_cast<uint16_t*>(dlogits));
  else
    route_scored_bwd_kernel<float><<<row_grid(T), dim3(256), 0, stream>>>(p, static_cast<const float*>(logits),
                                                                          static_cast<float*>(dlogits));
  return hipGetLastError();
}

}  // namespace moe
