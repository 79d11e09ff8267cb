// The norms around the layer and what joins it to the residual stream:
//   moe_norm       xn = N(x; w), N(v; w) = v * r(v) * (offset + w), r(v) = (mean(v^2) + eps)^-1/2
//   moe_block_out  out = res_scale * res + scale * gate * N(y; w_post), xn = N(out; w_next)
// and their gradients. All are streams over [T, emb] rows bound by HBM: every tensor is read once and
// written once, and a row stays in registers between its reduction and its use. That is why the
// norm after the layer, the residual sum and the next norm are one kernel (three would read and write
// the row between them: 18 bytes an element more in bf16), and why the sum over a token's expert rows
// can be taken in front of it.
//
// The tensors go through non-temporal loads and stores: a copy of 512 MiB runs at 6.1-6.3 TB/s so,
// at 5.5 without. Weights, which every row reads, stay cached.
#include <type_traits>

#include "common.h"
#include "kernels.h"
#include "lanes.h"

namespace moe {
namespace {

// 8 consecutive elements of a row as they lie in memory, fp32 or bf16.
template <bool NT, class V>
__device__ __forceinline__ V load_v(const V* p) {
  if constexpr (NT) return __builtin_nontemporal_load(p);
  else return *p;
}
template <bool NT, class V>
__device__ __forceinline__ void store_v(V v, V* p) {
  if constexpr (NT) __builtin_nontemporal_store(v, p);
  else *p = v;
}
template <bool F32>
struct Raw;
template <>
struct Raw<false> {
  u32x4_t a;
  template <bool NT>
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    a = load_v<NT>(reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p) + i));
  }
  __device__ __forceinline__ float operator[](int u) const { return (u & 1) ? bf16_hi(a[u >> 1]) : bf16_lo(a[u >> 1]); }
};
template <>
struct Raw<true> {
  f32x4_t a[2];
  template <bool NT>
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const f32x4_t* q = reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + i);
    a[0] = load_v<NT>(q);
    a[1] = load_v<NT>(q + 1);
  }
  __device__ __forceinline__ float operator[](int u) const { return a[u >> 2][u & 3]; }
};

template <bool NT>
__device__ __forceinline__ void store8(float* p, int64_t i, const float (&v)[8]) {
  f32x4_t* q = reinterpret_cast<f32x4_t*>(p + i);
  store_v<NT>(f32x4_t{v[0], v[1], v[2], v[3]}, q);
  store_v<NT>(f32x4_t{v[4], v[5], v[6], v[7]}, q + 1);
}
template <bool NT>
__device__ __forceinline__ void store8(uint16_t* p, int64_t i, const float (&v)[8]) {
  const u32x4_t o = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
  store_v<NT>(o, reinterpret_cast<u32x4_t*>(p + i));
}
template <bool NT>
__device__ __forceinline__ void store8(void* p, bool f32, int64_t i, const float (&v)[8]) {
  if (f32) store8<NT>(static_cast<float*>(p), i, v);
  else store8<NT>(static_cast<uint16_t*>(p), i, v);
}

// Weights and gates: of either type.
__device__ __forceinline__ void load8(const void* p, bool f32, int64_t i, float (&v)[8]) {
  if (f32) {
    const f32x4_t* q = reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + i);
    const f32x4_t a = q[0], b = q[1];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = a[u], v[4 + u] = b[u];
  } else {
    const u32x4_t a = ld16(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int u = 0; u < 4; ++u) v[2 * u] = bf16_lo(a[u]), v[2 * u + 1] = bf16_hi(a[u]);
  }
}
__device__ __forceinline__ float load1(const void* p, bool f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}
// offset + w[i..i+7]; 1 without a weight.
__device__ __forceinline__ void factor8(const void* w, bool f32, float offset, int i, float (&v)[8]) {
  if (!w) {
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = 1.0f;
    return;
  }
  load8(w, f32, i, v);
#pragma unroll
  for (int u = 0; u < 8; ++u) v[u] += offset;
}

// A row lies in L = 16 lanes, four rows a wave (rows of up to 256 elements), or in whole waves (L = 64).
//
// Sums over the `waves` waves of a row, of N values at once, in an order fixed by `waves`. Every wave of the workgroup
// calls it the same number of times; `turn` alternates the LDS rows, so that one barrier a call is enough (a wave
// writes a row again only after the barrier of the call between).
template <int L, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int waves, float (*sh)[16][3], int& turn) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = L == 16 ? row_sum(v[n]) : wave_sum(v[n]);
  if (L == 16 || waves == 1) return;
  const int wave = threadIdx.x >> 6, w0 = wave / waves * waves;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) sh[turn][wave][n] = v[n];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = 0;
  for (int w = w0; w < w0 + waves; ++w) {
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += sh[turn][w][n];
  }
  turn ^= 1;
}

constexpr int kGridRows = 1 << 21;  // workgroups along a grid's x: fewer than 2^32 lanes

// Forward, a workgroup a row (L = 16: sixteen rows), KC chunks of 8 elements a lane. SRC 0: x itself (moe_norm), 1: y
// given, 2: y = sum over the token's picks of expert rows.
template <int L, int KC, int SRC, bool XF32>
__global__ __launch_bounds__(L == 16 ? 256 : 1024) void block_out_kernel(int64_t T, int emb, BlockArgs b, const void* res, const uint16_t* __restrict__ y,
                                                         int k, const uint16_t* __restrict__ ys,
                                                         const int32_t* __restrict__ slot_row,
                                                         const float* __restrict__ topk_w, void* out,
                                                         uint16_t* __restrict__ xn, uint16_t* __restrict__ y_out) {
  __shared__ float sh[2][16][3];
  constexpr bool kNt = KC > 1;  // few rows (KC 1) fit the caches, where the next kernel finds them
  int turn = 0;
  const int G = L == 16 ? 16 : blockDim.x, lane = L == 16 ? threadIdx.x & 15 : threadIdx.x, waves = G >> 6;
  const int64_t b0 = (int64_t)blockIdx.y * kGridRows + blockIdx.x;
  const int64_t t = L == 16 ? b0 * 16 + (threadIdx.x >> 4) : b0, base = t * emb;
  if (t >= T) return;
  const int nch = emb / 8;
  const float inv = 1.0f / emb;

  Raw<XF32> x[KC];
#pragma unroll
  for (int i = 0; i < KC; ++i)
    if (i * G + lane < nch) x[i].template load<kNt>(res, base + (i * G + lane) * 8);
  float v[KC][8];
  if constexpr (SRC == 0) {
#pragma unroll
    for (int i = 0; i < KC; ++i)
#pragma unroll
      for (int u = 0; u < 8; ++u) v[i][u] = x[i][u];
  }
  if constexpr (SRC == 1) {
    Raw<false> q[KC];
#pragma unroll
    for (int i = 0; i < KC; ++i)
      if (i * G + lane < nch) q[i].template load<kNt>(y, base + (i * G + lane) * 8);
#pragma unroll
    for (int i = 0; i < KC; ++i)
#pragma unroll
      for (int u = 0; u < 8; ++u) v[i][u] = q[i][u];
  }
  if constexpr (SRC == 2) {
    const int64_t S = T * k;
    const int l = threadIdx.x & 63;
    int32_t my_r = -1;
    float my_w = 0;
    if (L == 64 && l < k) {
      const int32_t r = slot_row[t * k + l];
      if (r >= 0 && r < S) my_r = r, my_w = topk_w ? topk_w[t * k + l] : 1.0f;
    }
#pragma unroll
    for (int i = 0; i < KC; ++i) {
#pragma unroll
      for (int u = 0; u < 8; ++u) v[i][u] = 0;
    }
    // fused multiply-adds in pick order, as in the combine kernel; the rows of 8 picks in flight at once. The picks are
    // read from their lanes before any lane leaves, so lanes past the row's end read row ends again.
    for (int j0 = 0; j0 < k; j0 += 8) {
      u32x4_t q[KC][8];
      float ww[8];
      int32_t rr[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if constexpr (L == 16) {
          rr[u] = -1;
          ww[u] = 0;
          if (j0 + u < k) {
            const int32_t r = slot_row[t * k + j0 + u];
            if (r >= 0 && r < S) rr[u] = r, ww[u] = topk_w ? topk_w[t * k + j0 + u] : 1.0f;
          }
        } else {
          rr[u] = j0 + u < k ? __builtin_amdgcn_readlane(my_r, (j0 + u) & 63) : -1;
          ww[u] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(my_w), (j0 + u) & 63));
        }
#pragma unroll
        for (int i = 0; i < KC; ++i)
          if (rr[u] >= 0)
            q[i][u] = load_v<kNt>(
                reinterpret_cast<const u32x4_t*>(ys + (int64_t)rr[u] * emb + min(i * G + lane, nch - 1) * 8));
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (rr[u] < 0) continue;
#pragma unroll
        for (int i = 0; i < KC; ++i)
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            v[i][2 * m] = __builtin_fmaf(ww[u], bf16_lo(q[i][u][m]), v[i][2 * m]);
            v[i][2 * m + 1] = __builtin_fmaf(ww[u], bf16_hi(q[i][u][m]), v[i][2 * m + 1]);
          }
      }
    }
    if (y_out) {
#pragma unroll
      for (int i = 0; i < KC; ++i)
        if (i * G + lane < nch) store8<kNt>(y_out, base + (i * G + lane) * 8, v[i]);
    }
  }
  if constexpr (SRC > 0) {
    float r = b.scale;
    if (b.post) {
      float s[1] = {0};
#pragma unroll
      for (int i = 0; i < KC; ++i) {
        if (i * G + lane >= nch) continue;
#pragma unroll
        for (int u = 0; u < 8; ++u) s[0] = __builtin_fmaf(v[i][u], v[i][u], s[0]);
      }
      row_sums<L>(s, waves, sh, turn);
      r *= rsqrtf(s[0] * inv + b.eps);
    }
    if (b.gate_mode == kGateToken) r *= load1(b.gate, b.gate_f32, t);
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int n = (i * G + lane) * 8;
      if (n >= emb) continue;
      float f[8];
      if (b.post_weight) {
        factor8(b.post_weight, b.w_f32, b.offset, n, f);
#pragma unroll
        for (int u = 0; u < 8; ++u) v[i][u] *= f[u];
      }
      if (b.gate_mode == kGateChannel || b.gate_mode == kGateFull) {
        load8(b.gate, b.gate_f32, (b.gate_mode == kGateFull ? base : 0) + n, f);
#pragma unroll
        for (int u = 0; u < 8; ++u) v[i][u] *= f[u];
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) v[i][u] = __builtin_fmaf(r, v[i][u], b.res_scale * x[i][u]);
      store8<kNt>(out, XF32, base + n, v[i]);
    }
  }
  // the next norm takes the sum before it is rounded to the residual's type
  if (SRC > 0 && !xn) return;
  float s[1] = {0};
#pragma unroll
  for (int i = 0; i < KC; ++i) {
    if (i * G + lane >= nch) continue;
#pragma unroll
    for (int u = 0; u < 8; ++u) s[0] = __builtin_fmaf(v[i][u], v[i][u], s[0]);
  }
  row_sums<L>(s, waves, sh, turn);
  const float r = rsqrtf(s[0] * inv + b.eps);
#pragma unroll
  for (int i = 0; i < KC; ++i) {
    const int n = (i * G + lane) * 8;
    if (n >= emb) continue;
    float f[8];
    factor8(b.next_weight, b.w_f32, b.offset, n, f);
#pragma unroll
    for (int u = 0; u < 8; ++u) f[u] *= v[i][u] * r;
    store8<kNt>(xn, base + n, f);
  }
}

// Backward, for d = the gradient of out. With NEXT, d = dout + r (g - o c), g = dxn (offset + w_next), o = out,
// c = r^2 mean(g o). Then dres = res_scale d, and with dz = scale gate d: dy = dz, or with POST
// r_y (h - y c_y), h = dz (offset + w_post), c_y = r_y^2 mean(h y). Column sums (the weights' gradients dxn o r and
// dz y r_y, a channel gate's scale d z) are kept in registers over all rows of a workgroup and leave it as one
// partial row each, which colsum_kernel adds up in order.
// HASY false: d alone is wanted (moe_norm_bwd).
//
// A workgroup holds up to 512 / G rows at a time (G lanes a row, KC chunks of 8 elements a lane) and takes every
// gridDim.x-th such set. Weights, sums and a row fill the registers to two waves a SIMD, too few to hide the loads by
// switching, so the next set's rows are loaded before the present one is worked on (AHEAD).
constexpr int kBwdLanes = 512;

template <int KC, bool XF32, bool HASY, bool NEXT>
struct BwdRow {
  Raw<XF32> o[KC], d[KC];
  Raw<false> g[KC], y[KC];
};

template <int L, int KC, bool AHEAD, bool XF32, bool HASY, bool NEXT, bool POST, bool CHG>
__global__ __launch_bounds__(kBwdLanes) void block_out_bwd_kernel(int64_t T, int emb, int lanes, BlockArgs b, const void* dout,
                                                                  const uint16_t* __restrict__ y, const void* out,
                                                                  const uint16_t* __restrict__ dxn, void* dres,
                                                                  uint16_t* __restrict__ dy, void* __restrict__ dgate,
                                                                  float* __restrict__ part) {
  constexpr int kNext = 0, kPost = NEXT ? 1 : 0, kGate = kPost + (POST ? 1 : 0), kAcc = kGate + (CHG ? 1 : 0);
  __shared__ float sh[2][16][3];
  __shared__ float comb[kBwdLanes * 8];
  int turn = 0;
  const int G = L == 16 ? 16 : lanes, per = blockDim.x / G, grp = threadIdx.x / G, lane = threadIdx.x - grp * G, waves = G >> 6;
  const float inv = 1.0f / emb;
  float acc[kAcc > 0 ? kAcc : 1][KC][8] = {};
  // the norms' factors stay in registers where there is room for them
  constexpr bool kKeep = KC == 2;
  float keep_n[KC][8], keep_p[KC][8];
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int n = (i * G + lane) * 8;
      if (n >= emb) continue;
      if constexpr (NEXT) factor8(b.next_weight, b.w_f32, b.offset, n, keep_n[i]);
      if constexpr (POST) factor8(b.post_weight, b.w_f32, b.offset, n, keep_p[i]);
    }
  }
  const auto factor = [&](const float (&keep)[8], const void* w, int n, float (&f)[8]) {
    if constexpr (kKeep) {
#pragma unroll
      for (int u = 0; u < 8; ++u) f[u] = keep[u];
    } else {
      factor8(w, b.w_f32, b.offset, n, f);
    }
  };
  const bool need_y = HASY && y;
  using Row = BwdRow<KC, XF32, HASY, NEXT>;
  const auto fetch = [&](Row& q, int64_t t) {
    const int64_t base = t * emb;
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int n = (i * G + lane) * 8;
      if (n >= emb) continue;
      if constexpr (NEXT) {
        q.o[i].template load<true>(out, base + n);
        q.g[i].template load<true>(dxn, base + n);
      }
      if (dout) q.d[i].template load<true>(dout, base + n);
      if (need_y) q.y[i].template load<true>(y, base + n);
    }
  };
  const int64_t stride = (int64_t)gridDim.x * per, first = (int64_t)blockIdx.x * per + grp;
  Row next;
  if (AHEAD && first < T) fetch(next, first);
  for (int64_t t = first; t - grp < T; t += stride) {
    const bool on = t < T;  // groups past the last row go along for the barriers
    const int64_t base = t * emb;
    Row q;
    if constexpr (AHEAD) {
      q = next;
      if (t + stride < T) fetch(next, t + stride);
    } else {
      if (on) fetch(q, t);
    }
    float s[3] = {0, 0, 0};
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int n = (i * G + lane) * 8;
      if (!on || n >= emb) continue;
      float fn[8];
      if constexpr (NEXT) factor(keep_n[i], b.next_weight, n, fn);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if constexpr (NEXT) {
          s[0] = __builtin_fmaf(q.o[i][u], q.o[i][u], s[0]);
          s[1] = __builtin_fmaf(q.g[i][u] * fn[u], q.o[i][u], s[1]);
        }
        if constexpr (POST) s[2] = __builtin_fmaf(q.y[i][u], q.y[i][u], s[2]);
      }
    }
    if constexpr (NEXT || POST) row_sums<L>(s, waves, sh, turn);
    const float r = NEXT ? rsqrtf(s[0] * inv + b.eps) : 0.0f, c = r * r * (s[1] * inv);
    const float ry = POST ? rsqrtf(s[2] * inv + b.eps) : 1.0f;
    const bool token = HASY && b.gate_mode == kGateToken;
    const float tok = token && on ? load1(b.gate, b.gate_f32, t) : 1.0f;
    float h[KC][8], sum[1] = {0};
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int n = (i * G + lane) * 8;
      if (!on || n >= emb) continue;
      float d[8], fn[8], fp[8];
      if constexpr (NEXT) factor(keep_n[i], b.next_weight, n, fn);
      if constexpr (POST) factor(keep_p[i], b.post_weight, n, fp);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        d[u] = dout ? q.d[i][u] : 0.0f;
        if constexpr (NEXT) {
          d[u] = __builtin_fmaf(r, q.g[i][u] * fn[u] - q.o[i][u] * c, d[u]);
          acc[kNext][i][u] = __builtin_fmaf(q.g[i][u], q.o[i][u] * r, acc[kNext][i][u]);
        }
      }
      if (dres) {
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = b.res_scale * d[u];
        store8<true>(dres, XF32, base + n, v);
      }
      if constexpr (HASY) {
        // h = scale gate d (the token's gate comes in at the end), then times the post norm's factor
#pragma unroll
        for (int u = 0; u < 8; ++u) d[u] *= b.scale;
        if constexpr (CHG) {
          float gc[8];
          load8(b.gate, b.gate_f32, n, gc);
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            acc[kGate][i][u] = __builtin_fmaf(d[u], q.y[i][u] * ry * (POST ? fp[u] : 1.0f), acc[kGate][i][u]);
            d[u] *= gc[u];
          }
        }
        if (b.gate_mode == kGateFull) {
          float gt[8], dg[8];
          load8(b.gate, b.gate_f32, base + n, gt);
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            dg[u] = d[u] * (q.y[i][u] * ry * (POST ? fp[u] : 1.0f));
            d[u] *= gt[u];
          }
          if (dgate) store8<true>(dgate, b.gate_f32, base + n, dg);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if constexpr (POST) {
            acc[kPost][i][u] = __builtin_fmaf(tok * d[u], q.y[i][u] * ry, acc[kPost][i][u]);
            d[u] *= fp[u];
          }
          if (POST || token) sum[0] = __builtin_fmaf(d[u], q.y[i][u], sum[0]);
          h[i][u] = d[u];
        }
      }
    }
    if constexpr (HASY) {
      float cy = 0;
      if (POST || token) {
        row_sums<L>(sum, waves, sh, turn);
        cy = ry * ry * (sum[0] * inv);
        if (token && dgate && lane == 0 && on) static_cast<float*>(dgate)[t] = sum[0] * ry;
      }
      if (dy && on) {
        const float e = tok * ry;
#pragma unroll
        for (int i = 0; i < KC; ++i) {
          const int n = (i * G + lane) * 8;
          if (n >= emb) continue;
#pragma unroll
          for (int u = 0; u < 8; ++u) h[i][u] = e * (POST ? h[i][u] - q.y[i][u] * cy : h[i][u]);
          store8<true>(dy, base + n, h[i]);
        }
      }
    }
  }
  if (!part) return;
  // the groups' sums (of one wave's four by lane exchanges), then one partial row per sum
  const int sets = L == 16 ? blockDim.x >> 6 : per, set = L == 16 ? threadIdx.x >> 6 : grp;
  const bool holds = L != 16 || (threadIdx.x & 63) < 16;
#pragma unroll
  for (int a = 0; a < kAcc; ++a) {
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int n = (i * G + lane) * 8;
      if (i * G * 8 >= emb) continue;
      if constexpr (L == 16) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          acc[a][i][u] += __shfl_xor(acc[a][i][u], 16);
          acc[a][i][u] += __shfl_xor(acc[a][i][u], 32);
        }
      }
      if (sets > 1) {
        __syncthreads();
        if (holds) {
#pragma unroll
          for (int u = 0; u < 8; ++u) comb[u * kBwdLanes + set * G + lane] = acc[a][i][u];
        }
        __syncthreads();
        if (set == 0 && holds) {
          for (int p = 1; p < sets; ++p)
#pragma unroll
            for (int u = 0; u < 8; ++u) acc[a][i][u] += comb[u * kBwdLanes + p * G + lane];
        }
      }
      if (set == 0 && holds && n < emb) {
        f32x4_t* d = reinterpret_cast<f32x4_t*>(part + ((int64_t)a * gridDim.x + blockIdx.x) * emb + n);
        d[0] = f32x4_t{acc[a][i][0], acc[a][i][1], acc[a][i][2], acc[a][i][3]};
        d[1] = f32x4_t{acc[a][i][4], acc[a][i][5], acc[a][i][6], acc[a][i][7]};
      }
    }
  }
}

// Column sums of P partial rows: 64 columns a workgroup, 16 waves share the rows.
struct ColsumOut {
  float* p[3];
};
__global__ __launch_bounds__(1024) void colsum_kernel(int P, int emb, const float* __restrict__ part, ColsumOut out) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = blockIdx.x * 64 + lane;
  float* dst = out.p[blockIdx.y];
  if (!dst) return;
  const float* p = part + (int64_t)blockIdx.y * P * emb + (n < emb ? n : 0);
  float s = 0;
#pragma unroll 8
  for (int r = wave; r < P; r += 16) s += p[(int64_t)r * emb];
  red[wave][lane] = s;
  __syncthreads();
  if (wave) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) s += red[w][lane];
  if (n < emb) dst[n] = s;
}

// Lanes that hold a row at kc chunks of 8 a lane: 16, or whole waves.
constexpr int kSubEmb = 256;  // longest row of 16 lanes
int lanes_of(int emb, int kc) { return kc == 2 && emb <= kSubEmb ? 16 : (emb / 8 + 64 * kc - 1) / (64 * kc) * 64; }

// The backward's shape: two chunks a lane while 512 lanes hold the row so, else four.
struct BwdPlan {
  int kc, G, per, grid;
};
BwdPlan bwd_plan(int64_t T, int emb) {
  BwdPlan p;
  p.kc = emb <= 2 * 8 * kBwdLanes ? 2 : 4;
  p.G = lanes_of(emb, p.kc);
  p.per = kBwdLanes / p.G;
  const int64_t sets = (T + p.per - 1) / p.per;
  p.grid = (int)(sets < 256 ? sets : 256);  // one workgroup a compute unit
  return p;
}

template <int L, int KC, bool XF32>
void fwd(int64_t T, int emb, const BlockArgs& b, const void* res, const uint16_t* y, int k, const uint16_t* ys,
         const int32_t* slot_row, const float* w, void* out, uint16_t* xn, uint16_t* y_out, hipStream_t st) {
  const int64_t n = L == 16 ? (T + 15) / 16 : T;
  const dim3 grid((unsigned)(n < kGridRows ? n : kGridRows), (unsigned)((n + kGridRows - 1) / kGridRows));
  const dim3 block(L == 16 ? 256 : lanes_of(emb, KC));
  if (ys) block_out_kernel<L, KC, 2, XF32><<<grid, block, 0, st>>>(T, emb, b, res, y, k, ys, slot_row, w, out, xn, y_out);
  else if (y) block_out_kernel<L, KC, 1, XF32><<<grid, block, 0, st>>>(T, emb, b, res, y, k, ys, slot_row, w, out, xn, y_out);
  else block_out_kernel<L, KC, 0, XF32><<<grid, block, 0, st>>>(T, emb, b, res, y, k, ys, slot_row, w, out, xn, y_out);
}

template <int L, int KC, bool XF32>
void bwd(const BwdPlan& p, int64_t T, int emb, const BlockArgs& b, bool has_y, const void* dout, const uint16_t* y,
         const void* out, const uint16_t* dxn, void* dres, uint16_t* dy, void* dgate, float* part, hipStream_t st) {
  const bool post = b.post, chg = b.gate_mode == kGateChannel;
#define MOE_BWD(H, N, P, C)                                                                                         \
  block_out_bwd_kernel<L, KC, KC == 2 && !(XF32 && P && C), XF32, H, N, P, C><<<dim3(p.grid), dim3(p.per * p.G), 0, st>>>(T, emb, p.G, b, dout, y, \
                                                                                                out, dxn, dres, dy, dgate, part)
  if (!has_y) MOE_BWD(false, true, false, false);
  else if (dxn && post && chg) MOE_BWD(true, true, true, true);
  else if (dxn && post) MOE_BWD(true, true, true, false);
  else if (dxn && chg) MOE_BWD(true, true, false, true);
  else if (dxn) MOE_BWD(true, true, false, false);
  else if (post && chg) MOE_BWD(true, false, true, true);
  else if (post) MOE_BWD(true, false, true, false);
  else if (chg) MOE_BWD(true, false, false, true);
  else MOE_BWD(true, false, false, false);
#undef MOE_BWD
}

}  // namespace

hipError_t launch_block_out(int64_t T, int emb, const BlockArgs& b, const void* res, const uint16_t* y, int k,
                            const uint16_t* ys, const int32_t* slot_row, const float* topk_w, void* out, uint16_t* xn,
                            uint16_t* y_out, hipStream_t st) {
  if (T == 0) return hipSuccess;
  // Few rows: a chunk a lane, the shortest way through a row. Many: two, half the waves to add up (32768 rows of 2048:
  // 95 us against 106), and short rows four a wave (400000 rows of 128, norm alone: 36 us against 98).
  const auto go = [&](auto l, auto kc) {
    if (b.x_f32) fwd<decltype(l)::value, decltype(kc)::value, true>(T, emb, b, res, y, k, ys, slot_row, topk_w, out, xn, y_out, st);
    else fwd<decltype(l)::value, decltype(kc)::value, false>(T, emb, b, res, y, k, ys, slot_row, topk_w, out, xn, y_out, st);
  };
  using std::integral_constant;
  if (emb <= 8192 && T <= 256) go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (emb > kSubEmb) go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else go(integral_constant<int, 16>{}, integral_constant<int, 2>{});
  return hipGetLastError();
}

size_t block_bwd_workspace(int64_t T, int emb, int sums) { return (size_t)bwd_plan(T, emb).grid * sums * emb * 4; }

hipError_t launch_block_out_bwd(int64_t T, int emb, const BlockArgs& b, bool has_y, const void* dout, const uint16_t* y,
                                const void* out, const uint16_t* dxn, void* dres, uint16_t* dy, float* dpost,
                                float* dnext, void* dgate, float* part, hipStream_t st) {
  const BwdPlan p = bwd_plan(T, emb);
  if (T > 0) {
    const auto go = [&](auto l, auto kc) {
      if (b.x_f32) bwd<decltype(l)::value, decltype(kc)::value, true>(p, T, emb, b, has_y, dout, y, out, dxn, dres, dy, dgate, part, st);
      else bwd<decltype(l)::value, decltype(kc)::value, false>(p, T, emb, b, has_y, dout, y, out, dxn, dres, dy, dgate, part, st);
    };
    using std::integral_constant;
    if (p.G == 16) go(integral_constant<int, 16>{}, integral_constant<int, 2>{});
    else if (p.kc == 2) go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    else go(integral_constant<int, 64>{}, integral_constant<int, 4>{});
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  // the order of the kernel's partial sums; of no rows (T = 0) the sums are 0
  ColsumOut c{};
  int n = 0;
  const bool chg = b.gate_mode == kGateChannel;
  if (T == 0 || !has_y || dxn) c.p[n++] = dnext;
  if (has_y && b.post) c.p[n++] = dpost;
  if (has_y && chg) c.p[n++] = static_cast<float*>(dgate);
  if (c.p[0] || c.p[1] || c.p[2])
    colsum_kernel<<<dim3((emb + 63) / 64, n), dim3(1024), 0, st>>>(p.grid, emb, part, c);
  return hipGetLastError();
}

}  // namespace moe
