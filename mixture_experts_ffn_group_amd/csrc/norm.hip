// The norms around the layer and what joins it to the residual stream:
//   moe_norm       xn = N(x; w), N(v; w) = v * r(v) * (offset + w), r(v) = (mean(v^2) + eps)^-1/2
//   moe_block_out  out = res_scale * res + scale * gate * N(y; w_post), xn = N(out; w_next)
// and their gradients. All are streams over [T, emb] rows bound by HBM: every tensor is read once and
// written once, and a row stays in registers between its reduction and its use. That is why the
// norm after the layer, the residual sum and the next norm are one kernel (three would read and write
// the row between them: 18 bytes an element more in bf16), and why the sum over a token's expert rows
// can be taken in front of it.
//
// A row is held by G = 64, 128, 256 or 512 lanes, at most kCh chunks of 8 elements a lane: the
// fewest lanes that hold it, so that most rows need no LDS for their sums.
#include "common.h"
#include "kernels.h"
#include "lanes.h"

namespace moe {
namespace {

constexpr int kCh = 4;

// 8 consecutive elements, of fp32 or bf16, as floats.
__device__ __forceinline__ void load8(const void* p, bool f32, int64_t i, float (&v)[8]) {
  if (f32) {
    const f32x4_t a = *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + i);
    const f32x4_t b = *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + i + 4);
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = a[u], v[4 + u] = b[u];
  } else {
    const u32x4_t a = ld16(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int u = 0; u < 4; ++u) v[2 * u] = bf16_lo(a[u]), v[2 * u + 1] = bf16_hi(a[u]);
  }
}
__device__ __forceinline__ void store8(void* p, bool f32, int64_t i, const float (&v)[8]) {
  if (f32) {
    float* d = static_cast<float*>(p) + i;
    *reinterpret_cast<f32x4_t*>(d) = f32x4_t{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4_t*>(d + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
  } else {
    st16(static_cast<uint16_t*>(p) + i, u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                               pack_bf16x2(v[6], v[7])});
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

// Sums over the G lanes of a row, of N values at once, in an order fixed by G. Every lane of the workgroup calls it
// the same number of times; `turn` alternates the LDS rows, so one barrier a call is enough (a wave writes a row
// again only after the barrier of the call between).
template <int G, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*sh)[8][4], int& turn) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = wave_sum(v[n]);
  if constexpr (G > 64) {
    constexpr int kW = G / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) sh[turn][wave][n] = v[n];
    }
    __syncthreads();
    const int w0 = wave / kW * kW;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float s = 0;
#pragma unroll
      for (int w = 0; w < kW; ++w) s += sh[turn][w0 + w][n];
      v[n] = s;
    }
    turn ^= 1;
  }
}

template <int G>
constexpr int block_size() {
  return G < 256 ? 256 : G;
}

// Forward. SRC 0: x itself (moe_norm), 1: y given, 2: y = sum over the token's picks of expert rows.
template <int G, int SRC>
__global__ __launch_bounds__(block_size<G>()) void block_out_kernel(int64_t T, int emb, BlockArgs b, const void* res,
                                                                    const uint16_t* __restrict__ y, int k,
                                                                    const uint16_t* __restrict__ ys,
                                                                    const int32_t* __restrict__ slot_row,
                                                                    const float* __restrict__ topk_w, void* out,
                                                                    uint16_t* __restrict__ xn,
                                                                    uint16_t* __restrict__ y_out) {
  __shared__ float sh[2][8][4];
  int turn = 0;
  constexpr int kPer = block_size<G>() / G;
  const int lane = threadIdx.x % G;
  const int64_t t = (int64_t)blockIdx.x * kPer + threadIdx.x / G;
  const bool row_on = t < T;
  const int64_t base = (row_on ? t : T - 1) * emb;  // groups past the last row compute it again and store nothing
  const int nch = emb / 8;
  const float inv = 1.0f / emb;

  float v[kCh][8];
  if constexpr (SRC == 1) {
#pragma unroll
    for (int i = 0; i < kCh; ++i)
      if (i * G + lane < nch) load8(y, false, base + (i * G + lane) * 8, v[i]);
  }
  if constexpr (SRC == 2) {
    const int64_t tt = row_on ? t : T - 1, S = T * k;
    const int l = threadIdx.x & 63;
    int32_t my_r = -1;
    float my_w = 0;
    if (l < k) {
      const int32_t r = slot_row[tt * k + l];
      if (r >= 0 && r < S) my_r = r, my_w = topk_w ? topk_w[tt * k + l] : 1.0f;
    }
#pragma unroll
    for (int i = 0; i < kCh; ++i) {
#pragma unroll
      for (int u = 0; u < 8; ++u) v[i][u] = 0;
      if (i * G >= nch) continue;
      const bool on = i * G + lane < nch;
      for (int j0 = 0; j0 < k; j0 += 8) {
        u32x4_t q[8];
        float ww[8];
        bool use[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int32_t r = __shfl(my_r, (j0 + u) & 63);
          ww[u] = __shfl(my_w, (j0 + u) & 63);
          use[u] = on && j0 + u < k && r >= 0;
          if (use[u])
            q[u] = __builtin_nontemporal_load(
                reinterpret_cast<const u32x4_t*>(ys + (int64_t)r * emb + (i * G + lane) * 8));
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if (!use[u]) continue;
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            v[i][2 * m] = __builtin_fmaf(ww[u], bf16_lo(q[u][m]), v[i][2 * m]);
            v[i][2 * m + 1] = __builtin_fmaf(ww[u], bf16_hi(q[u][m]), v[i][2 * m + 1]);
          }
        }
      }
      if (y_out && on && row_on) store8(y_out, false, base + (i * G + lane) * 8, v[i]);
    }
  }
  if constexpr (SRC > 0) {
    float r = b.scale;
    if (b.post) {
      float s[1] = {0};
#pragma unroll
      for (int i = 0; i < kCh; ++i) {
        if (i * G + lane >= nch) continue;
#pragma unroll
        for (int u = 0; u < 8; ++u) s[0] = __builtin_fmaf(v[i][u], v[i][u], s[0]);
      }
      row_sums<G>(s, sh, turn);
      r *= rsqrtf(s[0] * inv + b.eps);
    }
    if (b.gate_mode == kGateToken) r *= load1(b.gate, b.gate_f32, row_on ? t : T - 1);
#pragma unroll
    for (int i = 0; i < kCh; ++i) {
      const int n = (i * G + lane) * 8;
      if (n >= emb) continue;
      float f[8], x[8];
      load8(res, b.x_f32, base + n, x);
      if (b.post && b.post_weight) {
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
      for (int u = 0; u < 8; ++u) v[i][u] = __builtin_fmaf(r, v[i][u], b.res_scale * x[u]);
      if (row_on) store8(out, b.x_f32, base + n, v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kCh; ++i)
      if (i * G + lane < nch) load8(res, b.x_f32, base + (i * G + lane) * 8, v[i]);
  }
  // the next norm takes the sum before it is rounded to the residual's type
  if (SRC > 0 && !xn) return;
  float s[1] = {0};
#pragma unroll
  for (int i = 0; i < kCh; ++i) {
    if (i * G + lane >= nch) continue;
#pragma unroll
    for (int u = 0; u < 8; ++u) s[0] = __builtin_fmaf(v[i][u], v[i][u], s[0]);
  }
  row_sums<G>(s, sh, turn);
  const float r = rsqrtf(s[0] * inv + b.eps);
#pragma unroll
  for (int i = 0; i < kCh; ++i) {
    const int n = (i * G + lane) * 8;
    if (n >= emb || !row_on) continue;
    float f[8];
    factor8(b.next_weight, b.w_f32, b.offset, n, f);
#pragma unroll
    for (int u = 0; u < 8; ++u) f[u] *= v[i][u] * r;
    store8(xn, false, base + n, f);
  }
}

// Backward, for d = the gradient of out. With NEXT, d = dout + r (g - o c), g = dxn (offset + w_next), o = out,
// c = r^2 mean(g o). Then dres = res_scale d, and with dz = scale gate d: dy = dz, or with POST
// r_y (h - y c_y), h = dz (offset + w_post), c_y = r_y^2 mean(h y). Column sums (the weights' gradients dxn o r and
// dz y r_y, a channel gate's scale d z) are kept in registers over all rows of a workgroup and leave it as one
// partial row each; moe_colsum adds those up in order.
// HASY false: d alone is wanted (moe_norm_bwd).
template <int G, bool HASY, bool NEXT, bool POST, bool CHG>
__global__ __launch_bounds__(block_size<G>()) void block_out_bwd_kernel(int64_t T, int emb, BlockArgs b, const void* dout,
                                                                        const uint16_t* __restrict__ y, const void* out,
                                                                        const uint16_t* __restrict__ dxn, void* dres,
                                                                        uint16_t* __restrict__ dy,
                                                                        void* __restrict__ dgate,
                                                                        float* __restrict__ part) {
  constexpr int kB = block_size<G>(), kPer = kB / G;
  constexpr int kAcc = (NEXT ? 1 : 0) + (POST ? 1 : 0) + (CHG ? 1 : 0);
  constexpr int kAccPost = NEXT ? 1 : 0, kAccGate = kAccPost + (POST ? 1 : 0);
  __shared__ float sh[2][8][4];
  __shared__ float comb[kPer > 1 ? kPer - 1 : 1][kPer > 1 ? G * 8 : 1];
  int turn = 0;
  const int lane = threadIdx.x % G, grp = threadIdx.x / G;
  const float inv = 1.0f / emb;
  float acc[kAcc > 0 ? kAcc : 1][kCh][8];
#pragma unroll
  for (int a = 0; a < kAcc; ++a)
#pragma unroll
    for (int i = 0; i < kCh; ++i)
#pragma unroll
      for (int u = 0; u < 8; ++u) acc[a][i][u] = 0;

  for (int64_t t0 = (int64_t)blockIdx.x * kPer; t0 < T; t0 += (int64_t)gridDim.x * kPer) {
    const bool row_on = t0 + grp < T;
    const int64_t t = row_on ? t0 + grp : T - 1;
    const int64_t base = t * emb;
    float d[kCh][8], yv[kCh][8];
    float s[3] = {0, 0, 0};
    float o[kCh][8], g[kCh][8];
#pragma unroll
    for (int i = 0; i < kCh; ++i) {
      const int n = (i * G + lane) * 8;
      if (n >= emb) continue;
      if constexpr (NEXT) {
        load8(out, b.x_f32, base + n, o[i]);
        load8(dxn, false, base + n, g[i]);
      }
      if (dout) load8(dout, b.x_f32, base + n, d[i]);
      else {
#pragma unroll
        for (int u = 0; u < 8; ++u) d[i][u] = 0;
      }
      if constexpr (HASY) {
        if (y) load8(y, false, base + n, yv[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kCh; ++i) {
      const int n = (i * G + lane) * 8;
      if (n >= emb) continue;
      if constexpr (NEXT) {
        float f[8];
        factor8(b.next_weight, b.w_f32, b.offset, n, f);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          s[0] = __builtin_fmaf(o[i][u], o[i][u], s[0]);
          s[1] = __builtin_fmaf(g[i][u] * f[u], o[i][u], s[1]);
        }
      }
      if constexpr (POST) {
#pragma unroll
        for (int u = 0; u < 8; ++u) s[2] = __builtin_fmaf(yv[i][u], yv[i][u], s[2]);
      }
    }
    if constexpr (NEXT || POST) row_sums<G>(s, sh, turn);
    const float r = NEXT ? rsqrtf(s[0] * inv + b.eps) : 0.0f, c = r * r * (s[1] * inv);
    const float ry = POST ? rsqrtf(s[2] * inv + b.eps) : 1.0f;
    const float tok = b.gate_mode == kGateToken ? load1(b.gate, b.gate_f32, t) : 1.0f;
    float q[1] = {0};
#pragma unroll
    for (int i = 0; i < kCh; ++i) {
      const int n = (i * G + lane) * 8;
      if (n >= emb) continue;
      if constexpr (NEXT) {
        float f[8];
        factor8(b.next_weight, b.w_f32, b.offset, n, f);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          d[i][u] += r * (g[i][u] * f[u] - o[i][u] * c);
          if (row_on) acc[0][i][u] = __builtin_fmaf(g[i][u], o[i][u] * r, acc[0][i][u]);
        }
      }
      if (row_on && dres) {
        float e[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) e[u] = b.res_scale * d[i][u];
        store8(dres, b.x_f32, base + n, e);
      }
      if constexpr (HASY) {
        float f[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) d[i][u] *= b.scale;
        if (POST) factor8(b.post_weight, b.w_f32, b.offset, n, f);
        else {
#pragma unroll
          for (int u = 0; u < 8; ++u) f[u] = 1.0f;
        }
        // d is scale * d now; z = y r_y f
        if (b.gate_mode == kGateChannel || b.gate_mode == kGateFull) {
          float gt[8], dg[8];
          load8(b.gate, b.gate_f32, (b.gate_mode == kGateFull ? base : 0) + n, gt);
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            dg[u] = d[i][u] * (yv[i][u] * ry * f[u]);
            if (CHG && row_on) acc[kAccGate < kAcc ? kAccGate : 0][i][u] += dg[u];
            d[i][u] *= gt[u];
          }
          if (b.gate_mode == kGateFull && dgate && row_on) store8(dgate, b.gate_f32, base + n, dg);
        }
        if (POST || b.gate_mode == kGateToken) {
#pragma unroll
          for (int u = 0; u < 8; ++u) q[0] = __builtin_fmaf(d[i][u] * f[u], yv[i][u], q[0]);
        }
        if constexpr (POST) {
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            if (row_on) acc[kAccPost < kAcc ? kAccPost : 0][i][u] = __builtin_fmaf(tok * d[i][u], yv[i][u] * ry, acc[kAccPost < kAcc ? kAccPost : 0][i][u]);
            d[i][u] *= f[u];
          }
        }
      }
    }
    if constexpr (HASY) {
      float cy = 0;
      if (POST || b.gate_mode == kGateToken) {
        row_sums<G>(q, sh, turn);
        cy = ry * ry * (q[0] * inv);
        if (b.gate_mode == kGateToken && dgate && lane == 0 && row_on) static_cast<float*>(dgate)[t] = q[0] * ry;
      }
      if (dy && row_on) {
#pragma unroll
        for (int i = 0; i < kCh; ++i) {
          const int n = (i * G + lane) * 8;
          if (n >= emb) continue;
          float e[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) e[u] = POST ? tok * ry * (d[i][u] - yv[i][u] * cy) : tok * d[i][u];
          store8(dy, false, base + n, e);
        }
      }
    }
  }
  if (!part) return;
  // the groups' sums, then one partial row per sum
#pragma unroll
  for (int a = 0; a < kAcc; ++a) {
#pragma unroll
    for (int i = 0; i < kCh; ++i) {
      const int n = (i * G + lane) * 8;
      if constexpr (kPer > 1) {
        if (i * G * 8 >= emb) continue;
        __syncthreads();
        if (grp > 0) {
#pragma unroll
          for (int u = 0; u < 8; ++u) comb[grp - 1][u * G + lane] = acc[a][i][u];
        }
        __syncthreads();
        if (grp == 0) {
#pragma unroll
          for (int p = 0; p < kPer - 1; ++p)
#pragma unroll
            for (int u = 0; u < 8; ++u) acc[a][i][u] += comb[p][u * G + lane];
        }
      }
      if (grp == 0 && n < emb) store8(part, true, ((int64_t)a * gridDim.x + blockIdx.x) * emb + n, acc[a][i]);
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

int lanes_of(int emb) {
  int g = 64;
  while (g * kCh * 8 < emb) g *= 2;
  return g;
}

// Workgroups of the backward: 2 a compute unit of the 256 (what their registers allow), fewer for few rows.
int bwd_grid(int64_t T, int emb) {
  const int g = lanes_of(emb), per = g < 256 ? 256 / g : 1;
  const int64_t n = (T + per - 1) / per;
  return (int)(n < 512 ? n : 512);
}

template <int G>
hipError_t fwd_g(int64_t T, int emb, const BlockArgs& b, const void* res, const uint16_t* y, int k, const uint16_t* ys,
                 const int32_t* slot_row, const float* w, void* out, uint16_t* xn, uint16_t* y_out, hipStream_t st) {
  constexpr int kB = block_size<G>(), kPer = kB / G;
  const dim3 grid((unsigned)((T + kPer - 1) / kPer));
  if (ys) block_out_kernel<G, 2><<<grid, kB, 0, st>>>(T, emb, b, res, y, k, ys, slot_row, w, out, xn, y_out);
  else if (y) block_out_kernel<G, 1><<<grid, kB, 0, st>>>(T, emb, b, res, y, k, ys, slot_row, w, out, xn, y_out);
  else block_out_kernel<G, 0><<<grid, kB, 0, st>>>(T, emb, b, res, y, k, ys, slot_row, w, out, xn, y_out);
  return hipGetLastError();
}

template <int G>
void bwd_g(int grid, int64_t T, int emb, const BlockArgs& b, bool has_y, const void* dout, const uint16_t* y,
           const void* out, const uint16_t* dxn, void* dres, uint16_t* dy, void* dgate, float* part, hipStream_t st) {
  constexpr int kB = block_size<G>();
  const bool post = b.post, chg = b.gate_mode == kGateChannel;
#define MOE_BWD(H, N, P, C) \
  block_out_bwd_kernel<G, H, N, P, C><<<dim3(grid), dim3(kB), 0, st>>>(T, emb, b, dout, y, out, dxn, dres, dy, dgate, part)
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
  switch (lanes_of(emb)) {
    case 64: return fwd_g<64>(T, emb, b, res, y, k, ys, slot_row, topk_w, out, xn, y_out, st);
    case 128: return fwd_g<128>(T, emb, b, res, y, k, ys, slot_row, topk_w, out, xn, y_out, st);
    case 256: return fwd_g<256>(T, emb, b, res, y, k, ys, slot_row, topk_w, out, xn, y_out, st);
    default: return fwd_g<512>(T, emb, b, res, y, k, ys, slot_row, topk_w, out, xn, y_out, st);
  }
}

size_t block_bwd_workspace(int64_t T, int emb, int sums) { return (size_t)bwd_grid(T, emb) * sums * emb * 4; }

hipError_t launch_block_out_bwd(int64_t T, int emb, const BlockArgs& b, bool has_y, const void* dout, const uint16_t* y,
                                const void* out, const uint16_t* dxn, void* dres, uint16_t* dy, float* dpost,
                                float* dnext, void* dgate, float* part, hipStream_t st) {
  const int grid = bwd_grid(T, emb);
  if (grid > 0) {
    switch (lanes_of(emb)) {
      case 64: bwd_g<64>(grid, T, emb, b, has_y, dout, y, out, dxn, dres, dy, dgate, part, st); break;
      case 128: bwd_g<128>(grid, T, emb, b, has_y, dout, y, out, dxn, dres, dy, dgate, part, st); break;
      case 256: bwd_g<256>(grid, T, emb, b, has_y, dout, y, out, dxn, dres, dy, dgate, part, st); break;
      default: bwd_g<512>(grid, T, emb, b, has_y, dout, y, out, dxn, dres, dy, dgate, part, st); break;
    }
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
    colsum_kernel<<<dim3((emb + 63) / 64, n), dim3(1024), 0, st>>>(grid, emb, part, c);
  return hipGetLastError();
}

}  // namespace moe
