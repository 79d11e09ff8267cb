// Activation checkpoints in 8 bits, and the elementwise half of their use in
// the layer's backward pass.
//
// Format (OCP microscaling, INT8 elements): 32 consecutive elements of a row
// share a power-of-two scale held as E8M0 (code c is 2^(c-127)); an element is
// an integer code in [-127, 127] worth code * 2^-6 * 2^(c-127). c is
// floor(log2(amax)) + 127 clamped to [1, 254], the code is v / step rounded to
// nearest (ties to even), step = 2^(c-133). An element is off by at most half
// a step, 2^-7 of the block's largest power of two (one step for a magnitude
// past 127.5 steps, which saturates). Integers rather than E4M3 elements: the
// step is the same over a block, so a normal row comes back with about a third
// of E4M3's error at the same 8.25 bits an element. Every value is a bf16
// number (7 significant bits and a power of two), so reading back into bf16
// rounds nothing. A block with a NaN or an infinity gets c = 255 and reads
// back as NaN.
//
// Layout: codes [rows][K] int8, scales [rows][K/32] bytes, both as the row lies.
#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

// Eight consecutive elements of a row per thread; four threads share a block, whose maximum takes two lane
// exchanges. Bound by memory, so the source is read past the caches (it is not read again here) and the codes,
// which the backward reads, are stored through them. 58.7 M bf16 values: 33-34 us, 5.2-5.4 TB/s; 100.7 M fp32
// values: 87 us, 5.8 TB/s.
template <bool BF16>
__global__ __launch_bounds__(256) void ckpt_quantize_kernel(const void* __restrict__ src, int64_t n8,
                                                            int8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  // n8 is a multiple of 4, so a block's four threads are in or out together
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += (int64_t)gridDim.x * 256) {
    float x[8];
    if (BF16) {
      const u32x4_t v =
          __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(src) + i * 8));
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        x[2 * m] = bf16_lo(v[m]);
        x[2 * m + 1] = bf16_hi(v[m]);
      }
    } else {
      const f32x4_t* f = reinterpret_cast<const f32x4_t*>(static_cast<const float*>(src) + i * 8);
      const f32x4_t a = __builtin_nontemporal_load(f), b = __builtin_nontemporal_load(f + 1);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        x[m] = a[m];
        x[4 + m] = b[m];
      }
    }
    uint32_t am = 0;
#pragma unroll
    for (int m = 0; m < 8; ++m) am = max(am, __float_as_uint(x[m]) & 0x7fffffffu);
    am = max(am, (uint32_t)__shfl_xor((int)am, 1));
    am = max(am, (uint32_t)__shfl_xor((int)am, 2));
    const int c = ckpt_scale_code(am);
    const float inv = ckpt_inv_step(c);
    const u32x2_t o = {ckpt_codes4(x[0], x[1], x[2], x[3], inv), ckpt_codes4(x[4], x[5], x[6], x[7], inv)};
    *reinterpret_cast<u32x2_t*>(codes + i * 8) = o;
    if ((i & 3) == 0) scales[i >> 2] = (uint8_t)c;
  }
}

// Bound by memory: 58.7 M values to bf16 in 29 us (6.1 TB/s, the codes partly from the Infinity Cache), 100.7 M
// in 48 us (6.4 TB/s).
// Eight elements per thread of destination row r, from source row row_index[r] / row_div (clamped) or r.
template <bool BF16>
__global__ __launch_bounds__(256) void ckpt_dequantize_kernel(const int8_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales, int64_t src_rows,
                                                              int K, const int32_t* __restrict__ row_index,
                                                              int row_div, int64_t M, void* __restrict__ dst) {
  const int per_row = K / 8;
  const int64_t n = M * per_row;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / per_row;
    const int c8 = (int)(i - r * per_row);
    int64_t sr = r;
    if (row_index) {
      sr = row_index[r] / row_div;
      sr = sr < 0 ? 0 : (sr >= src_rows ? src_rows - 1 : sr);
    }
    const u32x2_t v = *reinterpret_cast<const u32x2_t*>(codes + sr * K + (int64_t)c8 * 8);
    const float step = ckpt_step(scales[sr * (K / 32) + (c8 >> 2)]);
    float x[8];
#pragma unroll
    for (int m = 0; m < 8; ++m) x[m] = (float)((int32_t)(v[m >> 2] << (24 - 8 * (m & 3))) >> 24) * step;
    if (BF16) {
      u32x4_t o;
#pragma unroll
      for (int m = 0; m < 4; ++m) o[m] = pack_bf16x2(x[2 * m], x[2 * m + 1]);
      __builtin_nontemporal_store(o, reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(dst) + i * 8));
    } else {
      f32x4_t* f = reinterpret_cast<f32x4_t*>(static_cast<float*>(dst) + i * 8);
      // through the caches, which join the two halves of a lane's 32 bytes: past them 3.5 TB/s instead of 5.6
      f[0] = f32x4_t{x[0], x[1], x[2], x[3]};
      f[1] = f32x4_t{x[4], x[5], x[6], x[7]};
    }
  }
}

// SwiGLU backward from the 8-bit h = [gate | up] of row r, LPR lanes a row (64 / LPR rows a wave), 8 columns a
// lane and round. q = row_slot[r] (or r), w = slot_scale[q] (or 1), s = sigmoid(g):
//   a = g s u,  dh = [w da u s (1 + g (1 - s)) | w da g s],  dslot_scale[q] = sum_m da a (a unrounded)
// Bound by memory: 4 bytes read and 6 written a column; 262144 rows of 768 take 357-365 us, 5.6-5.7 TB/s by the
// counters too. The outputs are read by other kernels much later and the inputs not again: both go past the caches.
template <int LPR>
__global__ __launch_bounds__(256) void swiglu_bwd_ckpt_kernel(int64_t M, int mlp, const uint16_t* __restrict__ da,
                                                              const int8_t* __restrict__ hc,
                                                              const uint8_t* __restrict__ hs,
                                                              const int32_t* __restrict__ row_slot,
                                                              const float* __restrict__ slot_scale,
                                                              uint16_t* __restrict__ dh, uint16_t* __restrict__ a,
                                                              float* __restrict__ dscale) {
  const int lane = threadIdx.x & (LPR - 1);
  const int nch = mlp / 8;
  // (a launch holds 2^32 lanes of x at most)
  const int64_t r = (((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x) / LPR;
  if (r >= M) return;  // whole rows leave together; the sum below stays within a row's lanes
  const int64_t q = row_slot ? row_slot[r] : r;
  const bool inside = q >= 0 && q < M;
  const float w = inside ? (slot_scale ? slot_scale[q] : 1.0f) : 0.0f;
  float dot = 0.0f;
  for (int c = lane; c < nch; c += LPR) {
    const u32x4_t dv = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(da + r * mlp + c * 8));
    const u32x2_t gv = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(hc + r * 2 * mlp + c * 8));
    const u32x2_t uv = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(hc + r * 2 * mlp + mlp + c * 8));
    const float gst = ckpt_step(hs[r * (mlp / 16) + (c >> 2)]);
    const float ust = ckpt_step(hs[r * (mlp / 16) + mlp / 32 + (c >> 2)]);
    float og[8], ou[8], oa[8];
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      const float g = (float)((int32_t)(gv[m >> 2] << (24 - 8 * (m & 3))) >> 24) * gst;
      const float u = (float)((int32_t)(uv[m >> 2] << (24 - 8 * (m & 3))) >> 24) * ust;
      const float d = (m & 1) ? bf16_hi(dv[m >> 1]) : bf16_lo(dv[m >> 1]);
      const float s = 1.0f / (1.0f + expf(-g));
      const float gs = g * s;
      oa[m] = gs * u;
      dot = __builtin_fmaf(d, oa[m], dot);
      const float dw = d * w;
      og[m] = dw * u * (s * (1.0f + g * (1.0f - s)));
      ou[m] = dw * gs;
    }
    u32x4_t vg, vu, va;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      vg[m] = pack_bf16x2(og[2 * m], og[2 * m + 1]);
      vu[m] = pack_bf16x2(ou[2 * m], ou[2 * m + 1]);
      va[m] = pack_bf16x2(oa[2 * m], oa[2 * m + 1]);
    }
    __builtin_nontemporal_store(vg, reinterpret_cast<u32x4_t*>(dh + r * 2 * mlp + c * 8));
    __builtin_nontemporal_store(vu, reinterpret_cast<u32x4_t*>(dh + r * 2 * mlp + mlp + c * 8));
    if (a) __builtin_nontemporal_store(va, reinterpret_cast<u32x4_t*>(a + r * mlp + c * 8));
  }
  if (dscale) {
#pragma unroll
    for (int s = LPR / 2; s >= 1; s >>= 1) dot += __shfl_xor(dot, s);
    if (lane == 0 && inside) dscale[q] = dot;
  }
}

unsigned grid_of(int64_t items, int64_t per_block) {
  const int64_t b = (items + per_block - 1) / per_block;
  return (unsigned)(b < (int64_t(1) << 22) ? b : (int64_t(1) << 22));
}

}  // namespace

hipError_t launch_ckpt_quantize(const void* src, bool src_bf16, int64_t M, int K, int8_t* codes, uint8_t* scales,
                                hipStream_t stream) {
  const int64_t n8 = M * (K / 8);
  if (n8 == 0) return hipSuccess;
  if (src_bf16)
    ckpt_quantize_kernel<true><<<dim3(grid_of(n8, 256)), dim3(256), 0, stream>>>(src, n8, codes, scales);
  else
    ckpt_quantize_kernel<false><<<dim3(grid_of(n8, 256)), dim3(256), 0, stream>>>(src, n8, codes, scales);
  return hipGetLastError();
}

hipError_t launch_ckpt_dequantize(const int8_t* codes, const uint8_t* scales, int64_t src_rows, int K,
                                  const int32_t* row_index, int row_div, int64_t M, void* dst, bool dst_bf16,
                                  hipStream_t stream) {
  if (M == 0) return hipSuccess;
  const dim3 grid(grid_of(M * (K / 8), 256));
  if (dst_bf16)
    ckpt_dequantize_kernel<true><<<grid, dim3(256), 0, stream>>>(codes, scales, src_rows, K, row_index, row_div, M,
                                                                 dst);
  else
    ckpt_dequantize_kernel<false><<<grid, dim3(256), 0, stream>>>(codes, scales, src_rows, K, row_index, row_div, M,
                                                                  dst);
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd_ckpt(int64_t M, int mlp, const uint16_t* da, const int8_t* h_codes,
                                  const uint8_t* h_scales, const int32_t* row_slot, const float* slot_scale,
                                  uint16_t* dh, uint16_t* a, float* dslot_scale, hipStream_t stream) {
  if (M == 0) return hipSuccess;
  // lanes a row: the most of 64, 32, 16, 8 that keep more than three quarters of them busy over the
  // rounds. Against 64 throughout: 2^20 rows of 64 columns 671 -> 135 us, of 128 668 -> 250, 2^18 of 320 196 ->
  // 165. Against the fewest idle, whole rows on 8 lanes at an odd width: 448, 960 and 1984 columns 4.4, 4.2 and
  // 3.8 -> 5.7, 5.7 and 5.3 TB/s.
  const int nch = mlp / 8;
  int lpr = 64;
  while (lpr > 8 && nch * 4LL <= 3LL * ((nch + lpr - 1) / lpr) * lpr) lpr /= 2;
  const int64_t blocks = (M * lpr + 255) / 256;
  const unsigned gx = grid_of(blocks, 1);
  const dim3 grid(gx, (unsigned)((blocks + gx - 1) / gx)), block(256);
#define MOE_SWIGLU_BWD(L)                                                                                       \
  swiglu_bwd_ckpt_kernel<L><<<grid, block, 0, stream>>>(M, mlp, da, h_codes, h_scales, row_slot, slot_scale, dh, a, \
                                                        dslot_scale)
  if (lpr == 64) MOE_SWIGLU_BWD(64);
  else if (lpr == 32) MOE_SWIGLU_BWD(32);
  else if (lpr == 16) MOE_SWIGLU_BWD(16);
  else MOE_SWIGLU_BWD(8);
#undef MOE_SWIGLU_BWD
  return hipGetLastError();
}

}  // namespace moe
