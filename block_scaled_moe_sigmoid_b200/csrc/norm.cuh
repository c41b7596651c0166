// Residual addition, RMSNorm and MXFP8 quantisation in one pass over the row.
//
//   r  = x + residual, rounded to the residual's type (bf16 or fp32); without a residual, r = x
//   n  = r / sqrt(mean(r^2) + eps) * gamma          (fp32)
//   xn = bf16(n);  (q, scale) = the MX rule of quant_block_e4m3 on xn
//
// The norm reads the rounded r, so it is that of the residual the next layer will read, and the
// codes are made from the rounded xn, so they are the bytes that the layer's own quantiser makes
// of xn (two roundings, bf16 then E4M3, where one would do: prefill through xn and decode through
// q then see the same activations).
//
// Bound by memory: 2 (x) + 2 or 4 (residual) in, 2 or 4 (residual) + 2 (xn) + 1 + 1/32 out per
// element.  A row's team of threads keeps its elements in registers between the two uses, so each
// byte moves once.
#pragma once
#include "kernels.cuh"

namespace moe {

enum { NORM_RES_NONE = 0, NORM_RES_BF16 = 1, NORM_RES_F32 = 2 };
constexpr int kNormMaxCols = 32768;   // 1024 threads x 4 vectors of 8 elements

struct NormArgs {
  const uint16_t* x;
  const void* res;
  const float* gamma;
  float eps;
  int rows, cols;
  void* res_out;
  uint16_t* xn;
  uint8_t* q;
  uint8_t* scale;
};

__device__ __forceinline__ void unpack_bf16x8(const uint4& p, float (&v)[8]) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack_bf16x8(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    w[j] = *(const uint32_t*)&p;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// blockDim = (threads per row, a multiple of 32; rows per CTA).  Thread i of a row's team holds
// the 8-element vectors i, i + team, ... (V of them): 4 neighbouring lanes hold a 32-element block.
template <int RES, int V>
__global__ void __launch_bounds__(1024) add_rmsnorm_mxfp8_kernel(const NormArgs a) {
  __shared__ float part[32];
  griddep_wait();
  griddep_launch_dependents();
  const int team = blockDim.x;
  const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const int nvec = row < a.rows ? a.cols >> 3 : 0;
  const size_t base = (size_t)(row < a.rows ? row : 0) * a.cols;
  float v[V][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * team;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    if (c < nvec) {
      unpack_bf16x8(((const uint4*)(a.x + base))[c], v[i]);
      if constexpr (RES == NORM_RES_BF16) {
        float r[8];
        unpack_bf16x8(((const uint4*)((const uint16_t*)a.res + base))[c], r);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += r[j];
        const uint4 p = pack_bf16x8(v[i]);
        unpack_bf16x8(p, v[i]);
        if (a.res_out) ((uint4*)((uint16_t*)a.res_out + base))[c] = p;
      } else if constexpr (RES == NORM_RES_F32) {
        const float4* src = (const float4*)((const float*)a.res + base) + 2 * c;
        const float4 lo = src[0], hi = src[1];
        v[i][0] += lo.x; v[i][1] += lo.y; v[i][2] += lo.z; v[i][3] += lo.w;
        v[i][4] += hi.x; v[i][5] += hi.y; v[i][6] += hi.z; v[i][7] += hi.w;
        if (a.res_out) {
          float4* dst = (float4*)((float*)a.res_out + base) + 2 * c;
          dst[0] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
          dst[1] = make_float4(v[i][4], v[i][5], v[i][6], v[i][7]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
  }
  if (!a.xn && !a.q) return;   // the same for the whole grid
  // the row's sum of squares, in a fixed order: per thread, per warp, per team
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const int wpr = team >> 5;   // warps per row
  if (wpr > 1) {
    const int w = threadIdx.y * wpr + (threadIdx.x >> 5);
    if ((threadIdx.x & 31) == 0) part[w] = ss;
    __syncthreads();
    ss = 0.0f;
    for (int i = 0; i < wpr; ++i) ss += part[threadIdx.y * wpr + i];
  }
  const float inv = rsqrtf(ss / (float)a.cols + a.eps);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * team;
    const bool ok = c < nvec;
    if (ok) {
      const float4* g = (const float4*)a.gamma + 2 * c;
      const float4 lo = __ldg(g), hi = __ldg(g + 1);
      v[i][0] *= inv * lo.x; v[i][1] *= inv * lo.y; v[i][2] *= inv * lo.z; v[i][3] *= inv * lo.w;
      v[i][4] *= inv * hi.x; v[i][5] *= inv * hi.y; v[i][6] *= inv * hi.z; v[i][7] *= inv * hi.w;
    }
    const uint4 p = pack_bf16x8(v[i]);
    if (ok && a.xn) ((uint4*)(a.xn + base))[c] = p;
    if (a.q) {
      unpack_bf16x8(p, v[i]);
      float amax = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[i][j]));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int e = mx_scale_exp(amax, 8);
      const float s = pow2_neg(e);
      uint32_t w[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        w[j] = cvt_e4m3x2(v[i][4 * j] * s, v[i][4 * j + 1] * s) |
               (cvt_e4m3x2(v[i][4 * j + 2] * s, v[i][4 * j + 3] * s) << 16);
      if (ok) {
        ((uint2*)(a.q + base))[c] = make_uint2(w[0], w[1]);
        if ((c & 3) == 0) a.scale[(base >> 5) + (c >> 2)] = (uint8_t)(e + 127);
      }
    }
  }
}

}  // namespace moe
