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

// r of one vector from its x and residual; a bf16 r is stored here where it is wanted.
template <int RES>
__device__ __forceinline__ void norm_add(const NormArgs& a, size_t base, int c, const uint4& x, const uint4& r0, const uint4& r1,
                                         float (&v)[8]) {
  unpack_bf16x8(x, v);
  if constexpr (RES == NORM_RES_BF16) {
    float r[8];
    unpack_bf16x8(r0, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += r[j];
    const uint4 p = pack_bf16x8(v);
    unpack_bf16x8(p, v);
    if (a.res_out) ((uint4*)((uint16_t*)a.res_out + base))[c] = p;
  } else if constexpr (RES == NORM_RES_F32) {
    const uint32_t r[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += __uint_as_float(r[j]);
  }
}

// A warp's part of the row's sum of squares.
__device__ __forceinline__ float norm_warp_sum(float ss) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  return ss;
}

// xn and the MX codes of one vector (4 neighbouring lanes hold a 32-element block).
__device__ __forceinline__ void norm_store(const NormArgs& a, size_t base, int c, bool ok, float inv, float (&v)[8]) {
  if (ok) {
    const float4* g = (const float4*)a.gamma + 2 * c;
    const float4 lo = __ldg(g), hi = __ldg(g + 1);
    v[0] *= inv * lo.x; v[1] *= inv * lo.y; v[2] *= inv * lo.z; v[3] *= inv * lo.w;
    v[4] *= inv * hi.x; v[5] *= inv * hi.y; v[6] *= inv * hi.z; v[7] *= inv * hi.w;
  }
  const uint4 p = pack_bf16x8(v);
  if (ok && a.xn) ((uint4*)(a.xn + base))[c] = p;
  if (a.q) {
    unpack_bf16x8(p, v);
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int e = mx_scale_exp(amax, 8);
    const float s = pow2_neg(e);
    uint32_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      w[j] = cvt_e4m3x2(v[4 * j] * s, v[4 * j + 1] * s) | (cvt_e4m3x2(v[4 * j + 2] * s, v[4 * j + 3] * s) << 16);
    if (ok) {
      ((uint2*)(a.q + base))[c] = make_uint2(w[0], w[1]);
      if ((c & 3) == 0) a.scale[(base >> 5) + (c >> 2)] = (uint8_t)(e + 127);
    }
  }
}

// Thread i of a row's team (a multiple of 32 threads) holds the 8-element vectors i, i + team, ... (V of
// them).  The row's sum of squares is taken per thread, per warp, per team: a fixed order.

// A row per team, straight through registers; blockDim = (team, rows per CTA).
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
      uint4 r0 = {}, r1 = {};
      if constexpr (RES == NORM_RES_BF16) r0 = ((const uint4*)((const uint16_t*)a.res + base))[c];
      if constexpr (RES == NORM_RES_F32) {
        const uint4* src = (const uint4*)((const float*)a.res + base) + 2 * c;
        r0 = src[0];
        r1 = src[1];
      }
      norm_add<RES>(a, base, c, ((const uint4*)(a.x + base))[c], r0, r1, v[i]);
      if (RES == NORM_RES_F32 && a.res_out) {
        float4* dst = (float4*)((float*)a.res_out + base) + 2 * c;
        dst[0] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
        dst[1] = make_float4(v[i][4], v[i][5], v[i][6], v[i][7]);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
  }
  if (!a.xn && !a.q) return;   // the same for the whole grid
  ss = norm_warp_sum(ss);
  const int wpr = team >> 5;   // warps per row
  if (wpr > 1) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.y * wpr + (threadIdx.x >> 5)] = ss;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    ss = norm_warp_sum(lane < wpr ? part[threadIdx.y * wpr + lane] : 0.0f);
  }
  const float inv = __frsqrt_rn(ss / (float)a.cols + a.eps);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * team;
    norm_store(a, base, c, c < nvec, inv, v[i]);
  }
}

// Many wide rows: a resident grid walks the rows, a CTA each, and every thread keeps the loads of its
// next three rows in flight (cp.async into shared memory that only it reads, so nothing waits but the row's sum).
// 8192 x 7168 with a bf16 residual: 85.6 us, 6.2 TB/s, where a CTA per row takes 96 us (its loads stop
// while it reduces and stores).  With an fp32 residual a CTA per row has enough loads in flight (117 us,
// 6.5 TB/s) and the ring would hold too few rows (134 us).
constexpr int kNormDepth = 3, kNormStreamVecsPerThread = 2;
__device__ __forceinline__ void cp_async_16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
template <int RES>
__global__ void __launch_bounds__(1024) add_rmsnorm_mxfp8_stream_kernel(const NormArgs a) {
  static_assert(RES != NORM_RES_F32, "fp32 residuals take a CTA per row");
  constexpr int V = kNormStreamVecsPerThread;
  constexpr int PIECES = RES == NORM_RES_BF16 ? 2 : 1;   // 16-byte pieces of a vector: x, residual
  extern __shared__ uint4 ring[];                        // [kNormDepth][V][PIECES][threads]
  __shared__ float part[2][32];
  griddep_wait();
  griddep_launch_dependents();
  const int team = blockDim.x, tid = threadIdx.x, nvec = a.cols >> 3;
  auto slot = [&](int st, int i, int pc) { return ring + ((st * V + i) * PIECES + pc) * team + tid; };
  auto load = [&](long long row, int st) {
    if (row < a.rows) {
      const size_t base = (size_t)row * a.cols;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = tid + i * team;
        if (c >= nvec) continue;
        cp_async_16(slot(st, i, 0), (const uint4*)(a.x + base) + c);
        if constexpr (RES == NORM_RES_BF16) cp_async_16(slot(st, i, 1), (const uint4*)((const uint16_t*)a.res + base) + c);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int d = 0; d < kNormDepth; ++d) load(blockIdx.x + (long long)d * gridDim.x, d);
  int st = 0, turn = 0;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const size_t base = (size_t)row * a.cols;
    asm volatile("cp.async.wait_group %0;" ::"n"(kNormDepth - 1) : "memory");
    float v[V][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * team;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
      if (c < nvec) {
        uint4 r0 = {};
        if constexpr (RES == NORM_RES_BF16) r0 = *slot(st, i, 1);
        norm_add<RES>(a, base, c, *slot(st, i, 0), r0, r0, v[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    }
    load(row + (long long)kNormDepth * gridDim.x, st);
    if (++st == kNormDepth) st = 0;
    if (!a.xn && !a.q) continue;   // the same for the whole grid
    ss = norm_warp_sum(ss);
    if ((tid & 31) == 0) part[turn][tid >> 5] = ss;
    __syncthreads();   // the next turn writes the other half: one barrier a row is enough
    ss = norm_warp_sum((tid & 31) < team >> 5 ? part[turn][tid & 31] : 0.0f);
    const float inv = __frsqrt_rn(ss / (float)a.cols + a.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * team;
      norm_store(a, base, c, c < nvec, inv, v[i]);
    }
  }
}

}  // namespace moe
