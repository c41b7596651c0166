// Matrix products with MXFP4 weights for a few token rows (T <= 8): a stream of the weights.
//
//   FEW_LINEAR  y[t] = W x[t]                                    one matrix, x in MXFP8
//   FEW_GLU     h[t,j] = MX(glu(Wg x[t], Wu x[t]))               the experts e = idx[t][j]
//   FEW_DOWN    y[t] = bf16(ys[t] + sum_j w[t][j] Wd h[t,j])     the same experts
//
// With so few rows every weight byte is used once and the bytes are the cost: 17/32 byte per
// weight at the copy rate of the memory.  The work is one list of steps, a step being one 256-row
// x 128-column tile of packed weights (16 KB of codes, one contiguous block, and 1 KB of scales).
// CTA c of G takes the steps [c S / G, (c + 1) S / G): every SM streams the same number of bytes
// whatever the number of experts, rows or columns.  Where a CTA's range begins or ends inside a
// tile's contraction it writes an fp32 partial, and the CTA that arrives last at the tile's counter
// adds the partials in the order of the CTAs (a fixed order: results do not depend on timing) and
// finishes the tile.  No CTA waits for another.
//
// FEW_DOWN contracts over (expert, column) in one go: the routing weight is folded into the scale
// of h, and a token that does not use an expert contributes zeros there, so a tile of y needs no
// other sum.
//
// A step's products run on mma.sync m16n8k16 (f16 operands, fp32 accumulation): the 256 weight
// rows are M, the up to 8 tokens N.  E2M1 and E4M3 values are exact in f16 and so are their products in
// fp32; each 32-element block is summed on its own and then added to the fp32 accumulator times
// the two block scales.  tcgen05 would need the 128-row x 128-byte padded operand in shared memory
// per 64 bytes loaded; with N = 8 the legacy instruction is far from its own limit here.
//
// Lane (g, c) = (lane / 4, lane % 4) reads 4 bytes = 8 codes of a weight row's block: the fragment's
// logical k order is permuted the same way on both sides, so that each operand is one load.  The
// tile is loaded with the 64-byte swizzle, which makes those reads free of bank conflicts.
#pragma once
#include "gemm.cuh"
#include "kernels.cuh"

namespace moe {

enum { FEW_LINEAR = 0, FEW_GLU = 1, FEW_DOWN = 2 };
constexpr int kFewRows = 8;                    // tokens per call
constexpr int kFewWarps = 16;                  // consumer warps: 8 row groups x 2 halves of a step's columns
constexpr int kFewThreads = 32 * (kFewWarps + 1);
constexpr int kFewTile = 256 * 64;             // bytes of codes per step
constexpr int kFewHRow = 144;                  // h image: 128 codes, 4 scales, padding, per (pair, K tile)
constexpr int kFewHStride = 160;               // the same in shared memory: 8 tokens, no bank conflicts
constexpr int kFewRedStride = 260;             // floats between the tokens of the tile sums
constexpr int kFewPart = kFewRows * 256;       // floats of a partial
constexpr int kFewMaxCtas = 256;               // bound on the grid (sizes partials and counters)
constexpr int kFewMaxStages = 12;
constexpr int kFewSmemMax = 232448;
constexpr int kNoSlot = 0x7fffffff;              // the token does not use the expert
constexpr int kFewMaxX = 80 * 1024;            // bytes of MXFP8 codes a CTA keeps resident

struct FewArgs {
  int T, k, E;
  int m_tiles, k_tiles;   // of one matrix
  int rows;               // valid output rows (FEW_LINEAR, FEW_DOWN)
  int K;                  // columns of x (FEW_LINEAR, FEW_GLU)
  int stages;
  const uint8_t* sf;      // weight scales, [matrix][m-tile][k-tile][1 KB]
  const int* idx;
  const float* w;
  const uint16_t* x;      // bf16 x, quantised here, or
  const uint8_t* xq;      // its MXFP8 codes and scales
  const uint8_t* xs;
  uint8_t* himg;          // [T k][k-tile of the down product][144]
  const float* ys;        // shared expert's output, or NULL
  void* y;
  int y_f32;
  float* part;            // [2 per CTA][T][256]
  unsigned int* counters; // [CTAs], zero between launches
  unsigned int* status;
};

// Shared-memory layout (byte offsets from a 1024-byte aligned base); host and device agree on it.
struct FewSmem {
  int sf, xst, red, x, sx, tab, ctrl, total;
};
__host__ __device__ inline FewSmem few_smem(int mode, int T, int k, int K, int stages) {
  FewSmem s;
  int o = stages * kFewTile;
  s.sf = o; o += stages * 1024;
  s.xst = o; if (mode == FEW_DOWN) o += stages * kFewRows * kFewHStride;
  s.red = o; o += kFewRows * kFewRedStride * 4;
  s.x = o; if (mode != FEW_DOWN) o += T * (K + 32);
  s.sx = o; if (mode != FEW_DOWN) o += K / 32 * kFewRows * 4;
  s.tab = o; if (mode != FEW_LINEAR) o += (256 + (3 + 2 * kFewRows) * T * k) * 4;
  o = (o + 15) & ~15;
  s.ctrl = o; o += 2 * kFewMaxStages * 8 + 64;
  s.total = o + 1024;
  return s;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
// 8 E2M1 codes -> four f16 pairs, in code order
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// 8 E4M3 codes -> four f16 pairs
__device__ __forceinline__ void e4m3x8_to_f16(uint2 v, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b16 p0, p1, p2, p3;\n\t"
      "mov.b32 {p0, p1}, %4;\n\t"
      "mov.b32 {p2, p3}, %5;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, p0;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, p1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %2, p2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %3, p3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(v.x), "r"(v.y));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// E8M0 byte -> 2^(b - 127); b = 0 is the subnormal 2^-127
__device__ __forceinline__ float e8m0_f32(uint32_t b) { return __uint_as_float(max(b << 23, 0x00400000u)); }
__device__ __forceinline__ float e8m0_byte_f32(uint32_t word, int j) { return e8m0_f32((word >> (8 * j)) & 0xFFu); }

__device__ __forceinline__ void few_bar() {   // the consumer warps
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kFewWarps) : "memory");
}

template <int MODE, int ACT>
__global__ void __launch_bounds__(kFewThreads, 1)
    few_kernel(const __grid_constant__ FewArgs a, const __grid_constant__ CUtensorMap tmW) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const FewSmem L = few_smem(MODE, a.T, a.k, a.K, a.stages);
  uint64_t* full_bar = (uint64_t*)(smem + L.ctrl);
  uint64_t* empty_bar = full_bar + kFewMaxStages;
  volatile int* abort_flag = (volatile int*)(empty_bar + kFewMaxStages);
  volatile int* s_last = abort_flag + 1;
  int* s_fills = (int*)(abort_flag + 2);
  int* s_used = (int*)(abort_flag + 3);
  // tables of the routed modes
  uint32_t* bitmap = (uint32_t*)(smem + L.tab);             // experts some token uses
  int* prefix = (int*)(bitmap + 128);                       // used experts before each word
  int* elist = prefix + 128;                                // the used experts, ascending
  const int slots = a.T * a.k;
  int* s_idx = elist + slots;
  float* s_w = (float*)(s_idx + slots);
  int* hrow = (int*)(s_w + slots);                          // [used expert][8]: the token's first slot j with it, or none
  float* hw = (float*)(hrow + slots * kFewRows);            // [used expert][8]: its routing weight
  float* red = (float*)(smem + L.red);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(smem_u32(full_bar + s), 1);
      mbar_init(smem_u32(empty_bar + s), kFewWarps);
    }
    *abort_flag = 0;
    *s_fills = 0;
    fence_mbar_init();
    prefetch_tmap(&tmW);
  }
  griddep_wait();
  griddep_launch_dependents();

  int used = 1;
  if constexpr (MODE != FEW_LINEAR) {
    const int n = slots;
    for (int i = tid; i < 128; i += kFewThreads) bitmap[i] = 0;
    for (int i = tid; i < slots * kFewRows; i += kFewThreads) { hrow[i] = kNoSlot; hw[i] = 0.0f; }
    __syncthreads();
    for (int i = tid; i < n; i += kFewThreads) {
      const int e = a.idx[i];
      s_idx[i] = e;
      if (MODE == FEW_DOWN) s_w[i] = a.w[i];
      if (e >= 0 && e < a.E) atomicOr(&bitmap[e >> 5], 1u << (e & 31));
      else if (blockIdx.x == 0) atomicOr(a.status, MOE_DEV_ERR_BOUNDS);   // an id outside [0, E): skipped
    }
    __syncthreads();
    if (warp == 0) {
      int c[4], tot = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) { c[i] = tot; tot += __popc(bitmap[4 * lane + i]); }
      int inc = tot;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) prefix[4 * lane + i] = inc - tot + c[i];
      if (lane == 31) *s_used = inc;
    }
    __syncthreads();
    used = *s_used;
    for (int i = tid; i < n; i += kFewThreads) {
      const int e = s_idx[i];
      if (e < 0 || e >= a.E) continue;
      const int u = prefix[e >> 5] + __popc(bitmap[e >> 5] & ((1u << (e & 31)) - 1u));
      elist[u] = e;
      atomicMin(&hrow[u * kFewRows + i / a.k], i % a.k);
    }
    __syncthreads();
    if constexpr (MODE == FEW_DOWN) {
      for (int i = tid; i < used * kFewRows; i += kFewThreads) {
        const int j0 = hrow[i];
        if (j0 == kNoSlot) continue;
        const int t = i % kFewRows, e = elist[i / kFewRows];
        float w = 0.0f;   // an expert named twice by a token counts with both weights
        for (int j = j0; j < a.k; ++j)
          if (s_idx[t * a.k + j] == e) w += s_w[t * a.k + j];
        hw[i] = w;
      }
    }
  }
  if constexpr (MODE != FEW_DOWN) {
    // x resident: codes [T][K + 32], scales as floats [K / 32][8]
    const int nb = a.K >> 5;
    float* sx = (float*)(smem + L.sx);
    for (int i = tid; i < kFewRows * nb; i += kFewThreads) {
      const int t = i % kFewRows, b = i / kFewRows;
      float sc = 0.0f;
      if (t < a.T) {
        uint32_t code[8];
        if (a.x) {
          const uint4* src = (const uint4*)(a.x + (size_t)t * a.K + b * 32);
          uint4 in[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) in[q] = src[q];
          sc = e8m0_f32(quant_block_e4m3(in, code));
        } else {
          const uint4* src = (const uint4*)(a.xq + (size_t)t * a.K + b * 32);
          const uint4 lo = src[0], hi = src[1];
          code[0] = lo.x; code[1] = lo.y; code[2] = lo.z; code[3] = lo.w;
          code[4] = hi.x; code[5] = hi.y; code[6] = hi.z; code[7] = hi.w;
          sc = e8m0_f32(a.xs[(size_t)t * nb + b]);
        }
        uint4* dst = (uint4*)(smem + L.x + t * (a.K + 32) + b * 32);
        dst[0] = make_uint4(code[0], code[1], code[2], code[3]);
        dst[1] = make_uint4(code[4], code[5], code[6], code[7]);
      }
      sx[b * kFewRows + t] = sc;
    }
  }
  __syncthreads();

  // this CTA's steps
  const int tiles = MODE == FEW_GLU ? used * a.m_tiles : a.m_tiles;
  const int KT = MODE == FEW_DOWN ? used * a.k_tiles : a.k_tiles;
  const long long total = (long long)tiles * KT;
  const long long G = total < (long long)gridDim.x ? total : (long long)gridDim.x;
  const int c = blockIdx.x;
  const int s0 = c < G ? (int)(c * total / G) : 0, s1 = c < G ? (int)((c + 1) * total / G) : 0;

  if (warp == kFewWarps) {
    // ------------------------------------------------------------- producer
    const uint64_t pol = policy_evict_first();
    int stage = 0, fills = 0;
    uint32_t phase = 0;
    int tile = KT ? s0 / KT : 0, kk = KT ? s0 % KT : 0;
    for (int s = s0; s < s1; ++s) {
      int ok = 1;
      if (lane == 0) ok = mbar_wait(smem_u32(empty_bar + stage), phase ^ 1, a.status, abort_flag);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      int u = 0, m = tile, kt = kk;
      if (MODE == FEW_GLU) { u = tile / a.m_tiles; m = tile % a.m_tiles; }
      if (MODE == FEW_DOWN) { u = kk / a.k_tiles; kt = kk % a.k_tiles; }
      const int e = MODE == FEW_LINEAR ? 0 : elist[u];
      const size_t blk = ((size_t)e * a.m_tiles + m) * a.k_tiles + kt;
      const uint32_t bar = smem_u32(full_bar + stage);
      int j = kNoSlot;
      int nh = 0;
      if constexpr (MODE == FEW_DOWN) {
        if (lane < kFewRows) j = hrow[u * kFewRows + lane];
        nh = __popc(__ballot_sync(0xffffffffu, j != kNoSlot));
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, kFewTile + 1024 + nh * kFewHRow);
        tma_load_2d(smem_u32(smem + stage * kFewTile), &tmW, bar, 0, (int)(blk * 256), pol);
        bulk_load(smem_u32(smem + L.sf + stage * 1024), a.sf + blk * 1024, 1024, bar);
      }
      __syncwarp();
      if constexpr (MODE == FEW_DOWN) {
        if (j != kNoSlot)
          bulk_load(smem_u32(smem + L.xst + (stage * kFewRows + lane) * kFewHStride),
                    a.himg + ((size_t)(lane * a.k + j) * a.k_tiles + kt) * kFewHRow, kFewHRow, bar);
      }
      ++fills;
      if (++kk == KT) { kk = 0; ++tile; }
      if (++stage == a.stages) { stage = 0; phase ^= 1; }
    }
    if (lane == 0) *s_fills = fills;
  } else {
    // ------------------------------------------------------------- consumers
    const int g = lane >> 2, q = lane & 3, half = warp >> 3, wr = (warp & 7) * 16;
    const uint32_t row_off = (uint32_t)(wr + g) * 64 + q * 4;
    const uint32_t sw_off = (uint32_t)(((wr + g) & 31) * 16 + ((wr + g) >> 5) * 4);
    const uint32_t sw_off8 = (uint32_t)(((wr + g + 8) & 31) * 16 + ((wr + g + 8) >> 5) * 4);
    const uint32_t swz = (uint32_t)((g >> 1) & 3);
    int stage = 0;
    uint32_t phase = 0;
    int tile = KT ? s0 / KT : 0;
    int s = s0;
    while (s < s1) {
      const int kb = s - tile * KT;                       // this segment: K steps [kb, ke) of the tile
      const int ke = min(KT, kb + (s1 - s));
      float acc[2][4] = {};
      int u = 0, kt = kb;
      if (MODE == FEW_DOWN) { u = kb / a.k_tiles; kt = kb % a.k_tiles; }
      for (int kk = kb; kk < ke; ++kk) {
        int ok = 1;
        if (lane == 0) ok = mbar_wait(smem_u32(full_bar + stage), phase, a.status, abort_flag);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (ok) {
          const uint32_t sW = smem_u32(smem + stage * kFewTile), sS = smem_u32(smem + L.sf + stage * 1024);
          uint32_t sw[2][2];
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            sw[m][0] = lds32(sS + m * 512 + sw_off);
            sw[m][1] = lds32(sS + m * 512 + sw_off8);
          }
          uint32_t xrow = 0, xsc[2] = {0, 0};
          bool have;
          float w2[2] = {1.0f, 1.0f};
          if constexpr (MODE == FEW_DOWN) {
            const uint32_t st = smem_u32(smem + L.xst + stage * kFewRows * kFewHStride);
            have = hrow[u * kFewRows + g] != kNoSlot;
            xrow = st + g * kFewHStride;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int t = 2 * q + i;
              // a token that does not use the expert: its columns are zeros, its scale a finite one
              xsc[i] = hrow[u * kFewRows + t] != kNoSlot ? lds32(st + t * kFewHStride + 128) : 0u;
              w2[i] = hw[u * kFewRows + t];
            }
          } else {
            have = g < a.T;
            xrow = smem_u32(smem + L.x) + g * (a.K + 32) + kt * 128;
          }
#pragma unroll
          for (int jj = 0; jj < 2; ++jj) {
            const int j = 2 * half + jj;
            const uint2 xv = have ? lds64(xrow + 32 * j + 8 * q) : make_uint2(0u, 0u);
            uint32_t b[4];
            e4m3x8_to_f16(xv, b);
            float sx[2];
            if constexpr (MODE == FEW_DOWN) {
              sx[0] = e8m0_byte_f32(xsc[0], j) * w2[0];
              sx[1] = e8m0_byte_f32(xsc[1], j) * w2[1];
            } else {
              const uint2 v = lds64(smem_u32(smem + L.sx) + ((kt * 4 + j) * kFewRows + 2 * q) * 4);
              sx[0] = __uint_as_float(v.x);
              sx[1] = __uint_as_float(v.y);
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const uint32_t addr = sW + m * 8192 + row_off + ((j ^ swz) << 4);
              uint32_t lo[4], hi[4];
              e2m1x8_to_f16(lds32(addr), lo);
              e2m1x8_to_f16(lds32(addr + 512), hi);
              float p[4] = {};
              mma_f16(p, lo[0], hi[0], lo[1], hi[1], b[0], b[1]);
              mma_f16(p, lo[2], hi[2], lo[3], hi[3], b[2], b[3]);
              const float r0 = e8m0_byte_f32(sw[m][0], j), r1 = e8m0_byte_f32(sw[m][1], j);
              acc[m][0] = fmaf(p[0], r0 * sx[0], acc[m][0]);
              acc[m][1] = fmaf(p[1], r0 * sx[1], acc[m][1]);
              acc[m][2] = fmaf(p[2], r1 * sx[0], acc[m][2]);
              acc[m][3] = fmaf(p[3], r1 * sx[1], acc[m][3]);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(empty_bar + stage));
        }
        if (MODE == FEW_DOWN && ++kt == a.k_tiles) { kt = 0; ++u; }
        if (MODE != FEW_DOWN) ++kt;
        if (++stage == a.stages) { stage = 0; phase ^= 1; }
      }
      // ---- the segment's sums: red[t][row]
      few_bar();   // the previous segment's readers are done
      if (half == 1) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) red[(2 * q + (i & 1)) * kFewRedStride + m * 128 + wr + g + 8 * (i >> 1)] = acc[m][i];
      }
      few_bar();
      if (half == 0) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) red[(2 * q + (i & 1)) * kFewRedStride + m * 128 + wr + g + 8 * (i >> 1)] += acc[m][i];
      }
      few_bar();
      bool finish = true;
      if (kb != 0 || ke != KT) {
        // part of the tile's contraction: publish it; the last of the tile's CTAs adds them up
        float* mine = a.part + (size_t)(2 * c + (kb == 0 ? 1 : 0)) * kFewPart;
        for (int i = tid; i < a.T * 256; i += 32 * kFewWarps) mine[i] = red[(i >> 8) * kFewRedStride + (i & 255)];
        __threadfence();
        few_bar();
        const long long t0 = (long long)tile * KT;
        const int c_lo = (int)(((t0 + 1) * G - 1) / total), c_hi = (int)(((t0 + KT) * G - 1) / total);
        if (tid == 0) {
          const bool last = atomicAdd(a.counters + c_lo, 1u) == (unsigned)(c_hi - c_lo);
          if (last) a.counters[c_lo] = 0;
          __threadfence();
          *s_last = last;
        }
        few_bar();
        finish = *s_last;
        if (finish) {
          for (int i = tid; i < a.T * 256; i += 32 * kFewWarps) {
            float v = __ldcg(a.part + (size_t)(2 * c_lo + 1) * kFewPart + i);
            for (int p = c_lo + 1; p <= c_hi; ++p) v += __ldcg(a.part + (size_t)(2 * p) * kFewPart + i);
            red[(i >> 8) * kFewRedStride + (i & 255)] = v;
          }
          few_bar();
        }
      }
      if (finish) {
        if constexpr (MODE == FEW_GLU) {
          // a warp per (token, 32-channel block): glu, then the block's MX codes and scale
          const int ux = tile / a.m_tiles, m = tile % a.m_tiles;
          for (int i = warp; i < a.T * 4; i += kFewWarps) {
            const int t = i >> 2, b = i & 3, j = hrow[ux * kFewRows + t];
            if (j == kNoSlot) continue;
            const float v = glu_f<ACT>(red[t * kFewRedStride + 32 * b + lane], red[t * kFewRedStride + 128 + 32 * b + lane]);
            const uint32_t amax = __reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7FFFFFFFu);
            const int e = mx_exp_e4m3(amax);
            uint8_t* dst = a.himg + ((size_t)(t * a.k + j) * a.m_tiles + m) * kFewHRow;
            dst[32 * b + lane] = (uint8_t)(f32x2_to_e4m3x2(v * __uint_as_float((uint32_t)(127 - e) << 23), 0.0f) & 0xFFu);
            if (lane == 0) dst[128 + b] = (uint8_t)(e + 127);
          }
        } else {
          for (int i = tid; i < a.T * 256; i += 32 * kFewWarps) {
            const int t = i >> 8, r = i & 255, row = tile * 256 + r;
            if (row >= a.rows) continue;
            const size_t o = (size_t)t * a.rows + row;
            float v = red[t * kFewRedStride + r];
            if (MODE == FEW_DOWN && a.ys) v += a.ys[o];
            if (MODE == FEW_LINEAR && a.y_f32) ((float*)a.y)[o] = v;
            else ((__nv_bfloat16*)a.y)[o] = __float2bfloat16_rn(v);
          }
        }
      }
      s += ke - kb;
      ++tile;
    }
    if (MODE == FEW_DOWN && total == 0) {
      // every id was invalid: the shared expert's output alone
      for (size_t i = (size_t)c * 32 * kFewWarps + tid; i < (size_t)a.T * a.rows; i += (size_t)gridDim.x * 32 * kFewWarps)
        ((__nv_bfloat16*)a.y)[i] = __float2bfloat16_rn(a.ys ? a.ys[i] : 0.0f);
    }
  }
  __syncthreads();
  if (*abort_flag && tid == 0) {
    // a wait gave up: let the copies still in flight land before the CTA's shared memory is released
    const int f1 = *s_fills;
    for (int f = max(0, f1 - a.stages); f < f1; ++f)
      mbar_wait_drain(smem_u32(full_bar + f % a.stages), (uint32_t)(f / a.stages) & 1u);
  }
}

// Token-side scale blocks of the dense block-scaled GEMM, tile-major (tiling.cuh): one CTA per
// group-tile, one thread per row of its scale atoms.
__global__ void __launch_bounds__(256)
    linear_scale_tiles_kernel(const uint8_t* __restrict__ xs, int rows, int bn, int k_tiles, uint8_t* __restrict__ out) {
  griddep_wait();
  griddep_launch_dependents();
  const int gt = blockIdx.x, ntiles = (rows + bn - 1) / bn;
  const int n_per = tile_rows_per(rows, ntiles);
  const int n_valid = min(n_per, rows - gt * n_per);
  const int n = threadIdx.x;
  if (n_valid <= 0 || n >= ((((n_valid + 15) & ~15) + 127) >> 7) * 128) return;
  const bool valid = n < n_valid;
  const uint8_t* src = xs + (valid ? (size_t)(gt * n_per + n) * k_tiles * 4 : 0);
  uint8_t* dst = out + (size_t)gt * k_tiles * SF_TILE_BYTES + sf_atom_offset(n);
  for (int kt = blockIdx.y; kt < k_tiles; kt += gridDim.y)
    *(uint32_t*)(dst + (size_t)kt * SF_TILE_BYTES) = valid ? __ldg((const uint32_t*)(src + kt * 4)) : 0u;
}

// y = bf16(sum over s, in order, of part[s * stride + i])
__global__ void split_sum_bf16_kernel(const float* __restrict__ part, int nsplit, long long n, long long stride,
                                      __nv_bfloat16* __restrict__ y) {
  griddep_wait();
  griddep_launch_dependents();
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  float v = 0.0f;
  for (int s = 0; s < nsplit; ++s) v += __ldg(part + s * stride + i);
  y[i] = __float2bfloat16_rn(v);
}

}  // namespace moe
