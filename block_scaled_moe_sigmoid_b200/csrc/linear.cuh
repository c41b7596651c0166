// MXFP4 linear for more token rows than few.cuh takes: y = x W^T on tcgen05, whole tiles or split ones.
//
// A tile is 256 weight rows x up to NB token rows, its contraction K / 128 steps; a step loads 16 KB of
// codes (the tensor core reads E2M1 and E4M3 with one E8M0 scale per 32 elements) and the token rows.
// Up to 128 token rows make 28 or 56 tiles at N = 7168, and narrow outputs few at any length: too few for
// 148 SMs to take whole ones.  As in few.cuh the list of steps is then cut evenly, and fp32 partials are
// exchanged.  Here a second kernel adds them, in the order of the CTAs: a tile's partials are up to 176 KB
// each, and one CTA reading five of them takes longer than the products (39 us for 160 x 7168 x 7168,
// 19.5 with the second kernel).
//
// Bound, with tiles of up to 64 rows, by the issue of the MMAs and the weight stream (eight MMAs of 64
// columns take 384 of about 460 cycles a step), with higher ones by the rate at which shared memory fills.
// Measured (B200, weights from memory; in a short run, and without a pause): 7168 x 7168 with 64 rows
// 13.0 and 13.4 us, 300 rows 20.7 and 23.0, 1024 rows 50.2 and 59.8, 4096 rows 163 and 197 (2.6 and 2.1
// PFLOP/s).  Roles as in few.cuh, and warp 13, which makes the token
// scales' atoms.
#pragma once
#include "few.cuh"

namespace moe {

struct LinearArgs {
  int T, n_per, n_tiles;    // token rows, rows per token tile (a multiple of 16), token tiles
  int m_tiles, k_tiles;
  int N;
  int unit, ctas;           // steps that stay together (a whole tile, or 1), CTAs that share the units
  int per, rem;             // units per CTA; the first `rem` CTAs take one more
  const uint8_t* sf;        // weight scales [m-tile][k-tile][1 KB]
  const uint8_t* xs;        // token scales [T][4 k_tiles]
  void* y;
  int y_f32;
  float* part;              // [2 per CTA][n_per][256]
  unsigned int* status;
};
// First step of CTA c's part of the list, and the CTA with step s where a unit is one step.
__device__ __forceinline__ int linear_first_step(const LinearArgs& a, int c) { return (c * a.per + min(c, a.rem)) * a.unit; }
__device__ __forceinline__ int linear_cta_of(const LinearArgs& a, int s) {
  const int big = a.rem * (a.per + 1);
  return s < big ? s / (a.per + 1) : a.rem + (s - big) / a.per;
}

constexpr int kLinearThreads = kFewThreads + 32;   // few.cuh's roles, and warp 13

template <int NB>
struct LinearCfg {
  static constexpr int STAGES = NB > 64 ? 4 : 5;
  static constexpr int B_TILE = NB * 128;
  static constexpr int STAGE = kFewATile + B_TILE;
  static constexpr int SFB = NB > 128 ? 1024 : 512;
  static constexpr int SF = 1024 + SFB;
  static constexpr int CTRL = STAGES * (STAGE + SF);
  static constexpr int SMEM = CTRL + 512 + 1024;
  static constexpr int ACC_BUFS = 4 * NB + 16 * STAGES <= 512 ? 2 : 1;
  static constexpr int TMEM_SF = ACC_BUFS * 2 * NB;
  static_assert(STAGE % 1024 == 0 && NB % 16 == 0 && NB <= 256, "tile shape");
  static_assert(TMEM_SF + 16 * STAGES <= 512, "TMEM budget");
  static_assert(SMEM <= kFewSmemMax, "shared memory budget");
};

// V tokens' values of one output row, from row n of token tile nt on.
template <int V>
__device__ __forceinline__ void linear_store(const LinearArgs& a, int m, int nt, int n, int row, const float (&v)[V]) {
  const int o_row = m * 256 + row, t0 = nt * a.n_per + n;
  if (o_row >= a.N) return;
#pragma unroll
  for (int t = 0; t < V; ++t) {
    if (t0 + t >= a.T) break;
    const size_t o = (size_t)(t0 + t) * a.N + o_row;
    if (a.y_f32) ((float*)a.y)[o] = v[t];
    else ((__nv_bfloat16*)a.y)[o] = __float2bfloat16_rn(v[t]);
  }
}

template <int NB>
__global__ void __launch_bounds__(kLinearThreads, 1)
    linear_kernel(const __grid_constant__ LinearArgs a, const __grid_constant__ CUtensorMap tmW,
                  const __grid_constant__ CUtensorMap tmX) {
  using C = LinearCfg<NB>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sf = smem + STAGES * C::STAGE;
  uint64_t* full_bar = (uint64_t*)(smem + C::CTRL);
  uint64_t* empty_bar = full_bar + STAGES;
  uint64_t* sf_full = empty_bar + STAGES;
  uint64_t* acc_full = sf_full + STAGES;   // [2]
  uint64_t* acc_empty = acc_full + 2;      // [2]
  uint64_t* drain_bar = acc_empty + 2;
  uint64_t* drain_sf = drain_bar + 1;
  uint32_t* tmem_holder = (uint32_t*)(drain_sf + 1);
  volatile int* abort_flag = (volatile int*)(tmem_holder + 1);
  int* fills = (int*)(tmem_holder + 2);   // [6]: weight producer, token producer, scale warp, MMA halves, token scales

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(full_bar + s), 3);    // two producers, the scale warp's commit
      mbar_init(smem_u32(empty_bar + s), 2);   // both issuers
      mbar_init(smem_u32(sf_full + s), 2);     // the weights' scales, the tokens'
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(acc_full + b), 2);
      mbar_init(smem_u32(acc_empty + b), 8);
    }
    mbar_init(smem_u32(drain_bar), 2);
    mbar_init(smem_u32(drain_sf), 1);
    *abort_flag = 0;
    for (int r = 0; r < 6; ++r) fills[r] = 0;
    fence_mbar_init();
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  griddep_wait();
  griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_holder, 0);

  // this CTA's steps [s0, s1) of tiles x k_tiles; the token tiles of a weight tile follow one another
  const int KT = a.k_tiles, c = blockIdx.x;
  const int s0 = linear_first_step(a, c), s1 = linear_first_step(a, c + 1);
  struct Run { int m, nt, kb, n; };   // K tiles [kb, kb + n) of a tile
  auto run_at = [&](int s) {
    Run r;
    const int tile = s / KT;
    r.m = tile / a.n_tiles;
    r.nt = tile - r.m * a.n_tiles;
    r.kb = s - tile * KT;
    r.n = min(KT - r.kb, s1 - s);
    return r;
  };

  if (warp == 0) {
    // ------------------------------------------------------------- producer: weights
    if (lane == 0) {
      const uint64_t pol = policy_evict_first();
      int stage = 0, nfill = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int s = s0; s < s1 && ok;) {
        const Run r = run_at(s);
        const size_t blk = (size_t)r.m * KT + r.kb;
        for (int i = 0; i < r.n; ++i) {
          ok = mbar_wait(smem_u32(empty_bar + stage), phase ^ 1, a.status, abort_flag);
          if (!ok) break;
          const uint32_t sb = smem_u32(sf_full + stage), fb = smem_u32(full_bar + stage);
          mbar_arrive_expect_tx(sb, 1024);
          bulk_load(smem_u32(sf + stage * C::SF), a.sf + (blk + i) * 1024, 1024, sb);
          mbar_arrive_expect_tx(fb, kFewTile);
          tma_load_2d(smem_u32(smem + stage * C::STAGE), &tmW, fb, 0, (int)((blk + i) * 256), pol);
          ++nfill;
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
        s += r.n;
      }
      fills[0] = nfill;
    }
    __syncwarp();
  } else if (warp == 10) {
    // ------------------------------------------------------------- producer: token rows
    if (lane == 0) {
      const uint64_t pol = policy_evict_last();
      int stage = 0, nfill = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int s = s0; s < s1 && ok;) {
        const Run r = run_at(s);
        for (int i = 0; i < r.n; ++i) {
          ok = mbar_wait(smem_u32(empty_bar + stage), phase ^ 1, a.status, abort_flag);
          if (!ok) break;
          const uint32_t fb = smem_u32(full_bar + stage);
          mbar_arrive_expect_tx(fb, a.n_per * 128);   // the box: rows past T are zeros
          tma_load_2d(smem_u32(smem + stage * C::STAGE + kFewATile), &tmX, fb, (r.kb + i) * 128, r.nt * a.n_per, pol);
          ++nfill;
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
        s += r.n;
      }
      fills[1] = nfill;
    }
    __syncwarp();
  } else if (warp == 11) {
    // ------------------------------------------------------------- scale factors -> TMEM
    const uint64_t desc0 = smem_desc(smem_u32(sf), 16, 128, 0);
    const bool two = C::SFB > 512 && a.n_per > 128;
    int stage = 0, nfill = 0;
    uint32_t phase = 0;
    for (int s = s0; s < s1; ++s) {
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(sf_full + stage), phase, a.status, abort_flag))) break;
      ++nfill;
      tc_fence_after();
      const uint64_t desc = desc0 + (uint64_t)((stage * C::SF) >> 4);
      const uint32_t tsf = tmem_base + C::TMEM_SF + 16 * stage;
      if (elect_one()) {
        tc_cp_32x128b_warpx4(tsf, desc);
        tc_cp_32x128b_warpx4(tsf + 4, desc + (uint64_t)(512 >> 4));
        tc_cp_32x128b_warpx4(tsf + 8, desc + (uint64_t)(1024 >> 4));
        if (two) tc_cp_32x128b_warpx4(tsf + 12, desc + (uint64_t)(1536 >> 4));
        tc_commit(smem_u32(full_bar + stage));
      }
      __syncwarp();
      if (++stage == STAGES) { stage = 0; phase ^= 1; }
    }
    if (elect_one()) {
      tc_commit(smem_u32(drain_sf));   // every copy lands before TMEM is released
      mbar_wait_drain(smem_u32(drain_sf), 0);
      fills[2] = nfill;
    }
    __syncwarp();
  } else if (warp == 13) {
    // ------------------------------------------------------------- token scales
    // Each step's scale atoms, a word per token row (its four blocks of the K tile).  (In the warp above,
    // the stores would hold up the copies: 512 rows 34 us, not 28.)  A row's words of four K tiles are
    // loaded together, four steps ahead, where their 16 bytes are aligned: word by word the gather fetched
    // a sector per row and step.
    constexpr int WORDS = (NB + 31) / 32;
    const bool quads = KT % 4 == 0 && ((uintptr_t)a.xs & 15) == 0;
    uint4 cur[WORDS], next[WORDS];
    auto fetch = [&](uint4 (&q)[WORDS], const Run& r, int kt) {
#pragma unroll
      for (int w = 0; w < WORDS; ++w) {
        const int n = lane + 32 * w, t = r.nt * a.n_per + n;
        q[w] = make_uint4(0u, 0u, 0u, 0u);
        if (n < a.n_per && t < a.T) {
          const uint32_t* src = (const uint32_t*)a.xs + (size_t)t * KT + kt;
          if (quads) {
            q[w] = __ldg((const uint4*)src);
          } else {
            q[w].x = __ldg(src);
            if (kt + 1 < KT) q[w].y = __ldg(src + 1);
            if (kt + 2 < KT) q[w].z = __ldg(src + 2);
            if (kt + 3 < KT) q[w].w = __ldg(src + 3);
          }
        }
      }
    };
    int stage = 0, nfill = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int s = s0; s < s1 && ok;) {
      const Run r = run_at(s);
      fetch(next, r, r.kb & ~3);
      for (int kt = r.kb; kt < r.kb + r.n; ++kt) {
        if (kt == r.kb || (kt & 3) == 0) {
#pragma unroll
          for (int w = 0; w < WORDS; ++w) cur[w] = next[w];
          if ((kt & ~3) + 4 < r.kb + r.n) fetch(next, r, (kt & ~3) + 4);
        }
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(empty_bar + stage), phase ^ 1, a.status, abort_flag));
        if (!ok) break;
        uint8_t* atom = sf + stage * C::SF + 1024;
        const int j = kt & 3;
#pragma unroll
        for (int w = 0; w < WORDS; ++w)
          *(uint32_t*)(atom + sf_atom_offset(lane + 32 * w)) = j < 2 ? (j == 0 ? cur[w].x : cur[w].y) : (j == 2 ? cur[w].z : cur[w].w);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(sf_full + stage));
        ++nfill;
        if (++stage == STAGES) { stage = 0; phase ^= 1; }
      }
      s += r.n;
    }
    if (lane == 0) fills[5] = nfill;
  } else if (warp == 1 || warp == 12) {
    // ------------------------------------------------------------- MMA issuers, one per 128-row half
    const int h = warp == 12;
    const uint64_t desc0 = smem_desc(smem_u32(smem), 16, 1024, 2);
    uint32_t idesc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) idesc[j] = idesc_mx_e2m1_e4m3(128, a.n_per, j, j);
    int stage = 0, nfill = 0, nrun = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int s = s0; s < s1 && ok;) {
      const Run r = run_at(s);
      s += r.n;
      const int abuf = nrun % C::ACC_BUFS;
      const uint32_t acc_t = tmem_base + 2 * NB * abuf + NB * h;
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(acc_empty + abuf), (uint32_t)(nrun / C::ACC_BUFS & 1) ^ 1u, a.status, abort_flag));
      if (!ok) break;
      for (int i = 0; i < r.n; ++i) {
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(full_bar + stage), phase, a.status, abort_flag));
        if (!ok) break;
        tc_fence_after();
        const uint64_t a_desc = desc0 + (uint64_t)((stage * C::STAGE + h * 16384) >> 4);
        const uint64_t b_desc = desc0 + (uint64_t)((stage * C::STAGE + kFewATile) >> 4);
        const uint32_t tsf = tmem_base + C::TMEM_SF + 16 * stage;
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_mxf8f6f4(acc_t, a_desc + (uint64_t)((32 * j) >> 4), b_desc + (uint64_t)((32 * j) >> 4), idesc[j],
                         (tsf + 4 * h) | ((uint32_t)j << 30), (tsf + 8) | ((uint32_t)j << 30), i > 0 || j > 0);
          tc_commit(smem_u32(empty_bar + stage));
        }
        __syncwarp();
        ++nfill;
        if (++stage == STAGES) { stage = 0; phase ^= 1; }
      }
      if (!ok) break;
      if (elect_one()) tc_commit(smem_u32(acc_full + abuf));
      __syncwarp();
      ++nrun;
    }
    if (elect_one()) {
      tc_commit(smem_u32(drain_bar));   // every MMA has finished before TMEM is released
      mbar_wait_drain(smem_u32(drain_bar), 0);
      fills[3 + h] = nfill;
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- epilogue: a thread per weight row
    // (a wait that gives up does not leave the loop: all eight warps meet at the same barriers)
    const int q = warp & 3, half = (warp - 2) >> 2;
    const int row = half * 128 + q * 32 + lane;
    const int chunks = a.n_per >> 4;
    int nrun = 0;
    for (int s = s0; s < s1; ++nrun) {
      const Run r = run_at(s);
      s += r.n;
      const int abuf = nrun % C::ACC_BUFS;
      int ok = 1;
      if (lane == 0) ok = mbar_wait(smem_u32(acc_full + abuf), (uint32_t)(nrun / C::ACC_BUFS & 1), a.status, abort_flag);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      tc_fence_after();
      const uint32_t acc_t = tmem_base + 2 * NB * abuf + NB * half + ((uint32_t)(q * 32) << 16);
      const bool whole = r.n == KT;
      float* mine = a.part + (size_t)(2 * c + (r.kb == 0 ? 1 : 0)) * a.n_per * 256 + row;
      for (int ch = 0; ch < chunks; ++ch) {
        uint32_t u[16];
        tmem_ld16(acc_t + ch * 16, u);
        tmem_ld_wait();
        float v[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) v[t] = __uint_as_float(u[t]);
        if (whole) {
          linear_store(a, r.m, r.nt, ch * 16, row, v);
        } else {
#pragma unroll
          for (int t = 0; t < 16; ++t) __stcg(mine + (ch * 16 + t) * 256, v[t]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(smem_u32(acc_empty + abuf));
    }
  }
  __syncthreads();
  if (*abort_flag) {
    // a wait gave up: let the copies still in flight land before the CTA's shared memory is released
    if (tid == 0) {
      drain_ring(full_bar, STAGES, fills, 3, min(fills[3], fills[4]));
      const int sf_fills[2] = {fills[0], fills[5]};
      drain_ring(sf_full, STAGES, sf_fills, 2, fills[2]);
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// The partials of split tiles, added in the order of their CTAs: a CTA per (tile, 4 tokens), a thread
// per weight row, four CTAs' partials in flight.
__global__ void __launch_bounds__(256) linear_sum_kernel(const __grid_constant__ LinearArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int tile = blockIdx.x, n = 4 * blockIdx.y, row = threadIdx.x;
  const int t0 = tile * a.k_tiles;
  const int lo = linear_cta_of(a, t0), hi = linear_cta_of(a, t0 + a.k_tiles - 1);
  const int m = tile / a.n_tiles, nt = tile - m * a.n_tiles;
  if (lo == hi || nt * a.n_per + n >= a.T) return;   // one CTA had the whole tile and stored it
  const size_t slot = (size_t)a.n_per * 256;
  const float* p = a.part + 2 * lo * slot + n * 256 + row;
  float v[4] = {};
  for (int i = lo; i <= hi; i += 4, p += 8 * slot) {
    float u[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int t = 0; t < 4; ++t)
        u[j][t] = i + j <= hi ? __ldcg(p + (2 * j + (i + j == lo ? 1 : 0)) * slot + t * 256) : 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int t = 0; t < 4; ++t) v[t] += u[j][t];
  }
  linear_store(a, m, nt, n, row, v);
}

}  // namespace moe
